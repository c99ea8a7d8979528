// 4-bit weights with group scales: quantisation and its inverse.
//
// A weight is w[e][n][k] = (q - z) * s with one scale s and one zero point z for `group` (32, 64 or 128)
// consecutive columns of a row; without zero points z = 8.  Eight columns of a row are one 32-bit word:
// nibble i (0..3) holds column 2 i, nibble 4 + i column 2 i + 1, so that (word >> 4 i) & 0x000F000F puts two
// neighbouring columns into the halves of a register, the form the tensor cores' operands have.  Scales and
// zero points are [E][G][n] (rows adjacent): 16 rows of a group are one 32-byte sector.
//
//   symmetric:    s = up5(max |x| / 7),       q = clamp(rint(x / s), -8, 7) + 8
//   zero points:  lo = min(0, min x), hi = max(0, max x), s = up4((hi - lo) / 15),
//                 z = clamp(rint(-lo / s), 0, 15),  q = clamp(rint(x / s) + z, 0, 15)
// up5 / up4 is the next number with 5 / 4 significant bits: |q - z| <= 8 / <= 15 then makes (q - z) s a number
// of at most 8 significant bits, a bf16 exactly, and no product with these weights rounds them again.  It
// costs the step 2% / 5% of its width on average.
//
// Both kernels stream: a CTA covers 32 rows x 256 columns, a warp a row of it at a time (a word per lane), so
// that a group is 4, 8 or 16 neighbouring lanes (its extremes by shuffles) and the 32 rows' scales of a group
// leave as one 64-byte piece through shared memory.  No division per element: r = rint(x * (1 / s)) is put
// right by the remainder x - r s, which is exact in fp32 (r s has at most 9 significant bits and lies on x's
// grid or a coarser one).
#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace w4 {

constexpr int kRows = 32;   // rows of a CTA's tile
constexpr int kCols = 256;  // columns: a word (8 columns) per lane

// rint(x / s) exactly, ties to even: the product with the reciprocal is at most a step off
__device__ __forceinline__ float round_quotient(float x, float s, float inv, float half) {
    float r = rintf(x * inv);
    const float rem = fmaf(-r, s, x);
    const bool odd = (static_cast<int>(r) & 1) != 0;
    if (rem > half || (rem == half && odd)) r += 1.f;
    else if (rem < -half || (rem == -half && odd)) r -= 1.f;
    return r;
}

template <int DT, bool ZERO>
__global__ void __launch_bounds__(256) quantize_w4_kernel(const void* __restrict__ x, int64_t n, int k, int group, int G,
                                                          uint32_t* __restrict__ q, uint16_t* __restrict__ s,
                                                          uint8_t* __restrict__ z) {
    __shared__ uint16_t s_sh[kCols / 32][kRows];
    __shared__ uint8_t z_sh[kCols / 32][kRows];
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t e = blockIdx.y, r0 = (int64_t)blockIdx.x * kRows;  // expert, first row
    const int lanes = group >> 3;  // lanes of a group
    const int words = k >> 3;
    for (int c0 = 0; c0 < k; c0 += kCols) {
        const int col = c0 + 8 * lane;
        const bool in = col < k;
        float v[kRows / 8][8];
#pragma unroll
        for (int i = 0; i < kRows / 8; ++i) {
            const int64_t row = r0 + warp + 8 * i;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = 0.f;  // columns past the end take no part: 0 moves no extreme
            if (in && row < n) load8<DT>(x, (e * n + row) * k + col, v[i]);
        }
#pragma unroll
        for (int i = 0; i < kRows / 8; ++i) {
            const int64_t row = r0 + warp + 8 * i;
            uint32_t top = 0;  // |x| as bits: orders NaN above everything
            float lo = 0.f, hi = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                top = max(top, __float_as_uint(v[i][j]) & 0x7FFFFFFFu);
                if (ZERO) {
                    lo = fminf(lo, v[i][j]);
                    hi = fmaxf(hi, v[i][j]);
                }
            }
            for (int o = lanes >> 1; o > 0; o >>= 1) {
                top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                if (ZERO) {
                    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
                    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
                }
            }
            // the scale: the least number of BITS significant bits with STEPS * s >= range, decided exactly
            // (STEPS * s has at most 8 significant bits; the range is a sum of two floats, taken in double)
            constexpr int BITS = ZERO ? 4 : 5;
            constexpr float STEPS = ZERO ? 15.f : 7.f;
            constexpr uint32_t ULP = 1u << (24 - BITS);
            const double range = ZERO ? (double)hi - (double)lo : (double)__uint_as_float(top);
            const bool finite = top < 0x7B800000u;  // |x| < 2^120
            float sc = 1.f;
            if (top != 0 && finite) {
                const float t = (float)range * (1.f / STEPS);  // within 2 ulp
                uint32_t b = (__float_as_uint(t) + ULP - 1) & ~(ULP - 1);
                while ((double)(STEPS * __uint_as_float(b)) < range) b += ULP;
                while (b > ULP && (double)(STEPS * __uint_as_float(b - ULP)) >= range) b -= ULP;
                sc = fmaxf(__uint_as_float(b), 0x1p-100f);
            }
            const float inv = 1.f / sc, half = 0.5f * sc;
            float zp = 8.f;
            if (ZERO) zp = finite ? fminf(fmaxf(round_quotient(-lo, sc, inv, half), 0.f), 15.f) : 8.f;
            uint32_t word = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float r = 0.f;
                if (finite) r = round_quotient(v[i][j], sc, inv, half);
                const int code = static_cast<int>(fminf(fmaxf(r + zp, 0.f), 15.f));
                word |= (uint32_t)code << (4 * (j / 2 + 4 * (j & 1)));
            }
            if (in && row < n) q[(e * n + row) * words + (col >> 3)] = word;
            if ((lane & (lanes - 1)) == 0) {
                // a value that is not finite (or >= 2^120) makes its group's scale NaN: it shows in every product
                s_sh[lane / lanes][warp + 8 * i] = finite ? (uint16_t)f32_to_bf16_bits(sc) : (uint16_t)0x7FC0u;
                if (ZERO) z_sh[lane / lanes][warp + 8 * i] = (uint8_t)static_cast<int>(zp);
            }
        }
        __syncthreads();
        const int ng = kCols / group, g0 = c0 / group;
        for (int i = threadIdx.x; i < ng * kRows; i += blockDim.x) {
            const int g = i / kRows, r = i % kRows;
            if (g0 + g < G && r0 + r < n) {
                const int64_t at = (e * G + g0 + g) * n + r0 + r;
                s[at] = s_sh[g][r];
                if (ZERO) z[at] = z_sh[g][r];
            }
        }
        __syncthreads();
    }
}

template <int DT, bool ZERO>
__global__ void __launch_bounds__(256) dequantize_w4_kernel(const uint32_t* __restrict__ q, const uint16_t* __restrict__ s,
                                                            const uint8_t* __restrict__ z, int64_t n, int k, int group,
                                                            int G, void* __restrict__ out) {
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t e = blockIdx.y, r0 = (int64_t)blockIdx.x * kRows;
    const int words = k >> 3;
    for (int c0 = 0; c0 < k; c0 += kCols) {
        const int col = c0 + 8 * lane;
        if (col >= k) continue;
#pragma unroll
        for (int i = 0; i < kRows / 8; ++i) {
            const int64_t row = r0 + warp + 8 * i;
            if (row >= n) continue;
            const uint32_t word = __ldg(q + (e * n + row) * words + (col >> 3));
            const int64_t at = (e * G + col / group) * n + row;
            const float sc = bf16_bits_to_f32(__ldg(s + at));
            const float zp = ZERO ? (float)__ldg(z + at) : 8.f;
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = ((float)((word >> (4 * (j / 2 + 4 * (j & 1)))) & 15u) - zp) * sc;
            store8<DT>(out, (e * n + row) * k + col, v);
        }
    }
}

}  // namespace w4

cudaError_t launch_quant_w4(const Ctx& c, const void* x, int dt, int E, int64_t n, int k, int group, uint8_t* q,
                            uint16_t* s, uint8_t* z) {
    const dim3 grid((unsigned)((n + w4::kRows - 1) / w4::kRows), (unsigned)E);
    const int G = (k + group - 1) / group;
    uint32_t* qw = reinterpret_cast<uint32_t*>(q);
    if (dt == DT_BF16) {
        if (z) return launch(w4::quantize_w4_kernel<DT_BF16, true>, grid, dim3(256), 0, c, x, n, k, group, G, qw, s, z);
        return launch(w4::quantize_w4_kernel<DT_BF16, false>, grid, dim3(256), 0, c, x, n, k, group, G, qw, s, z);
    }
    if (z) return launch(w4::quantize_w4_kernel<DT_F32, true>, grid, dim3(256), 0, c, x, n, k, group, G, qw, s, z);
    return launch(w4::quantize_w4_kernel<DT_F32, false>, grid, dim3(256), 0, c, x, n, k, group, G, qw, s, z);
}

cudaError_t launch_dequant_w4(const Ctx& c, const uint8_t* q, const uint16_t* s, const uint8_t* z, int E, int64_t n, int k,
                              int group, void* out, int dt) {
    const dim3 grid((unsigned)((n + w4::kRows - 1) / w4::kRows), (unsigned)E);
    const int G = (k + group - 1) / group;
    const uint32_t* qw = reinterpret_cast<const uint32_t*>(q);
    if (dt == DT_BF16) {
        if (z) return launch(w4::dequantize_w4_kernel<DT_BF16, true>, grid, dim3(256), 0, c, qw, s, z, n, k, group, G, out);
        return launch(w4::dequantize_w4_kernel<DT_BF16, false>, grid, dim3(256), 0, c, qw, s, z, n, k, group, G, out);
    }
    if (z) return launch(w4::dequantize_w4_kernel<DT_F32, true>, grid, dim3(256), 0, c, qw, s, z, n, k, group, G, out);
    return launch(w4::dequantize_w4_kernel<DT_F32, false>, grid, dim3(256), 0, c, qw, s, z, n, k, group, G, out);
}

}  // namespace moe
