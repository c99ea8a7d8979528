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
// Both kernels stream, a warp per row and 256 columns at a time (a word per lane; kAhead such pieces in flight), so
// that a group is 4, 8 or 16 neighbouring lanes and its extremes are shuffles.  The scales of neighbouring rows are
// neighbours in memory: a CTA's 8 rows, and the next CTA's, meet in L2 sectors.  Memory should bound both; per
// element there is no division and no conversion: t = x * (1 / s) + 1.5 * 2^23 has the rounded quotient in its
// low bits, and the remainder x - r s, which is exact in fp32 (r s has at most 9 significant bits and lies on x's
// grid or a coarser one), moves it by a step where 1 / s was not exact enough, and ties to even.
#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace w4 {

constexpr int kWarps = 8;   // rows of a CTA
constexpr int kCols = 256;  // columns of a piece: a word (8 columns) per lane
constexpr int kAhead = 4;  // pieces in flight

// Offset by 0x4B400000: rint(x / s) exactly, ties to even.  half_bits: those of s / 2.
__device__ __forceinline__ int round_quotient(float x, float s, float inv, uint32_t half_bits) {
    const float t = fmaf(x, inv, 12582912.f);  // a step off at most
    int r = __float_as_int(t);
    const float rem = fmaf(12582912.f - t, s, x);
    // past a half: a step towards x; on it: that step where r is odd (above the number before the half)
    if (fabsf(rem) > __uint_as_float(half_bits - (r & 1))) r += (__float_as_int(rem) >> 31) | 1;
    return r;
}

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

template <int DT, bool ZERO>
__global__ void __launch_bounds__(32 * kWarps) quantize_w4_kernel(const void* __restrict__ x, int64_t n, int k, int group,
                                                                  int G, uint32_t* __restrict__ q,
                                                                  uint16_t* __restrict__ s, uint8_t* __restrict__ z) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t e = blockIdx.y, row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (row >= n) return;
    const int lanes = group >> 3, lg = __ffs(group) - 1;  // lanes of a group; its size is a power of two
    const int64_t in = (e * n + row) * k;
    uint32_t* out = q + (in >> 3);
    for (int c0 = 8 * lane; c0 < k + 8 * lane; c0 += kAhead * kCols) {
        float vv[kAhead][8];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
#pragma unroll
            for (int j = 0; j < 8; ++j) vv[i][j] = 0.f;  // columns past the end take no part: 0 moves no extreme
            if (c0 + i * kCols < k) load8<DT>(x, in + c0 + i * kCols, vv[i]);
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int col = c0 + i * kCols;
            float(&v)[8] = vv[i];
            // extremes of the group, negated where they are low; a NaN stays
            float hi = 0.f, low = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                hi = max_nan(hi, ZERO ? v[j] : fabsf(v[j]));
                if (ZERO) low = max_nan(low, -v[j]);
            }
            for (int o = lanes >> 1; o > 0; o >>= 1) {
                hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
                if (ZERO) low = max_nan(low, __shfl_xor_sync(0xffffffffu, low, o));
            }
            // the scale: the least number of BITS significant bits with STEPS * s >= range, decided exactly
            // (STEPS * s has at most 8 significant bits, so it compares with the rounded range as with the exact
            // one, but for equality)
            constexpr int BITS = ZERO ? 4 : 5;
            constexpr float STEPS = ZERO ? 15.f : 7.f;
            constexpr uint32_t ULP = 1u << (24 - BITS);
            const float range = ZERO ? hi + low : hi;
            const bool finite = hi < 0x1p120f && low < 0x1p120f;
            auto covers = [&](uint32_t b) {
                const float c = STEPS * __uint_as_float(b);
                return ZERO && c == range ? (double)c >= (double)hi + (double)low : c >= range;
            };
            float sc = 1.f;
            if (range != 0.f && finite) {
                uint32_t b = (__float_as_uint(range * (1.f / STEPS)) + ULP - 1) & ~(ULP - 1);  // a step off at most
                if (!covers(b)) b += ULP;
                else if (b > ULP && covers(b - ULP)) b -= ULP;
                sc = fmaxf(__uint_as_float(b), 0x1p-100f);
            }
            const float inv = __fdividef(1.f, sc);
            const uint32_t half = __float_as_uint(0.5f * sc);
            int zp = 8;
            if (ZERO && finite) zp = min(max(round_quotient(low, sc, inv, half) - 0x4B400000, 0), 15);
            // (without zero points the codes are 1..15, as 7 s covers the range: their offsets add up to a constant)
            uint32_t word = ZERO ? 0u : (8u - 0x4B400000u) * 0x11111111u;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int r = round_quotient(v[j], sc, inv, half);
                const uint32_t code = ZERO ? (uint32_t)min(max(r - 0x4B400000 + zp, 0), 15) : (uint32_t)r;
                word += code << (4 * (j / 2 + 4 * (j & 1)));
            }
            if (!finite) word = 0x88888888u;
            if (col < k) {
                out[col >> 3] = word;
                if ((lane & (lanes - 1)) == 0) {
                    const int64_t at = (e * G + (col >> lg)) * n + row;
                    // a value that is not finite (or >= 2^120) makes its group's scale NaN: it shows in every product
                    s[at] = finite ? (uint16_t)f32_to_bf16_bits(sc) : (uint16_t)0x7FC0u;
                    if (ZERO) z[at] = (uint8_t)zp;
                }
            }
        }
    }
}

template <int DT, bool ZERO>
__global__ void __launch_bounds__(32 * kWarps) dequantize_w4_kernel(const uint32_t* __restrict__ q,
                                                                    const uint16_t* __restrict__ s,
                                                                    const uint8_t* __restrict__ z, int64_t n, int k,
                                                                    int group, int G, void* __restrict__ out) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t e = blockIdx.y, row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (row >= n) return;
    const int64_t at0 = (e * n + row) * k;
    const int lg = __ffs(group) - 1;
    constexpr int C = DT == DT_F32 ? 4 : 8;  // columns of a lane: 16 bytes of output, so that a warp's stores are whole lines
    for (int c0 = C * lane; c0 < k; c0 += kAhead * 32 * C) {
        uint32_t word[kAhead];
        uint16_t sc[kAhead];
        uint8_t zp[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int col = c0 + i * 32 * C;
            word[i] = 0;
            sc[i] = 0;
            zp[i] = 8;
            if (col < k) {
                word[i] = __ldg(q + ((at0 + col) >> 3)) >> (col & 4 ? 8 : 0);  // (columns 4..7 lie 8 bits on)
                const int64_t at = (e * G + (col >> lg)) * n + row;
                sc[i] = __ldg(s + at);
                if (ZERO) zp[i] = __ldg(z + at);
            }
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int col = c0 + i * 32 * C;
            if (col >= k) break;
            // 2^23 + code has the code in its low bits
            const float f = bf16_bits_to_f32(sc[i]), base = 8388608.f + (float)zp[i];
            float v[C];
#pragma unroll
            for (int j = 0; j < C; ++j)
                v[j] = (__uint_as_float(0x4B000000u | ((word[i] >> (4 * (j / 2 + 4 * (j & 1)))) & 15u)) - base) * f;
            if constexpr (C == 4)
                *reinterpret_cast<float4*>(static_cast<float*>(out) + at0 + col) = make_float4(v[0], v[1], v[2], v[3]);
            else store8<DT>(out, at0 + col, v);
        }
    }
}

}  // namespace w4

cudaError_t launch_quant_w4(const Ctx& c, const void* x, int dt, int E, int64_t n, int k, int group, uint8_t* q,
                            uint16_t* s, uint8_t* z) {
    const dim3 grid((unsigned)((n + w4::kWarps - 1) / w4::kWarps), (unsigned)E);
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
    const dim3 grid((unsigned)((n + w4::kWarps - 1) / w4::kWarps), (unsigned)E);
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
