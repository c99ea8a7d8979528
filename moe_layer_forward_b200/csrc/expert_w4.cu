// 4-bit experts for few rows per expert: a stream of weights past a handful of token rows.
//
//   gate/up   h[r] = SiLU(Wg x[r]) * (Wu x[r])       down   y[r] = Wd h[r],      w = (q - z) * s
//
// Two kernels around the same stream:
//   stream_w4_kernel  one product over expert-contiguous rows (counts, offsets as written by the permutation),
//                     optionally read through a slot -> token map
//   picks_w4_kernel   gate/up, down and the weighted sum in one cooperative launch, straight from the router's
//                     picks topk_idx [T][k] (T k <= 256): every CTA sorts the picks by expert itself, so a token
//                     needs no permutation and no permuted copy.  h and y are fp32: the form for single tokens
//                     loses nothing between the router and the output.  While a CTA waits for the others' h, its
//                     first weights of down are on their way already.
//
// What bounds it: the weights' bytes.  At 6.5 TB/s each SM has to take 23 bytes, 46 weights, per clock, so every
// step is counted in instructions per weight.  Unpacking to bf16 and scaling there takes 2 per weight and left
// the stream issue-bound at a quarter of the bandwidth (gate/up of 128 tokens, 8 rows per expert: 486 us).
//
// The products therefore run on the codes as they are: masking a word's low and its high nibbles gives eight
// unsigned bytes in three instructions, and mma.sync m16n8k32 on bytes (32-bit sums, exact) takes them straight
// from registers at twice the multiply-adds of the bf16 form (measured 1950 against 990 per clock and SM; the E4M3
// form is no instruction of its own here: it converts both operands first).  The wide tensor cores would want
// the weights in shared or tensor memory, a round trip that pays only for many rows (expert_w4_tc.cu).
//
// The token rows are the operand that is split: per group of columns, a power of two c takes the largest
// magnitude to 2 or 3 signed bytes, X = rint(x c) = 256 x1 + x0 (or 65536 x2 + 256 x1 + x0), and every byte is a
// set of columns of the product.  Two bytes round a group's rows to 2^-15 of its largest value, a hundredth
// of what rounding the output to bf16 does; three, for fp32 outputs, to 2^-23.  Scale and zero point come
// after the group's integer sum P:  y += s / c * (P - z * sum X).
//
// Layout.  A unit is 16 weight rows over the whole K: 8 gate and the 8 up rows of the same features (then the
// accumulators of a thread hold g and u of the same element), or 16 rows of down.  Warps are independent: each
// streams its units through a ring of its own (cp.async, 256 columns a stage), with no barrier between warps.
// Thread (g, t) = (lane / 4, lane % 4) takes GP = group / 32 consecutive words of every group of rows g and
// g + 8, word t GP + i in MMA i: any order of K will do as long as A and B agree, and the token rows are stored
// in the order that masking gives (columns 0 4 1 5 | 2 6 3 7 of a word).  16-byte pieces are swizzled with the
// row times GP so that those reads meet no bank twice.  The units of all experts form one list, cut evenly over
// the CTAs; a CTA stages the token rows of the experts its share touches, as many experts at a time as fit.
// The 8 columns of an MMA are one byte of 8 token rows; up to 4 rows (2 with three bytes) share a single MMA.
#include <cooperative_groups.h>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace w4s {

constexpr int kWarps = 16;
constexpr int kThreads = 32 * kWarps;
constexpr int kStages = 4;
constexpr int kStageCols = 256;
// a warp's ring: kStages pieces of 16 rows x 128 bytes of codes; the scales and zero points of the same stages
constexpr int kCodeBytes = 16 * (kStageCols / 2);
constexpr int kZeroOff = (kStageCols / 32) * 32;              // [group][16 rows] bf16, then [group][16 rows] u8
constexpr int kScaleBytes = kZeroOff + (kStageCols / 32) * 16;
constexpr int kScales = kWarps * kStages * kCodeBytes;
constexpr int kRingBytes = kScales + kWarps * kStages * kScaleBytes;
constexpr int kSmemLimit = 232448;
constexpr int kMaxPicks = 256;
constexpr int kListed = 512;
constexpr int kMaxRows = 32 * 8;  // staged rows: 32 chunks of at most 8
static_assert(kThreads >= kMaxPicks, "a thread per pick");

// one product over the experts' rows
struct Phase {
    const uint8_t* q0;  // gate (rows 0..7 of a unit) or down
    const uint8_t* q1;  // up (rows 8..15) or down
    const uint16_t* s0;
    const uint16_t* s1;
    const uint8_t* z0;
    const uint8_t* z1;
    const void* x;  // token rows [rows][K]: bf16, or (down of picks) fp32
    void* out;      // [rows][n_out]: bf16, or (picks) fp32
    int K, n_out, G;
    int xcap;      // token rows that fit in shared memory
    int x_stride;  // bytes of a staged row
};

struct Args {
    Phase ph[2];             // gate/up, down (segments: ph[0] alone, either of them)
    const int32_t* gather;   // segments: slot i reads row gather[i] of act_rows rows
    const int32_t* counts;   // segments
    const int32_t* offsets;  // segments
    const int32_t* picks;    // picks: topk_idx
    const float* weights;    // picks: topk_w
    const void* residual;    // picks
    void* out;               // picks
    int32_t* status;
    int P;  // picks: T k;  segments: rows of the buffers
    int top_k;
    int act_rows;
    int E;
    int chunk_rows;  // token rows of one pass over an expert's weights (<= 8)
    int r_dt, out_dt;
};

struct Aux {
    int vstart[kMaxExperts + 1];  // chunks before expert e
    uint8_t chunk_e[kListed];     // expert of chunk v, for the first of them
    int cnt[kMaxExperts];
    int off[kMaxExperts];
    int16_t order[kMaxPicks];  // picks sorted by expert, stable
    int16_t id[kMaxPicks];
    // the current batch's chunks: expert, first row, rows, first staged row
    int b_n;
    int be[32], bfirst[32], bn[32], brow[32];
    int src[kMaxRows];  // input row of a staged row
};
constexpr int kAuxBytes = (sizeof(Aux) + 127) & ~127;

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp8(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void mma(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    asm("mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// two fp32 operations in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(r)
        : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)),
          "l"(*reinterpret_cast<uint64_t*>(&c)));
    return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
    return *reinterpret_cast<float2*>(&r);
}

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
    return *reinterpret_cast<float2*>(&r);
}

template <bool V>
struct Bool {
    static constexpr bool value = V;
};

constexpr int kMagic = 0x4B400000;  // the bits of 1.5 * 2^23: plus an integer below 2^22 they are that number's sum

// four signed bytes, lowest first, of the low bytes of four integers
__device__ __forceinline__ uint32_t bytes4(int a, int b, int c, int d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

__device__ __forceinline__ int meta_rows(int xcap) { return (xcap + 1) & ~1; }

// chunks before every expert, and (picks) the rows before it; one warp
template <bool PICKS>
__device__ __forceinline__ void expert_prefixes(Aux& aux, int E, int chunk_rows, int lane) {
    int loc[8], cnt[8], sum = 0, rsum = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int e = lane * 8 + i;
        cnt[i] = e < E ? aux.cnt[e] : 0;
        loc[i] = (cnt[i] + chunk_rows - 1) / chunk_rows;
        sum += loc[i];
        rsum += cnt[i];
    }
    int incl = sum, rincl = rsum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int n = __shfl_up_sync(0xffffffffu, incl, o), r = __shfl_up_sync(0xffffffffu, rincl, o);
        if (lane >= o) {
            incl += n;
            rincl += r;
        }
    }
    int run = incl - sum, rrun = rincl - rsum;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int e = lane * 8 + i;
        if (e < E) {
            aux.vstart[e] = run;
            if (PICKS) aux.off[e] = rrun;
            for (int v = run; v < run + loc[i] && v < kListed; ++v) aux.chunk_e[v] = (uint8_t)e;
        }
        run += loc[i];
        rrun += cnt[i];
    }
    if (lane == 31) aux.vstart[E] = incl;
}

// 8 values of a token row; h of the picks was written by other CTAs of the same launch
template <bool F32X>
__device__ __forceinline__ void load_row8(const void* x, int64_t at, float (&v)[8]) {
    if constexpr (F32X) {
        const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(x) + at);
        const float4 a = __ldcg(q), b = __ldcg(q + 1);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        load8<DT_BF16>(x, at, v);
    }
}

// One product.  TM: bytes of a token row's value.  GP: 32-column pieces of a group.  before_rows() is called once,
// by all threads, when the first weights are on their way and before the first token row is read.
template <bool SWIGLU, bool PICKS, int TM, int GP, bool ZERO, class Hook>
__device__ __forceinline__ void stream(const Args& args, const Phase& p, uint8_t* smem, Hook before_rows) {
    constexpr bool F32X = PICKS && !SWIGLU;  // token rows are fp32
    constexpr int GROUP = 32 * GP;
    constexpr int NG = kStageCols / GROUP;  // groups of a stage
    Aux& aux = *reinterpret_cast<Aux*>(smem + kRingBytes);
    // [G][rows] 1 / c, then per byte [G][rows] where the group's integer sum starts (without zero points: kMagic - 8
    // times the sum of the byte; with them: the sum)
    const int mrows = meta_rows(p.xcap);
    float* meta = reinterpret_cast<float*>(smem + kRingBytes + kAuxBytes);
    const int mplane = p.G * mrows;
    uint8_t* xs = smem + kRingBytes + kAuxBytes + (((1 + TM) * mplane * 4 + 15) & ~15);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int E = args.E;

    constexpr int UROWS = SWIGLU ? 8 : 16;  // output columns of a unit
    const int nu = p.n_out / UROWS;         // units of one pass over an expert
    // units of all experts (few rows: far below 2^31), cut evenly
    const int total = aux.vstart[E] * nu, share = total / (int)gridDim.x, rest = total - share * (int)gridDim.x;
    const int u_begin = (int)blockIdx.x * share + min((int)blockIdx.x, rest);
    const int u_end = u_begin + share + ((int)blockIdx.x < rest ? 1 : 0);
    const int nstage = (p.K + kStageCols - 1) / kStageCols;
    const int pieces = p.K / 32;  // 32-column pieces of a row
    const int KP = p.G * GROUP;   // columns of a staged row: zeros past K
    const int g = lane >> 2, t = lane & 3;

    // expert and first row of chunk v
    auto find = [&](int v, int& e, int& first, int& n) {
        if (v < kListed) {
            e = aux.chunk_e[v];
        } else {
            int lo = 0, hi = E - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (aux.vstart[mid] <= v) lo = mid; else hi = mid - 1;
            }
            e = lo;
        }
        first = (v - aux.vstart[e]) * args.chunk_rows;
        n = min(args.chunk_rows, aux.cnt[e] - first);
    };

    bool hooked = false;
    for (int b0 = u_begin; b0 < u_end;) {
        // ---- a batch: the chunks from the current one on whose rows fit together (32 at most)
        const int v0 = b0 / nu;
        __syncthreads();  // the last batch's rows and table have been read
        if (warp == 0) {
            const int v = v0 + lane;
            int e = 0, first = 0, n = 0;
            const bool in = v < aux.vstart[E] && v * nu < u_end;
            if (in) find(v, e, first, n);
            const int even = (n + 1) & ~1;  // chunks start at even rows: two rows' meta is one read
            int incl = even;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int m = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += m;
            }
            aux.be[lane] = e;
            aux.bfirst[lane] = first;
            aux.bn[lane] = n;
            aux.brow[lane] = incl - even;
            const uint32_t fit = __ballot_sync(0xffffffffu, in && incl - even + n <= p.xcap);
            if (lane == 0) aux.b_n = __popc(fit);  // a prefix of the lanes; one chunk always fits
        }
        __syncthreads();
        const int nv = aux.b_n;
        const int base_u = b0 - v0 * nu;  // units are counted from chunk v0's first
        const int end_u = min(u_end, (v0 + nv) * nu) - v0 * nu;

        // ---- this warp's units (base + warp, + kWarps, ...): the copies run kStages - 1 stages ahead
        int iu = base_u + warp, ist = 0, islot = 0;
        // this lane's share of a stage: piece lane % 8 of rows lane / 8 + 4 j, and a scale and zero point piece
        const uint8_t* src[4] = {};
        const uint8_t* zp = nullptr;
        const uint16_t* sp = nullptr;
        const int r0 = lane >> 3;
        uint32_t dst_c = smem_addr(smem) + warp * kStages * kCodeBytes + r0 * 128;
        uint32_t dst_s = smem_addr(smem) + kScales + warp * kStages * kScaleBytes;
        const uint32_t at0 = ((lane & 7) ^ ((r0 * GP) & 7)) << 4, at1 = at0 ^ (GP == 1 ? 64u : 0u);  // rows 4 j + r0: j even, odd
        auto issue_next = [&]() {
            if (iu < end_u) {
                if (ist == 0) {
                    const int v = iu / nu, un = iu - v * nu;
                    const int64_t e = aux.be[v];
                    const int64_t row = e * p.n_out + un * UROWS + r0;
                    src[0] = p.q0 + row * (p.K / 2) + (lane & 7) * 16;
                    src[2] = SWIGLU ? p.q1 + row * (p.K / 2) + (lane & 7) * 16 : src[0] + 4 * (int64_t)p.K;
                    src[1] = src[0] + 2 * p.K;
                    src[3] = src[2] + 2 * p.K;
                    const int64_t at = (e * p.G + (lane >> 1)) * p.n_out + un * UROWS + (SWIGLU ? 0 : 8 * (lane & 1));
                    sp = (SWIGLU && (lane & 1) ? p.s1 : p.s0) + at;
                    if (ZERO) zp = (SWIGLU && (lane & 1) ? p.z1 : p.z0) + at;
                }
                if (ist * 8 + (lane & 7) < pieces) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) cp16(dst_c + islot * kCodeBytes + j * 512 + (j & 1 ? at1 : at0), src[j]);
                }
                if (lane < 2 * NG && ist * NG + (lane >> 1) < p.G) {
                    cp16(dst_s + islot * kScaleBytes + lane * 16, sp);
                    if (ZERO) cp8(dst_s + islot * kScaleBytes + kZeroOff + lane * 8, zp);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) src[j] += kStageCols / 2;
                sp += NG * p.n_out;
                if (ZERO) zp += NG * p.n_out;
                if (++islot == kStages) islot = 0;
                if (++ist == nstage) {
                    ist = 0;
                    iu += kWarps;
                }
            }
            cp_commit();  // a group per step, empty ones too: the waits count groups
        };
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) issue_next();

        if (!hooked) {
            before_rows();
            hooked = true;
        }
        // ---- stage the batch's token rows as bytes: a warp per (row, 256 columns), a lane per word of 8 columns;
        // the loads of several such pieces are in flight together
        const int all_rows = aux.brow[nv - 1] + aux.bn[nv - 1];
        for (int r = tid; r < all_rows; r += kThreads) {
            int ci = 0;
            while (ci + 1 < nv && aux.brow[ci + 1] <= r) ++ci;
            const int rr = r - aux.brow[ci];
            int src = -1;  // the spare row after an odd chunk
            if (rr < aux.bn[ci]) {
                src = aux.off[aux.be[ci]] + aux.bfirst[ci] + rr;
                if constexpr (PICKS) {
                    const int pick = aux.order[src];
                    src = F32X ? pick : pick / args.top_k;
                } else if (args.gather) {
                    src = args.gather[src];
                    if (src < 0 || src >= args.act_rows) {
                        set_status(args.status, DEV_BAD_COUNT);
                        src = 0;
                    }
                }
            }
            aux.src[r] = src;
        }
        __syncthreads();
        const int blocks = (KP + 255) >> 8, items = all_rows * blocks;
        constexpr int kAhead = F32X ? 2 : 4;
        for (int it0 = warp; it0 < items; it0 += kAhead * kWarps) {
            float vv[kAhead][8];
            int rows[kAhead], cols[kAhead];
#pragma unroll
            for (int q = 0; q < kAhead; ++q) {
                const int it = it0 + q * kWarps;
                rows[q] = it / blocks;
                cols[q] = (it - rows[q] * blocks) * 256 + lane * 8;
#pragma unroll
                for (int j = 0; j < 8; ++j) vv[q][j] = 0.f;
                const int src = it < items ? aux.src[rows[q]] : -1;
                if (src < 0) rows[q] = -1;
                else if (cols[q] < p.K) load_row8<F32X>(p.x, (int64_t)src * p.K + cols[q], vv[q]);
            }
#pragma unroll
            for (int q = 0; q < kAhead; ++q) {
                const int r = rows[q], c = cols[q];
                if (r < 0) continue;
                float(&v)[8] = vv[q];
                uint8_t* dst = xs + r * p.x_stride;
                uint32_t top = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(v[j]) & 0x7FFFFFFFu);
#pragma unroll
                for (int o = 2 * GP; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                // c = 2^k: |X| <= 1.984375 * 2^14 (2^22 with three bytes) = 127 * 256, whose signed bytes all fit; k is
                // one less where the top value is more than 1.984375 times a power of two
                int k = (TM == 2 ? 14 : 22) - ((int)(top >> 23) - 127) - ((top & 0x7FFFFFu) > 0x7E0000u ? 1 : 0);
                k = max(-118, min(100, k));
                const float cs = __uint_as_float((uint32_t)(127 + k) << 23);
                // a value that is not finite shows in every output of its row
                const bool finite = top < 0x7F800000u;
                const float inv = finite ? __uint_as_float((uint32_t)(127 - k) << 23) : __uint_as_float(0x7FC00000u);
                int X[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) X[j] = finite ? __float2int_rn(v[j] * cs) : 0;
                const bool in = c < KP, first = in && (lane & (4 * GP - 1)) == 0;
                float* m = meta + (c / GROUP) * mrows + r;
                if (first) m[0] = inv;
                int sums[2] = {0, 0};  // two bytes' sums to a register: below 2^15 in magnitude
#pragma unroll
                for (int i = 0; i < TM; ++i) {  // the lowest byte, signed, then what it leaves
                    uint2 w;                    // columns 0 4 1 5 | 2 6 3 7
                    w.x = bytes4(X[0], X[4], X[1], X[5]);
                    w.y = bytes4(X[2], X[6], X[3], X[7]);
                    if (in) *reinterpret_cast<uint2*>(dst + i * KP + c) = w;
                    sums[i / 2] += __dp4a((int)w.x, 0x01010101, __dp4a((int)w.y, 0x01010101, 0)) * (i % 2 ? 65536 : 1);
#pragma unroll
                    for (int j = 0; j < 8; ++j) X[j] = (X[j] + 128) >> 8;
                }
#pragma unroll
                for (int o = 2 * GP; o > 0; o >>= 1)
#pragma unroll
                    for (int i = 0; i < (TM + 1) / 2; ++i) sums[i] += __shfl_xor_sync(0xffffffffu, sums[i], o);
                if (first)
#pragma unroll
                    for (int i = 0; i < TM; ++i) {
                        const int low = (int)(int16_t)(sums[i / 2] & 0xFFFF);
                        const int sum = i % 2 ? (sums[i / 2] - low) >> 16 : low;
                        m[(1 + i) * mplane] = __int_as_float(ZERO ? sum : kMagic - 8 * sum);
                    }
            }
        }
        __syncthreads();

        int slot = 0;
        // one unit with its n token rows.  PACKED: the 8 columns hold all bytes of up to PR rows (column = byte * PR
        // + row); else they are 8 rows and every byte is a product of its own.
        auto unit = [&](auto packed_c, int u) {
            constexpr bool PACKED = decltype(packed_c)::value;
            constexpr int PR = 8 / TM;              // rows of a packed product
            constexpr int BYTES = PACKED ? 1 : TM;  // products
            const int v = u / nu, un = u - v * nu;
            const int e = aux.be[v], first = aux.bfirst[v], n = aux.bn[v], xrow = aux.brow[v];
            // [0]: weight row g, [1]: row g + 8; the pair: columns 2 t, 2 t + 1
            float2 acc[2];
            acc[0] = acc[1] = make_float2(0.f, 0.f);
            // this lane's column of B and its two columns of the sums (rows past the chunk repeat others of it)
            const uint8_t* xg = xs + (xrow + min(PACKED ? g % PR : g, n - 1)) * p.x_stride + t * (8 * GP) +
                                (PACKED ? min(g / PR, TM - 1) * KP : 0);
            const float* mg = meta + xrow + min(PACKED ? (2 * t) % PR : 2 * t, (n - 1) & ~1);
            const int mc = (1 + (PACKED ? min(2 * t / PR, TM - 1) : 0)) * mplane;
            for (int st = 0; st < nstage; ++st) {
                cp_wait<kStages - 2>();
                __syncwarp();
                // word t GP of group 0 of row g; other groups' pieces differ by an exclusive or, row g + 8 lies 1024 on
                const int code_at = (warp * kStages + slot) * kCodeBytes + g * 128 +
                                    ((((g * GP) & 7) ^ (t * GP / 4)) << 4) + (t * GP % 4) * 4;
                const uint8_t* sc = smem + kScales + (warp * kStages + slot) * kScaleBytes;
                auto do_group = [&](int gi) {
                    uint32_t lo[GP], hi[GP];
                    const uint8_t* codes = smem + (code_at ^ (gi * GP * 16));
                    if constexpr (GP == 4) {
                        const uint4 a = *reinterpret_cast<const uint4*>(codes);
                        const uint4 b = *reinterpret_cast<const uint4*>(codes + 1024);
                        lo[0] = a.x; lo[1] = a.y; lo[2] = a.z; lo[3] = a.w;
                        hi[0] = b.x; hi[1] = b.y; hi[2] = b.z; hi[3] = b.w;
                    } else if constexpr (GP == 2) {
                        const uint2 a = *reinterpret_cast<const uint2*>(codes);
                        const uint2 b = *reinterpret_cast<const uint2*>(codes + 1024);
                        lo[0] = a.x; lo[1] = a.y;
                        hi[0] = b.x; hi[1] = b.y;
                    } else {
                        lo[0] = *reinterpret_cast<const uint32_t*>(codes);
                        hi[0] = *reinterpret_cast<const uint32_t*>(codes + 1024);
                    }
                    // the integer sums start at kMagic - z * (sum of the bytes): read as floats they are then
                    // 1.5 * 2^23 plus the group's sum, with no conversion
                    int part[BYTES][4];
                    int z_lo = 0, z_hi = 0;
                    if (ZERO) {
                        z_lo = sc[kZeroOff + gi * 16 + g];
                        z_hi = sc[kZeroOff + gi * 16 + 8 + g];
                    }
#pragma unroll
                    for (int k = 0; k < BYTES; ++k) {
                        const int2 m = *reinterpret_cast<const int2*>(mg + mc + k * mplane);
                        part[k][0] = ZERO ? kMagic - z_lo * m.x : m.x;
                        part[k][1] = ZERO ? kMagic - z_lo * m.y : m.y;
                        part[k][2] = ZERO ? kMagic - z_hi * m.x : m.x;
                        part[k][3] = ZERO ? kMagic - z_hi * m.y : m.y;
                    }
                    constexpr int WI = GP == 1 ? 1 : 2;  // words of a token-row read
#pragma unroll
                    for (int w = 0; w < GP; w += WI) {
                        uint32_t a[WI][4];
#pragma unroll
                        for (int j = 0; j < WI; ++j) {
                            a[j][0] = lo[w + j] & 0x0F0F0F0Fu;
                            a[j][1] = hi[w + j] & 0x0F0F0F0Fu;
                            a[j][2] = (lo[w + j] >> 4) & 0x0F0F0F0Fu;
                            a[j][3] = (hi[w + j] >> 4) & 0x0F0F0F0Fu;
                        }
#pragma unroll
                        for (int k = 0; k < BYTES; ++k) {
                            const uint8_t* xp = xg + k * KP + w * 8;
                            if constexpr (WI == 2) {
                                const uint4 x = *reinterpret_cast<const uint4*>(xp);
                                mma(part[k], a[0][0], a[0][1], a[0][2], a[0][3], x.x, x.y);
                                mma(part[k], a[WI - 1][0], a[WI - 1][1], a[WI - 1][2], a[WI - 1][3], x.z, x.w);
                            } else {
                                const uint2 x = *reinterpret_cast<const uint2*>(xp);
                                mma(part[k], a[0][0], a[0][1], a[0][2], a[0][3], x.x, x.y);
                            }
                        }
                    }
                    // ---- y += s / c * (P - z sum X)
                    const uint16_t* ss = reinterpret_cast<const uint16_t*>(sc + gi * 32);
                    const float s_lo = bf16_bits_to_f32(ss[g]), s_hi = bf16_bits_to_f32(ss[8 + g]);
                    const float2 magic = make_float2(-12582912.f, -12582912.f), k256 = make_float2(256.f, 256.f);
                    const float2 inv = *reinterpret_cast<const float2*>(mg);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float2 d = make_float2(0.f, 0.f);
#pragma unroll
                        for (int k = BYTES - 1; k >= 0; --k) {
                            const float2 f =
                                add2(make_float2(__int_as_float(part[k][2 * h]), __int_as_float(part[k][2 * h + 1])), magic);
                            d = k == BYTES - 1 ? f : fma2(d, k256, f);
                        }
                        const float f = h ? s_hi : s_lo;
                        acc[h] = fma2(mul2(d, inv), make_float2(f, f), acc[h]);
                    }
                    xg += GROUP;
                    mg += mrows;
                };
                const int ng = p.G - st * NG;
#pragma unroll
                for (int gi = 0; gi < NG; ++gi) {
                    if (gi >= ng) break;
                    do_group(gi);
                }
                __syncwarp();  // every lane has read the slot that the next copies overwrite
                if (++slot == kStages) slot = 0;
                issue_next();
            }
            if constexpr (PACKED) {  // the bytes of a row are columns of neighbouring lanes
                const int b = 2 * t / PR;
                const float k = b == 0 ? 1.f : (b == 1 ? 256.f : (b < TM ? 65536.f : 0.f));
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float2& a = acc[h];
                    a.x = b < TM ? a.x * k : 0.f;
                    a.y = b < TM ? a.y * k : 0.f;
#pragma unroll
                    for (int o = PR / 2; o < 4; o <<= 1) {
                        a.x += __shfl_xor_sync(0xffffffffu, a.x, o);
                        a.y += __shfl_xor_sync(0xffffffffu, a.y, o);
                    }
                }
            }
            // ---- outputs: weight rows g (and g + 8) of the unit for token rows 2 t, 2 t + 1
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int r = 2 * t + j;
                if (r >= n) continue;  // (packed: n <= PR, so the lanes of the first byte store)
                const float lo = j ? acc[0].y : acc[0].x, hi = j ? acc[1].y : acc[1].x;
                int64_t row = aux.off[e] + first + r;
                if constexpr (PICKS) row = aux.order[row];
                if constexpr (SWIGLU) {
                    const float h = lo / (1.0f + expf(-lo)) * hi;
                    const int64_t at = row * p.n_out + un * 8 + g;
                    if constexpr (PICKS) static_cast<float*>(p.out)[at] = h;
                    else static_cast<uint16_t*>(p.out)[at] = (uint16_t)f32_to_bf16_bits(h);
                } else {
                    const int64_t at = row * p.n_out + un * 16 + g;
                    if constexpr (PICKS) {
                        static_cast<float*>(p.out)[at] = lo;
                        static_cast<float*>(p.out)[at + 8] = hi;
                    } else {
                        static_cast<uint16_t*>(p.out)[at] = (uint16_t)f32_to_bf16_bits(lo);
                        static_cast<uint16_t*>(p.out)[at + 8] = (uint16_t)f32_to_bf16_bits(hi);
                    }
                }
            }
        };
        for (int u = base_u + warp; u < end_u; u += kWarps) {
            if (aux.bn[u / nu] <= 8 / TM) unit(Bool<true>{}, u);
            else unit(Bool<false>{}, u);
        }
        b0 = v0 * nu + end_u;
    }
    cp_wait<0>();  // (empty groups only: every ring is drained)
    if (!hooked) before_rows();
}

// One product over expert-contiguous rows.
template <bool SWIGLU, int GP, bool ZERO>
__global__ void __launch_bounds__(kThreads, 1) stream_w4_kernel(const Args p) {
    extern __shared__ __align__(128) uint8_t smem[];
    Aux& aux = *reinterpret_cast<Aux*>(smem + kRingBytes);
    pdl_wait();
    for (int e = threadIdx.x; e < p.E; e += kThreads) {
        int o, n;
        if (!clamp_segment(p.offsets[e], p.counts[e], p.P, o, n) && blockIdx.x == 0) set_status(p.status, DEV_BAD_COUNT);
        aux.cnt[e] = n;
        aux.off[e] = o;
    }
    __syncthreads();
    if (threadIdx.x < 32) expert_prefixes<false>(aux, p.E, p.chunk_rows, threadIdx.x);
    __syncthreads();
    pdl_trigger();
    stream<SWIGLU, false, 2, GP, ZERO>(p, p.ph[0], smem, [] {});
}

__device__ __forceinline__ float2 load2(const void* p, int dt, int64_t at) {
    if (dt == DT_BF16) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(p) + at);
        return make_float2(bf16_bits_to_f32(w & 0xFFFFu), bf16_bits_to_f32(w >> 16));
    }
    return *reinterpret_cast<const float2*>(static_cast<const float*>(p) + at);
}

// The expert MLP of a few tokens: a cooperative launch of one CTA per SM.
template <int TM, int GP, bool ZERO>
__global__ void __launch_bounds__(kThreads, 1) picks_w4_kernel(const Args p) {
    extern __shared__ __align__(128) uint8_t smem[];
    Aux& aux = *reinterpret_cast<Aux*>(smem + kRingBytes);
    const int tid = threadIdx.x;
    namespace cg = cooperative_groups;
    const cg::grid_group grid = cg::this_grid();

    // ---- which picks belong to which expert
    if (p.P <= 32) {
        // one warp: experts in the order of their first picks
        if (tid < 32) {
            const int id = tid < p.P ? p.picks[tid] : -1;
            const bool ok = id >= 0 && id < p.E;
            if (tid < p.P && !ok && blockIdx.x == 0) set_status(p.status, DEV_BAD_EXPERT_ID);
            aux.id[tid] = (int16_t)(ok ? id : -1);
            const uint32_t valid = __ballot_sync(0xffffffffu, ok);
            const uint32_t peers = ok ? __match_any_sync(valid, id) : 1u << tid;
            const int n = __popc(peers), lead = __ffs(peers) - 1;
            const int chunks = (n + p.chunk_rows - 1) / p.chunk_rows;
            const int own = ok && lead == tid ? n + (chunks << 16) : 0;  // rows, and chunks above them
            int incl = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int m = __shfl_up_sync(0xffffffffu, incl, o);
                if (tid >= o) incl += m;
            }
            const int before = __shfl_sync(0xffffffffu, incl - own, lead);
            const int row = before & 0xFFFF, v = before >> 16;
            if (ok) aux.order[row + __popc(peers & ((1u << tid) - 1u))] = (int16_t)tid;
            if (own) {
                aux.off[id] = row;
                aux.cnt[id] = n;
                aux.vstart[id] = v;
                for (int c = 0; c < chunks; ++c) aux.chunk_e[v + c] = (uint8_t)id;
            }
            if (tid == 31) aux.vstart[p.E] = incl >> 16;
        }
        __syncthreads();
    } else {
        // a stable counting sort
        for (int e = tid; e < p.E; e += kThreads) aux.cnt[e] = 0;
        int my = -1, rank = 0;
        if (tid < p.P) {
            my = p.picks[tid];
            if (my < 0 || my >= p.E) {
                my = -1;
                if (blockIdx.x == 0) set_status(p.status, DEV_BAD_EXPERT_ID);
            }
            aux.id[tid] = (int16_t)my;
        }
        __syncthreads();
        if (my >= 0) {
            for (int o = 0; o < tid; ++o) rank += aux.id[o] == my;
            atomicAdd(&aux.cnt[my], 1);
        }
        __syncthreads();
        if (tid < 32) expert_prefixes<true>(aux, p.E, p.chunk_rows, tid);
        __syncthreads();
        if (my >= 0) aux.order[aux.off[my] + rank] = (int16_t)tid;
    }

    stream<true, true, TM, GP, ZERO>(p, p.ph[0], smem, [] {});
    stream<false, true, TM, GP, ZERO>(p, p.ph[1], smem, [&] { grid.sync(); });
    grid.sync();

    // ---- out = residual + sum_i w_i y_i in pick order, two columns per thread
    const int d = p.ph[1].n_out, T = p.P / p.top_k;
    const float* y = static_cast<const float*>(p.ph[1].out);
    const int64_t pairs = (int64_t)T * d / 2;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + tid; i < pairs; i += (int64_t)gridDim.x * kThreads) {
        const int64_t t = 2 * i / d, col = 2 * i - t * d;
        float2 yv[kMaxTopK];
#pragma unroll
        for (int k = 0; k < kMaxTopK; ++k) {
            yv[k] = make_float2(0.f, 0.f);
            if (k < p.top_k && aux.id[t * p.top_k + k] >= 0)
                yv[k] = __ldcg(reinterpret_cast<const float2*>(y + (t * p.top_k + k) * d + col));
        }
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kMaxTopK; ++k)
            if (k < p.top_k && aux.id[t * p.top_k + k] >= 0) {
                const float w = __ldg(p.weights + t * p.top_k + k);
                sum.x = fmaf(w, yv[k].x, sum.x);
                sum.y = fmaf(w, yv[k].y, sum.y);
            }
        const float2 r = load2(p.residual, p.r_dt, t * d + col);
        if (p.out_dt == DT_BF16)
            *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + t * d + col) = pack_bf16x2(r.x + sum.x, r.y + sum.y);
        else
            *reinterpret_cast<float2*>(static_cast<float*>(p.out) + t * d + col) = make_float2(r.x + sum.x, r.y + sum.y);
    }
}

// the token rows' place in shared memory; false where K is too long for one row
static bool plan_rows(int bytes, int gp, Phase& p, size_t& smem) {
    const int KP = p.G * 32 * gp;
    // a row's distance modulo 128 bytes: 8 rows' reads (16 bytes of every 32, 16, or 8) then meet no bank twice
    const int want = gp == 4 ? 16 : (gp == 2 ? 64 : 32);
    p.x_stride = ((bytes * KP - want + 127) / 128) * 128 + want;
    const int meta = (1 + bytes) * p.G * 4;  // of a row
    const int fixed = kRingBytes + kAuxBytes + meta + 16;
    p.xcap = (kSmemLimit - fixed) / (p.x_stride + meta);
    if (p.xcap < 1) return false;
    if (p.xcap > kMaxRows) p.xcap = kMaxRows;
    const size_t need = fixed + (size_t)p.xcap * (p.x_stride + meta);
    if (need > smem) smem = need;
    return true;
}

// launch one CTA per SM; cooperative: all of them run at once, so that they may wait for one another
static cudaError_t go(void (*kern)(const Args), bool (&attr_done)[64], const Ctx& c, const Args& a, size_t smem,
                      bool cooperative) {
    if (c.device < 0 || c.device >= 64) return cudaErrorInvalidDevice;
    if (!attr_done[c.device]) {
        const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
        if (err != cudaSuccess) return err;
        attr_done[c.device] = true;
    }
    return cooperative ? launch_cooperative(kern, dim3(c.num_sms), dim3(kThreads), smem, c, a)
                       : launch(kern, dim3(c.num_sms), dim3(kThreads), smem, c, a);
}

template <bool SWIGLU, int GP, bool ZERO>
static cudaError_t run_segments(const Ctx& c, Args a) {
    size_t smem = 0;
    if (!plan_rows(2, GP, a.ph[0], smem)) return cudaErrorInvalidValue;
    a.chunk_rows = a.ph[0].xcap < 8 ? a.ph[0].xcap : 8;
    static bool attr_done[64] = {};
    return go(stream_w4_kernel<SWIGLU, GP, ZERO>, attr_done, c, a, smem, false);
}

template <bool SWIGLU>
static cudaError_t run_segments_group(const Ctx& c, const Args& a, int group) {
    const bool z = a.ph[0].z0 != nullptr;
    if (group == 32) return z ? run_segments<SWIGLU, 1, true>(c, a) : run_segments<SWIGLU, 1, false>(c, a);
    if (group == 64) return z ? run_segments<SWIGLU, 2, true>(c, a) : run_segments<SWIGLU, 2, false>(c, a);
    return z ? run_segments<SWIGLU, 4, true>(c, a) : run_segments<SWIGLU, 4, false>(c, a);
}

template <int TM, int GP, bool ZERO>
static cudaError_t run_picks(const Ctx& c, Args a) {
    size_t smem = 0;
    if (!plan_rows(TM, GP, a.ph[0], smem) || !plan_rows(TM, GP, a.ph[1], smem)) return cudaErrorInvalidValue;
    const int least = a.ph[0].xcap < a.ph[1].xcap ? a.ph[0].xcap : a.ph[1].xcap;
    a.chunk_rows = least < 8 ? least : 8;
    static bool attr_done[64] = {};
    return go(picks_w4_kernel<TM, GP, ZERO>, attr_done, c, a, smem, true);
}

template <int TM>
static cudaError_t run_picks_group(const Ctx& c, const Args& a, int group) {
    const bool z = a.ph[0].z0 != nullptr;
    if (group == 32) return z ? run_picks<TM, 1, true>(c, a) : run_picks<TM, 1, false>(c, a);
    if (group == 64) return z ? run_picks<TM, 2, true>(c, a) : run_picks<TM, 2, false>(c, a);
    return z ? run_picks<TM, 4, true>(c, a) : run_picks<TM, 4, false>(c, a);
}

static Phase phase(const W4& w0, const W4& w1, int group, int K, int n_out, const void* x, void* out) {
    Phase p{};
    p.q0 = w0.q; p.s0 = w0.s; p.z0 = w0.z;
    p.q1 = w1.q; p.s1 = w1.s; p.z1 = w1.z;
    p.x = x;
    p.out = out;
    p.K = K;
    p.n_out = n_out;
    p.G = (K + group - 1) / group;
    return p;
}

static Args segment_args(const int32_t* counts, const int32_t* offsets, int S, int E, int32_t* status) {
    Args a{};
    a.counts = counts;
    a.offsets = offsets;
    a.P = S;
    a.E = E;
    a.status = status;
    return a;
}

}  // namespace w4s

cudaError_t launch_picks_w4(const Ctx& c, const void* v, const W4& Wg, const W4& Wu, const W4& Wd, int group,
                            const int32_t* idx, const float* w, const void* residual, int r_dt, int T, int k, int E, int d,
                            int d_ff, float* h, float* y, void* out, int out_dt, int32_t* status) {
    w4s::Args a{};
    a.ph[0] = w4s::phase(Wg, Wu, group, d, d_ff, v, h);
    a.ph[1] = w4s::phase(Wd, Wd, group, d_ff, d, h, y);
    a.picks = idx;
    a.weights = w;
    a.residual = residual;
    a.out = out;
    a.status = status;
    a.P = T * k;
    a.top_k = k;
    a.E = E;
    a.r_dt = r_dt;
    a.out_dt = out_dt;
    return out_dt == DT_F32 ? w4s::run_picks_group<3>(c, a, group) : w4s::run_picks_group<2>(c, a, group);
}

cudaError_t launch_gate_up_w4(const Ctx& c, const void* xp, const W4& Wg, const W4& Wu, int group, const int32_t* counts,
                              const int32_t* offsets, int S, int E, int d, int d_ff, void* h, int32_t* status,
                              const int32_t* gather, int act_rows) {
    if (S == 0) return cudaSuccess;
    if (!w4_few_rows(S, E, group)) {
        if (gather) return cudaErrorInvalidValue;
        return launch_gate_up_w4_tc(c, xp, Wg, Wu, group, counts, offsets, S, E, d, d_ff, h, status);
    }
    w4s::Args a = w4s::segment_args(counts, offsets, S, E, status);
    a.ph[0] = w4s::phase(Wg, Wu, group, d, d_ff, xp, h);
    a.gather = gather;
    a.act_rows = act_rows;
    return w4s::run_segments_group<true>(c, a, group);
}

cudaError_t launch_down_w4(const Ctx& c, const void* h, const W4& Wd, int group, const int32_t* counts,
                           const int32_t* offsets, int S, int E, int d, int d_ff, void* y, int32_t* status) {
    if (S == 0) return cudaSuccess;
    if (!w4_few_rows(S, E, group)) return launch_down_w4_tc(c, h, Wd, group, counts, offsets, S, E, d, d_ff, y, status);
    w4s::Args a = w4s::segment_args(counts, offsets, S, E, status);
    a.ph[0] = w4s::phase(Wd, Wd, group, d_ff, d, h, y);
    return w4s::run_segments_group<false>(c, a, group);
}

}  // namespace moe
