// 4-bit experts for few rows per expert: a stream of weights past a handful of token rows.
//
//   gate/up   h[r] = SiLU(Wg x[r]) * (Wu x[r])       down   y[r] = Wd h[r],      w = bf16((q - z) * s)
//
// Two forms of the same kernel:
//   segments  rows are expert-contiguous (counts, offsets as written by the permutation), optionally read
//             through a slot -> token map
//   picks     straight from the router's picks topk_idx [T][k] (T k <= 256): every CTA sorts the picks by
//             expert itself, so a token needs no permutation and no permuted copy.  h is kept as two bf16
//             terms (h = hi + lo to 16 bits), which ride as two sets of columns of the same products, and the
//             outputs are fp32: the form for single tokens loses nothing between the router and the output.
//
// What bounds it: the weights' bytes.  At 6.5 TB/s each SM has to take 23 bytes, 46 weights, per clock, so every
// step below is counted in instructions per weight.  A CUDA-core product of one row would need an FMA per
// weight on top of the unpacking and could not keep up; mma.sync m16n8k16 takes the unpacked weights straight
// from registers as its A operand (16 weight rows) with up to 8 token rows as B.  The wide tensor cores read
// their operands from shared or tensor memory; that round trip pays only for many rows (expert_w4_tc.cu).
//
// Layout.  A unit is 16 weight rows over the whole K: 8 gate and the 8 up rows of the same features (then the
// accumulators of a thread hold g and u of the same element), or 16 rows of down.  Warps are independent: each
// streams its units through a ring of its own (cp.async, 256 columns a stage, 16-byte pieces swizzled by row),
// with no barrier between warps.  Thread (g, t) = (lane / 4, lane % 4) takes word t of every 32-column piece of
// rows g and g + 8: K inside a piece is permuted alike in A and B, so a word's four pairs feed two MMAs and
// the B operand is 16 consecutive bytes of token row g.  The units of all experts form one list, cut evenly
// over the CTAs; a CTA stages the token rows of the experts its share touches in shared memory, as many
// experts at a time as fit.
#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace w4s {

constexpr int kWarps = 16;
constexpr int kThreads = 32 * kWarps;
constexpr int kStageCols = 256;
constexpr int kCodeBytes = 16 * (kStageCols / 2);            // 16 rows x 128 bytes
constexpr int kScaleOff = kCodeBytes;                        // [group][16 rows] bf16
constexpr int kZeroOff = kScaleOff + (kStageCols / 32) * 32; // [group][16 rows] u8
constexpr int kStageBytes = kZeroOff + (kStageCols / 32) * 16;
constexpr int kStages = 4;
constexpr int kRingBytes = kWarps * kStages * kStageBytes;
constexpr int kSmemLimit = 232448;
constexpr int kMaxPicks = 256;

struct Args {
    const uint8_t* q0;  // gate (rows 0..7 of a unit) or down
    const uint8_t* q1;  // up (rows 8..15) or down
    const uint16_t* s0;
    const uint16_t* s1;
    const uint8_t* z0;
    const uint8_t* z1;
    const uint16_t* x;  // token rows bf16 [rows][K]; picks / down: the hi rows, the lo rows after them
    const int32_t* gather;   // segments: slot i reads row gather[i] of act_rows rows
    const int32_t* counts;   // segments
    const int32_t* offsets;  // segments
    const int32_t* picks;    // picks: topk_idx
    int P;                   // picks: T k;  segments: rows of the buffers
    int top_k;
    int act_rows;
    int E, K, n_out, G, group;
    int chunk_rows;  // rows of one pass over an expert's weights (<= 8 NT; 8 with two terms)
    int xcap;        // token rows that fit in shared memory
    int x_stride;    // bytes of a staged row
    void* out;       // gate/up: h bf16 (picks: hi rows, then lo rows);  down: y (segments bf16, picks fp32)
    int32_t* slot_out;  // picks, gate/up: identity slot map for the combine, -1 for a bad id
    int32_t* status;
};

struct Aux {
    int vstart[kMaxExperts + 1];  // chunks before expert e
    int cnt[kMaxExperts];
    int off[kMaxExperts];
    int16_t order[kMaxPicks];  // picks sorted by expert, stable
    int16_t id[kMaxPicks];
    // the current batch's chunks: expert, first row, rows, first staged row
    int b_n;
    int be[32], bfirst[32], bn[32], brow[32];
};

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
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ void lds128(uint32_t a, uint32_t (&v)[4]) {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(a));
}
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b) {
    const __nv_bfloat162 r = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
    const __nv_bfloat162 r = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}
// four bf16 pairs of a word: 0x4300 | q is 128 + q, minus 128 + z exactly, times s with one rounding (none with
// the quantiser's scales)
__device__ __forceinline__ void unpack(uint32_t w, uint32_t zz, uint32_t ss, uint32_t (&p)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = mul2(sub2(((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u, zz), ss);
}

// NT: column sets of 8 token rows.  PICKS: the form above.  For picks / down (TERMS) set 0 is hi, set 1 lo.
template <bool SWIGLU, bool PICKS, int NT, bool ZERO>
__global__ void __launch_bounds__(kThreads, 1) stream_w4_kernel(const Args p) {
    constexpr bool TERMS = PICKS && !SWIGLU;
    static_assert(!TERMS || NT == 2, "hi and lo columns");
    constexpr int XR = TERMS ? 2 : 1;  // staged rows per token row
    extern __shared__ __align__(128) uint8_t smem[];
    Aux& aux = *reinterpret_cast<Aux*>(smem + kRingBytes);
    uint8_t* xs = smem + kRingBytes + ((sizeof(Aux) + 127) & ~size_t(127));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int E = p.E;

    pdl_wait();
    // ---- which rows belong to which expert
    int my_pick = -1, my_rank = 0;
    if constexpr (PICKS) {
        for (int e = tid; e < E; e += kThreads) aux.cnt[e] = 0;
        int my = -1;
        if (tid < p.P) {
            my = p.picks[tid];
            if (my < 0 || my >= E) {
                my = -1;
                if (blockIdx.x == 0) set_status(p.status, DEV_BAD_EXPERT_ID);
            }
            aux.id[tid] = (int16_t)my;
            if (SWIGLU && blockIdx.x == 0) p.slot_out[tid] = my < 0 ? -1 : tid;
        }
        __syncthreads();
        int rank = 0;
        if (my >= 0) {
            for (int o = 0; o < tid; ++o) rank += aux.id[o] == my;
            atomicAdd(&aux.cnt[my], 1);
        }
        my_pick = my;
        my_rank = rank;
    } else {
        for (int e = tid; e < E; e += kThreads) {
            int o, n;
            if (!clamp_segment(p.offsets[e], p.counts[e], p.P, o, n) && blockIdx.x == 0)
                set_status(p.status, DEV_BAD_COUNT);
            aux.cnt[e] = n;
            aux.off[e] = o;
        }
    }
    __syncthreads();
    if (warp == 0) {  // exclusive prefixes over the experts: chunks, and (picks) rows
        int loc[8], cnt[8], sum = 0, rsum = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int e = lane * 8 + i;
            cnt[i] = e < E ? aux.cnt[e] : 0;
            loc[i] = (cnt[i] + p.chunk_rows - 1) / p.chunk_rows;
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
            }
            run += loc[i];
            rrun += cnt[i];
        }
        if (lane == 31) aux.vstart[E] = incl;
    }
    __syncthreads();
    if (PICKS && my_pick >= 0) aux.order[aux.off[my_pick] + my_rank] = (int16_t)tid;
    pdl_trigger();

    constexpr int UROWS = SWIGLU ? 8 : 16;  // output columns of a unit
    const int nu = p.n_out / UROWS;         // units of one pass over an expert
    const int64_t total = (int64_t)aux.vstart[E] * nu;
    const int64_t u_begin = total * blockIdx.x / gridDim.x, u_end = total * (blockIdx.x + 1) / gridDim.x;
    const int nstage = (p.K + kStageCols - 1) / kStageCols;
    const int pieces = p.K / 32;  // 32-column pieces of a row
    const int NG = kStageCols / p.group;
    const int gp = p.group / 32;  // pieces of a group
    const uint32_t ring = smem_addr(smem) + warp * kStages * kStageBytes;
    const uint32_t xbase = smem_addr(xs);
    const int g = lane >> 2, t = lane & 3;

    // expert and first row of chunk v
    auto find = [&](int v, int& e, int& first, int& n) {
        int lo = 0, hi = E - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (aux.vstart[mid] <= v) lo = mid; else hi = mid - 1;
        }
        e = lo;
        first = (v - aux.vstart[e]) * p.chunk_rows;
        n = min(p.chunk_rows, aux.cnt[e] - first);
    };
    // the ring's copies of one stage of unit (e, un)
    auto issue = [&](int e, int un, int st, int slot) {
        const uint32_t dst = ring + slot * kStageBytes;
        const int64_t half_row = (int64_t)e * p.n_out + un * UROWS;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = j * 32 + lane, r = i >> 3, c = i & 7;
            const int64_t row = half_row + (SWIGLU ? (r & 7) : r);
            const uint8_t* src = (SWIGLU && r >= 8 ? p.q1 : p.q0) + row * (p.K / 2) + st * (kStageCols / 2) + c * 16;
            if (st * 8 + c < pieces) cp16(dst + r * 128 + ((c ^ (r & 7)) << 4), src);
        }
        if (lane < 2 * NG) {
            const int gr = st * NG + (lane >> 1), h = lane & 1;
            if (gr < p.G) {
                const int64_t at = ((int64_t)e * p.G + gr) * p.n_out + un * UROWS + (SWIGLU ? 0 : 8 * h);
                cp16(dst + kScaleOff + lane * 16, (SWIGLU && h ? p.s1 : p.s0) + at);
                if (ZERO) cp8(dst + kZeroOff + lane * 8, (SWIGLU && h ? p.z1 : p.z0) + at);
            }
        }
    };

    for (int64_t b0 = u_begin; b0 < u_end;) {
        // ---- a batch: the chunks from the current one on whose rows fit together (32 at most)
        const int v0 = (int)(b0 / nu);
        __syncthreads();  // the last batch's rows and table have been read
        if (warp == 0) {
            const int v = v0 + lane;
            int e = 0, first = 0, n = 0;
            const bool in = v < aux.vstart[E] && (int64_t)v * nu < u_end;
            if (in) find(v, e, first, n);
            int incl = n * XR;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int m = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += m;
            }
            aux.be[lane] = e;
            aux.bfirst[lane] = first;
            aux.bn[lane] = n;
            aux.brow[lane] = incl - n * XR;
            const uint32_t fit = __ballot_sync(0xffffffffu, in && incl <= p.xcap);
            if (lane == 0) aux.b_n = __popc(fit);  // a prefix of the lanes; one chunk always fits
        }
        __syncthreads();
        const int nv = aux.b_n;
        const int base_u = (int)(b0 - (int64_t)v0 * nu);  // units are counted from chunk v0's first
        const int end_u = (int)(min(u_end, (int64_t)(v0 + nv) * nu) - (int64_t)v0 * nu);

        // ---- stage its token rows (asynchronously), then start this warp's weights
        const int all_rows = aux.brow[nv - 1] + aux.bn[nv - 1] * XR;
        for (int r = warp, ci = 0; r < all_rows; r += kWarps) {
            while (ci + 1 < nv && aux.brow[ci + 1] <= r) ++ci;
            const int n = aux.bn[ci], rr = r - aux.brow[ci];
            const int at = aux.off[aux.be[ci]] + aux.bfirst[ci] + (TERMS && rr >= n ? rr - n : rr);
            int64_t src = at;
            if constexpr (PICKS) {
                const int pick = aux.order[at];
                src = TERMS ? (rr >= n ? p.P : 0) + pick : pick / p.top_k;  // a chunk's hi rows, then its lo rows
            } else if (p.gather) {
                src = p.gather[at];
                if (src < 0 || src >= p.act_rows) {
                    if (lane == 0) set_status(p.status, DEV_BAD_COUNT);
                    src = 0;
                }
            }
            const uint16_t* row = p.x + src * p.K;
            const uint32_t dst = xbase + r * p.x_stride;
            for (int c = lane; c < p.K / 8; c += 32) cp16(dst + c * 16, row + c * 8);
        }
        cp_commit();
        int iu = base_u + warp;  // the unit whose stages are being issued: base + warp, + kWarps, ...
        int ist = 0, islot = 0, ie = 0, iun = 0;
        auto issue_next = [&]() {
            if (iu < end_u) {
                if (ist == 0) {
                    const int v = iu / nu;
                    ie = aux.be[v];
                    iun = iu - v * nu;
                }
                issue(ie, iun, ist, islot);
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
        cp_wait<kStages - 1>();  // the token rows
        __syncthreads();

        int slot = 0;
        for (int u = base_u + warp; u < end_u; u += kWarps) {
            const int v = u / nu, un = u - v * nu;
            const int e = aux.be[v], first = aux.bfirst[v], n = aux.bn[v], xrow = aux.brow[v];
            float acc[NT][4];
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
            // this lane's token row of each column set (rows past the chunk give zeros)
            uint32_t xa[NT];
            bool live[NT];
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                live[i] = TERMS ? g < n : g + 8 * i < n;
                xa[i] = xbase + (xrow + g + (TERMS ? i * n : 8 * i)) * p.x_stride + t * 16;
            }
            for (int st = 0; st < nstage; ++st) {
                cp_wait<kStages - 2>();
                __syncwarp();
                const uint32_t base = ring + slot * kStageBytes;
                // sums of one stage, added to the running ones in fp32: the tensor cores' own sums are truncated
                float part[NT][4];
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) part[i][j] = 0.f;
                uint32_t s_lo = 0, s_hi = 0, z_lo = 0x43084308u, z_hi = 0x43084308u;
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    if (st * 8 + c >= pieces) break;
                    if ((c & (gp - 1)) == 0) {
                        const int gr = c / gp;
                        s_lo = lds16(base + kScaleOff + gr * 32 + 2 * g) * 0x00010001u;
                        s_hi = lds16(base + kScaleOff + gr * 32 + 16 + 2 * g) * 0x00010001u;
                        if (ZERO) {
                            z_lo = 0x43004300u + lds8(base + kZeroOff + gr * 16 + g) * 0x00010001u;
                            z_hi = 0x43004300u + lds8(base + kZeroOff + gr * 16 + 8 + g) * 0x00010001u;
                        }
                    }
                    const uint32_t wa = base + g * 128 + ((c ^ g) << 4) + t * 4;
                    uint32_t a[4], b[4];
                    unpack(lds32(wa), z_lo, s_lo, a);
                    unpack(lds32(wa + 8 * 128), z_hi, s_hi, b);
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        uint32_t x[4] = {0u, 0u, 0u, 0u};
                        if (live[i]) lds128(xa[i] + (st * 8 + c) * 64, x);
                        mma(part[i], a[0], b[0], a[1], b[1], x[0], x[1]);
                        mma(part[i], a[2], b[2], a[3], b[3], x[2], x[3]);
                    }
                }
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] += part[i][j];
                __syncwarp();  // every lane has read the slot that the next copies overwrite
                if (++slot == kStages) slot = 0;
                issue_next();
            }
            // ---- outputs: rows g (and g + 8) of the unit for token rows 2 t, 2 t + 1 of each set
            if constexpr (SWIGLU) {
                uint16_t* h = static_cast<uint16_t*>(p.out);
                const int f = un * 8 + g;
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int r = 8 * i + 2 * t + j;
                        if (r >= n) continue;
                        const float gv = acc[i][j], uv = acc[i][2 + j];
                        const float hv = gv / (1.0f + expf(-gv)) * uv;
                        const uint32_t hb = f32_to_bf16_bits(hv);
                        if constexpr (PICKS) {
                            const int64_t pick = aux.order[aux.off[e] + first + r];
                            h[pick * p.n_out + f] = (uint16_t)hb;
                            h[(pick + p.P) * p.n_out + f] = (uint16_t)f32_to_bf16_bits(hv - bf16_bits_to_f32(hb));
                        } else {
                            h[(int64_t)(aux.off[e] + first + r) * p.n_out + f] = (uint16_t)hb;
                        }
                    }
            } else {
                const int o = un * 16 + g;
                if constexpr (TERMS) {
                    float* y = static_cast<float*>(p.out);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int r = 2 * t + j;
                        if (r >= n) continue;
                        const int64_t pick = aux.order[aux.off[e] + first + r];
                        y[pick * p.n_out + o] = acc[0][j] + acc[NT - 1][j];
                        y[pick * p.n_out + o + 8] = acc[0][2 + j] + acc[NT - 1][2 + j];
                    }
                } else {
                    uint16_t* y = static_cast<uint16_t*>(p.out);
#pragma unroll
                    for (int i = 0; i < NT; ++i)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const int r = 8 * i + 2 * t + j;
                            if (r >= n) continue;
                            uint16_t* row = y + (int64_t)(aux.off[e] + first + r) * p.n_out + o;
                            row[0] = (uint16_t)f32_to_bf16_bits(acc[i][j]);
                            row[8] = (uint16_t)f32_to_bf16_bits(acc[i][2 + j]);
                        }
                }
            }
        }
        cp_wait<0>();  // (empty groups only: the ring is drained)
        b0 = (int64_t)v0 * nu + end_u;
    }
}

// token rows per pass and their place in shared memory; false where K is too long for one row
static bool plan_rows(int K, int NT, bool terms, Args& a, size_t& smem) {
    const size_t fixed = kRingBytes + ((sizeof(Aux) + 127) & ~size_t(127));
    a.x_stride = ((K * 2 + 127) & ~127) + 64;  // rows half a 128-byte line apart: the B reads touch every bank once
    a.xcap = (int)((kSmemLimit - fixed) / a.x_stride);
    const int per = terms ? 2 : 1;
    a.chunk_rows = terms ? 8 : 8 * NT;
    if (a.chunk_rows * per > a.xcap) a.chunk_rows = a.xcap / per;
    smem = fixed + (size_t)a.xcap * a.x_stride;
    return a.chunk_rows >= 1;
}

template <bool SWIGLU, bool PICKS, int NT, bool ZERO>
static cudaError_t run(const Ctx& c, Args a) {
    size_t smem = 0;
    if (!plan_rows(a.K, NT, PICKS && !SWIGLU, a, smem)) return cudaErrorInvalidValue;
    auto kern = stream_w4_kernel<SWIGLU, PICKS, NT, ZERO>;
    static bool attr_done[64] = {};
    if (c.device < 0 || c.device >= 64) return cudaErrorInvalidDevice;
    if (!attr_done[c.device]) {
        cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
        if (err != cudaSuccess) return err;
        attr_done[c.device] = true;
    }
    return launch(kern, dim3(c.num_sms), dim3(kThreads), smem, c, a);
}

template <bool SWIGLU, bool PICKS, int NT>
static cudaError_t run_z(const Ctx& c, const Args& a) {
    return a.z0 ? run<SWIGLU, PICKS, NT, true>(c, a) : run<SWIGLU, PICKS, NT, false>(c, a);
}

static Args base_args(const W4& w0, const W4& w1, int group, int E, int K, int n_out) {
    Args a{};
    a.q0 = w0.q; a.s0 = w0.s; a.z0 = w0.z;
    a.q1 = w1.q; a.s1 = w1.s; a.z1 = w1.z;
    a.E = E;
    a.K = K;
    a.n_out = n_out;
    a.group = group;
    a.G = (K + group - 1) / group;
    return a;
}

}  // namespace w4s

cudaError_t launch_gate_up_w4_picks(const Ctx& c, const void* v, const W4& Wg, const W4& Wu, int group,
                                    const int32_t* idx, int T, int k, int E, int d, int d_ff, void* h, int32_t* slot,
                                    int32_t* status) {
    w4s::Args a = w4s::base_args(Wg, Wu, group, E, d, d_ff);
    a.x = static_cast<const uint16_t*>(v);
    a.picks = idx;
    a.P = T * k;
    a.top_k = k;
    a.out = h;
    a.slot_out = slot;
    a.status = status;
    // an expert has at most T rows unless a token names it twice: one set of columns covers up to 8
    return T <= 8 ? w4s::run_z<true, true, 1>(c, a) : w4s::run_z<true, true, 2>(c, a);
}

cudaError_t launch_down_w4_picks(const Ctx& c, const void* h, const W4& Wd, int group, const int32_t* idx, int T, int k,
                                 int E, int d, int d_ff, float* y, int32_t* status) {
    w4s::Args a = w4s::base_args(Wd, Wd, group, E, d_ff, d);
    a.x = static_cast<const uint16_t*>(h);
    a.picks = idx;
    a.P = T * k;
    a.top_k = k;
    a.out = y;
    a.status = status;
    return w4s::run_z<false, true, 2>(c, a);
}

cudaError_t launch_gate_up_w4(const Ctx& c, const void* xp, const W4& Wg, const W4& Wu, int group, const int32_t* counts,
                              const int32_t* offsets, int S, int E, int d, int d_ff, void* h, int32_t* status,
                              const int32_t* gather, int act_rows) {
    if (S == 0) return cudaSuccess;
    w4s::Args a = w4s::base_args(Wg, Wu, group, E, d, d_ff);
    a.x = static_cast<const uint16_t*>(xp);
    a.gather = gather;
    a.act_rows = act_rows;
    a.counts = counts;
    a.offsets = offsets;
    a.P = S;
    a.out = h;
    a.status = status;
    return S <= 2 * E ? w4s::run_z<true, false, 1>(c, a) : w4s::run_z<true, false, 2>(c, a);
}

cudaError_t launch_down_w4(const Ctx& c, const void* h, const W4& Wd, int group, const int32_t* counts,
                           const int32_t* offsets, int S, int E, int d, int d_ff, void* y, int32_t* status) {
    if (S == 0) return cudaSuccess;
    w4s::Args a = w4s::base_args(Wd, Wd, group, E, d_ff, d);
    a.x = static_cast<const uint16_t*>(h);
    a.counts = counts;
    a.offsets = offsets;
    a.P = S;
    a.out = y;
    a.status = status;
    return S <= 2 * E ? w4s::run_z<false, false, 1>(c, a) : w4s::run_z<false, false, 2>(c, a);
}

}  // namespace moe
