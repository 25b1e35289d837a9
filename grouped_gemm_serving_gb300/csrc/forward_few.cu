// moe_forward_few: the whole expert layer for a few tokens (generating a token at
// a time for each sequence of a batch) in two kernels.
//
// With e = ids[t, j] the picks of token t and w[t, j] their weights:
//   [g | u] = W1[e] x[t],   h = silu(g) u,   out[t] = sum_j w[t, j] W2[e] h.
// Every weight of an expert that some token picked is read once, which bounds the
// layer: 2 operations a weight and token against 2 bytes (bf16) or 1 (e4m3).
//
// Routing takes no kernel of its own: every block of both kernels routes all
// tokens itself (they are few) and keeps, per expert, the set of its tokens as a
// 64-bit mask.  Row r of an expert is its r-th token in ascending order, so the
// masks' bit counts are the offsets, the permutation and its inverse.
//
// A block's unit is 16 weight rows (8 features' gate and up rows, or 16 output
// features) of one expert against up to 32 of its rows.  Eight warps split the
// contraction: a lane loads 16 bytes of weight rows l / 4 and l / 4 + 8 straight
// into registers, and warp-level m16n8k16 MMAs multiply them with the same bytes
// of up to 8 rows of x (the order of the contraction's elements within a step is
// the lanes' own, the same for both operands).  A ninth warp adds the eight
// partial sums in warp order and finishes the unit while the others go on to the
// next.
//
// FP8 weights are converted to bf16 on the way (exact) and each 128 columns'
// partial sum is multiplied by its block's scale in fp32.  x and h stay bf16:
// quantising them would save no weight bytes, and cost accuracy.
//
// The first kernel writes h, rounded to bf16 (the type of the MMA's operand).  The
// second one is launched programmatically, has its first weights under way when
// it waits for h, and writes fp32 rows y; the block that brings the last of a
// 16-feature column's units sums each token's rows in slot order and rounds once.
#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"
#include "route.cuh"

namespace {

constexpr int kStream = 8;                      // warps that stream weights
constexpr int kThreads = 32 * (kStream + 1);
constexpr int kRows = 16;                       // weight rows of a unit
constexpr int kBatch = 6;                       // steps whose loads are in flight together
constexpr int kMaxT = 64;                       // tokens: the bits of a mask
constexpr int kMaxSlots = 1024;
constexpr int kMaxE = 256;
constexpr int kMaxChunks = kMaxE + kMaxSlots / 32;

struct Args {
    // routing
    const float* logits;
    const float* bias;
    const uint8_t* mask;
    int32_t* ids;
    float* w;
    int T, E, k, renormalize;
    // product
    const uint4* x;           // GATED: x [T, nx], else h [T*k, nx]
    const uint4* W;           // GATED: [E, 2F, nv], else [E, F, nv]
    const float* scales;      // FP8: a scale per 128 x 128 block of W
    int nv, nx, F;            // vectors of a weight row and of a row of x; features
    __nv_bfloat16* h;         // GATED: [T*k, F] out
    float* part;              // else: y [ceil(F/16), T*k, 16], then summed into
    __nv_bfloat16* out;       // [T, F]
    int* arrived;             // per 16 output features: units done (zeroed by the first kernel)
    int columns;              // their number
    int* err;
};

// What a block knows of the routing.
struct Plan {
    uint32_t tokens[kMaxE][2];          // the expert's tokens
    int base[kMaxE];                    // its first row
    short chunk_expert[kMaxChunks];     // up to R rows of an expert each
    short chunk_row[kMaxChunks];        // the first of them, counted from the expert's
    uint8_t token[kMaxSlots];           // a row's token
    short slot_id[kMaxSlots];
    float slot_w[kMaxSlots];
    int chunks;
};

__device__ __forceinline__ uint4 load_once(const uint4* p) {   // weights: read once, not kept in L1
    uint4 v;
    asm("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
        : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
        : "l"(__cvta_generic_to_global(p)));
    return v;
}

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two e4m3 values as two bf16: through fp16 and fp32, both exact, and a bf16's
// 8 significant bits hold an e4m3's 4, so cutting fp32 in half is exact too.
__device__ __forceinline__ uint32_t bf16x2_of_e4m3x2(uint32_t two) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    return __byte_perm(__float_as_uint(f.x), __float_as_uint(f.y), 0x7632);
}

// Routes all tokens.  The first block of the first kernel (`record`) also writes
// the picks and weights out and reports invalid ones.
template <int R>
__device__ void make_plan(const Args& a, Plan& P, bool record) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i < 2 * a.E; i += kThreads) (&P.tokens[0][0])[i] = 0;
    __syncthreads();
    const auto take = [&](int t, int s, int id, bool changed) {
        if (a.mask && a.mask[s]) {
            changed |= id != a.E;
            id = a.E;
        }
        if (id < 0 || id > a.E) {
            if (record) moe::raise_device_error(a.err, MOE_DEVERR_ROUTE);
            changed = true;
            id = a.E;
        }
        if (record && changed && a.ids) a.ids[s] = id;
        P.slot_id[s] = static_cast<short>(id);
        if (id < a.E) atomicOr(&P.tokens[id][t >> 5], 1u << (t & 31));
    };
    if (a.logits) {
        for (int t = warp; t < a.T; t += kStream + 1) {
            const float* row = a.logits + static_cast<int64_t>(t) * a.E;
            float w;
            int id;
            if (a.E <= 32) id = moe::top_picks<1>(row, a.bias, a.E, a.k, a.renormalize, w);
            else if (a.E <= 64) id = moe::top_picks<2>(row, a.bias, a.E, a.k, a.renormalize, w);
            else if (a.E <= 128) id = moe::top_picks<4>(row, a.bias, a.E, a.k, a.renormalize, w);
            else id = moe::top_picks<8>(row, a.bias, a.E, a.k, a.renormalize, w);
            if (lane < a.k) {
                const int s = t * a.k + lane;
                P.slot_w[s] = w;
                if (record && a.w) a.w[s] = w;
                take(t, s, id, true);
            }
        }
    } else {
        for (int s = tid; s < a.T * a.k; s += kThreads) {
            P.slot_w[s] = a.w[s];
            take(s / a.k, s, a.ids[s], false);
        }
    }
    __syncthreads();
    if (warp == 0) {
        int rows = 0, chunks = 0;
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const int e = e0 + lane;
            const int n = e < a.E ? __popc(P.tokens[e][0]) + __popc(P.tokens[e][1]) : 0;
            const int c = (n + R - 1) / R;
            int at = n, first = c;   // inclusive sums over the lanes
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int p = __shfl_up_sync(0xffffffffu, at, off), q = __shfl_up_sync(0xffffffffu, first, off);
                if (lane >= off) {
                    at += p;
                    first += q;
                }
            }
            if (n) {
                P.base[e] = rows + at - n;
                for (int i = 0; i < c; ++i) {
                    P.chunk_expert[chunks + first - c + i] = static_cast<short>(e);
                    P.chunk_row[chunks + first - c + i] = static_cast<short>(i * R);
                }
            }
            rows += __shfl_sync(0xffffffffu, at, 31);
            chunks += __shfl_sync(0xffffffffu, first, 31);
        }
        if (lane == 0) P.chunks = chunks;
    }
    __syncthreads();
    for (int e = tid; e < a.E; e += kThreads) {
        uint64_t left = P.tokens[e][0] | static_cast<uint64_t>(P.tokens[e][1]) << 32;
        if (left == 0) continue;   // base is not set
        for (int r = P.base[e]; left; ++r, left &= left - 1) P.token[r] = static_cast<uint8_t>(__ffsll(left) - 1);
    }
    __syncthreads();
}

__device__ __forceinline__ int rows_of(const Plan& P, int e) { return __popc(P.tokens[e][0]) + __popc(P.tokens[e][1]); }

// The row of token t among the rows of expert e, which it picked.
__device__ __forceinline__ int row_of(const Plan& P, int e, int t) {
    const uint32_t below = (1u << (t & 31)) - 1;
    return P.base[e] + (t < 32 ? __popc(P.tokens[e][0] & below) : __popc(P.tokens[e][0]) + __popc(P.tokens[e][1] & below));
}

// This warp's share of one unit: weight rows w0 and w1 (this lane's two) against
// NB groups of 8 rows of x, xr[b] this lane's row of group b (NULL: none).  `wait`:
// the kernel that writes x may still run.  s0, s1: the scales of the two weight
// rows' blocks.
template <bool FP8, int NB>
__device__ __forceinline__ void share(const uint4* w0, const uint4* w1, const float* s0, const float* s1, int lo, int hi,
                                      const uint4* const (&xr)[NB], bool wait, float (&d)[NB][4]) {
    const int c = threadIdx.x & 3;
    const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) d[b][i] = 0.0f;
    for (int v0 = lo; v0 < hi; v0 += 4 * kBatch) {
        uint4 r0[kBatch], r1[kBatch];
        float f0[kBatch / 2], f1[kBatch / 2];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const bool in = v0 + 4 * i + c < hi;
            r0[i] = in ? load_once(w0 + v0 + 4 * i + c) : zero;
            r1[i] = in ? load_once(w1 + v0 + 4 * i + c) : zero;
            if (FP8 && i % 2 == 0) {   // 8 vectors are 128 columns
                const bool is = v0 + 4 * i < hi;
                f0[i / 2] = is ? __ldg(s0 + (v0 + 4 * i) / 8) : 0.0f;
                f1[i / 2] = is ? __ldg(s1 + (v0 + 4 * i) / 8) : 0.0f;
            }
        }
        if (wait) {
            moe::wait_for_primary();
            wait = false;
        }
        if (!FP8) {
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const int v = v0 + 4 * i + c;
                    const uint4 xv = xr[b] && v < hi ? xr[b][v] : zero;
                    mma(d[b], r0[i].x, r1[i].x, r0[i].y, r1[i].y, xv.x, xv.y);
                    mma(d[b], r0[i].z, r1[i].z, r0[i].w, r1[i].w, xv.z, xv.w);
                }
            }
        } else {
#pragma unroll
            for (int p = 0; p < kBatch / 2; ++p) {
                float t[NB][4];
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int i = 0; i < 4; ++i) t[b][i] = 0.0f;
#pragma unroll
                for (int i = 2 * p; i < 2 * p + 2; ++i) {
                    const int v = v0 + 4 * i + c;
                    const uint32_t a0[4] = {r0[i].x, r0[i].y, r0[i].z, r0[i].w};
                    const uint32_t a1[4] = {r1[i].x, r1[i].y, r1[i].z, r1[i].w};
                    uint32_t xs[NB][8];
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        const bool in = xr[b] && v < hi;
                        const uint4 xa = in ? xr[b][2 * v] : zero, xb = in ? xr[b][2 * v + 1] : zero;
                        xs[b][0] = xa.x, xs[b][1] = xa.y, xs[b][2] = xa.z, xs[b][3] = xa.w;
                        xs[b][4] = xb.x, xs[b][5] = xb.y, xs[b][6] = xb.z, xs[b][7] = xb.w;
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t m0 = bf16x2_of_e4m3x2(a0[j] & 0xFFFF), m2 = bf16x2_of_e4m3x2(a0[j] >> 16);
                        const uint32_t m1 = bf16x2_of_e4m3x2(a1[j] & 0xFFFF), m3 = bf16x2_of_e4m3x2(a1[j] >> 16);
#pragma unroll
                        for (int b = 0; b < NB; ++b) mma(t[b], m0, m1, m2, m3, xs[b][2 * j], xs[b][2 * j + 1]);
                    }
                }
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    d[b][0] = fmaf(f0[p], t[b][0], d[b][0]);
                    d[b][1] = fmaf(f0[p], t[b][1], d[b][1]);
                    d[b][2] = fmaf(f1[p], t[b][2], d[b][2]);
                    d[b][3] = fmaf(f1[p], t[b][3], d[b][3]);
                }
            }
        }
    }
    if (wait) moe::wait_for_primary();
}

// Named barriers between the streaming warps and the ninth, two of each kind for
// the two buffers of partial sums.
__device__ __forceinline__ void bar_sync(int id) { asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(kThreads) : "memory"); }
__device__ __forceinline__ void bar_arrive(int id) { asm volatile("bar.arrive %0, %1;" ::"r"(id), "n"(kThreads) : "memory"); }
constexpr int kFull = 1, kEmpty = 3;

// R: the most rows of a unit (8, 16 or 32).
template <bool FP8, bool GATED, int R>
__global__ void __maxnreg__(112)   // two blocks an SM
few_tokens_kernel(const Args a) {
    __shared__ Plan P;
    __shared__ float4 red[2][R / 8][kStream][32];   // turn, group of 8 rows, warp, lane
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2;
    if (GATED) {
        if (blockIdx.x == 0)
            for (int i = threadIdx.x; i < a.columns; i += kThreads) a.arrived[i] = 0;
        moe::launch_dependents();   // the second product may take its place beside this one
    }
    make_plan<R>(a, P, GATED && blockIdx.x == 0);
    constexpr int kFeatures = GATED ? kRows / 2 : kRows;
    const int per = (a.F + kFeatures - 1) / kFeatures;   // units of a chunk
    const int units = P.chunks * per;
    int turn = 0, done = 0;
    if (warp < kStream) {
        // this warp's vectors of every row: whole 128-byte lines
        const int slice = ((a.nv + 8 * kStream - 1) / (8 * kStream)) * 8;
        const int lo = min(a.nv, warp * slice), hi = min(a.nv, lo + slice);
        const int blocks_k = a.nv / 8;   // FP8: scales of a row
        bool wait = !GATED;
        for (int unit = blockIdx.x; unit < units; unit += gridDim.x, turn ^= 1, ++done) {
            const int c = unit / per, f0 = (unit - c * per) * kFeatures;
            const int e = P.chunk_expert[c], r0 = P.chunk_row[c];
            const int p = P.base[e] + r0, rows = min(R, rows_of(P, e) - r0);
            // lane l's rows: features f0 + l / 4 (gate, up), or f0 + l / 4 and + 8; past the
            // last feature the last one again, whose sums are not stored
            const int n0 = min(f0 + g, a.F - 1), n1 = GATED ? a.F + n0 : min(f0 + g + 8, a.F - 1);
            const int64_t first = static_cast<int64_t>(e) * (GATED ? 2 : 1) * a.F;
            const uint4* w0 = a.W + (first + n0) * a.nv;
            const uint4* w1 = a.W + (first + n1) * a.nv;
            const float *s0 = nullptr, *s1 = nullptr;
            if (FP8) {   // an expert's rows fill whole blocks but for the second product's last
                const int64_t blocks_n = ((GATED ? 2 : 1) * static_cast<int64_t>(a.F) + 127) / 128;
                s0 = a.scales + (e * blocks_n + n0 / 128) * blocks_k;
                s1 = a.scales + (e * blocks_n + n1 / 128) * blocks_k;
            }
            const auto go = [&](auto nb) {
                constexpr int NB = decltype(nb)::value;
                const uint4* xr[NB];
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const int r = 8 * b + g;
                    xr[b] = r < rows ? a.x + static_cast<int64_t>(GATED ? P.token[p + r] : p + r) * a.nx : nullptr;
                }
                float d[NB][4];
                share<FP8, NB>(w0, w1, s0, s1, lo, hi, xr, wait, d);
                if (done >= 2) bar_sync(kEmpty + turn);
#pragma unroll
                for (int b = 0; b < NB; ++b) red[turn][b][warp][lane] = make_float4(d[b][0], d[b][1], d[b][2], d[b][3]);
            };
            if (R == 8 || rows <= 8) go(std::integral_constant<int, 1>());
            else if (R == 16 || rows <= 16) go(std::integral_constant<int, (R >= 16 ? 2 : 1)>());
            else go(std::integral_constant<int, R / 8>());
            wait = false;
            bar_arrive(kFull + turn);
        }
        if (wait) moe::wait_for_primary();
        // the ninth warp arrives once for every unit: take the last two as well
        for (int i = max(0, done - 2); i < done; ++i) bar_sync(kEmpty + (i & 1));
    } else {
        if (!GATED) moe::wait_for_primary();
        const int rows_all = a.T * a.k;
        for (int unit = blockIdx.x; unit < units; unit += gridDim.x, turn ^= 1) {
            const int c = unit / per, f0 = (unit - c * per) * kFeatures;
            const int e = P.chunk_expert[c], r0 = P.chunk_row[c];
            const int p = P.base[e] + r0, rows = min(R, rows_of(P, e) - r0);
            bar_sync(kFull + turn);
            for (int b = 0; 8 * b < rows; ++b) {
                float4 s = red[turn][b][0][lane];
#pragma unroll
                for (int i = 1; i < kStream; ++i) {
                    const float4 v = red[turn][b][i][lane];
                    s.x += v.x;
                    s.y += v.y;
                    s.z += v.z;
                    s.w += v.w;
                }
                const float top[2] = {s.x, s.y}, bottom[2] = {s.z, s.w};   // weight rows l / 4 and l / 4 + 8
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int row = 8 * b + 2 * (lane & 3) + j;
                    if (row >= rows) continue;
                    if (GATED) {
                        if (f0 + g < a.F)
                            a.h[static_cast<int64_t>(p + row) * a.F + f0 + g] =
                                __float2bfloat16_rn(top[j] / (1.0f + expf(-top[j])) * bottom[j]);
                    } else {
                        float* y = a.part + (static_cast<int64_t>(f0 / kRows) * rows_all + p + row) * kRows;
                        y[g] = top[j];
                        y[g + 8] = bottom[j];
                    }
                }
            }
            bar_arrive(kEmpty + turn);
            if (GATED) continue;
            // the last of this column's units sums every token's rows
            __threadfence();
            __syncwarp();
            int before = 0;
            if (lane == 0) before = atomicAdd(&a.arrived[f0 / kRows], 1);
            if (__shfl_sync(0xffffffffu, before, 0) != P.chunks - 1) continue;
            __threadfence();
            const float* y = a.part + static_cast<int64_t>(f0 / kRows) * rows_all * kRows;
            const int f = 2 * (lane & 7);
            for (int t = lane >> 3; t < a.T; t += 4) {
                float2 sum = make_float2(0.0f, 0.0f);
                for (int j = 0; j < a.k; ++j) {
                    const int id = P.slot_id[t * a.k + j];
                    if (id == a.E) continue;
                    const float w = P.slot_w[t * a.k + j];
                    const float2 v = __ldcg(reinterpret_cast<const float2*>(y + row_of(P, id, t) * kRows + f));
                    sum.x = fmaf(w, v.x, sum.x);
                    sum.y = fmaf(w, v.y, sum.y);
                }
                if (f0 + f < a.F)
                    *reinterpret_cast<uint32_t*>(a.out + static_cast<int64_t>(t) * a.F + f0 + f) = moe::pack_bf16x2(sum.x, sum.y);
            }
        }
    }
    if (!GATED && P.chunks == 0) {   // no token has an expert
        moe::wait_for_primary();
        for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < static_cast<int64_t>(a.T) * a.F;
             i += static_cast<int64_t>(gridDim.x) * kThreads)
            a.out[i] = __float2bfloat16_rn(0.0f);
    }
}

template <bool FP8, int R>
moe_status_t launch(const Args& a1, const Args& a2, cudaStream_t s) {
    static std::atomic<int> resident[2][moe::kMaxDevices];
    const int g1 = moe::resident_blocks(reinterpret_cast<const void*>(few_tokens_kernel<FP8, true, R>), kThreads, 0, resident[0]);
    const int g2 = moe::resident_blocks(reinterpret_cast<const void*>(few_tokens_kernel<FP8, false, R>), kThreads, 0, resident[1]);
    if (g1 <= 0 || g2 <= 0) return MOE_ERR_CUDA;
    // As many blocks as give each the same number of units if every slot has an
    // expert of its own: a last round that only some have leaves too few loads in
    // flight.
    const int chunks = a1.T * a1.k < a1.E ? a1.T * a1.k : a1.E;
    const auto blocks = [&](int units_of_chunk, int most) {
        const int64_t units = static_cast<int64_t>(units_of_chunk) * chunks;
        const int64_t rounds = (units + most - 1) / most;
        return static_cast<int>((units + rounds - 1) / rounds);
    };
    few_tokens_kernel<FP8, true, R><<<blocks((a1.F + 7) / 8, g1), kThreads, 0, s>>>(a1);
    MOE_CHECK_LAUNCH();
    return moe::launch_after(few_tokens_kernel<FP8, false, R>, dim3(blocks((a2.F + 15) / 16, g2)), kThreads, 0, s, a2);
}

template <bool FP8>
moe_status_t launch_for(const Args& a1, const Args& a2, cudaStream_t s) {
    if (a1.T <= 8) return launch<FP8, 8>(a1, a2, s);
    if (a1.T <= 16) return launch<FP8, 16>(a1, a2, s);
    return launch<FP8, 32>(a1, a2, s);
}

bool valid_sizes(const moe_forward_args* a) {
    if (a->T < 1 || a->E < 1 || a->E > kMaxE || a->k < 1 || a->k > a->E || a->k > 32) return false;
    if (a->H < 8 || a->H % 8 || a->I < 8 || a->I % 8) return false;
    if (a->dtype == MOE_FP8_E4M3_B128) return a->H % 128 == 0 && a->I % 128 == 0;
    return a->dtype == MOE_BF16;
}

// More tokens than a mask has bits, more slots than a block keeps, rows whose
// vectors 32 bits do not count, and what only moe_forward does.
bool supported(const moe_forward_args* a) {
    return a->T <= kMaxT && a->T * a->k <= kMaxSlots && a->H <= (1 << 20) && a->I <= (1 << 20) && a->flags == 0;
}

struct Layout {
    size_t arrived, h, part, total;
};

Layout layout(const moe_forward_args* a) {
    Layout l{};
    size_t off = 0;
    const auto take = [&off](size_t bytes) {
        const size_t at = off;
        off += (bytes + 255) & ~static_cast<size_t>(255);
        return at;
    };
    const size_t rows = static_cast<size_t>(a->T) * a->k, columns = (a->H + kRows - 1) / kRows;
    l.arrived = take(columns * sizeof(int));
    l.h = take(rows * a->I * 2);
    l.part = take(columns * rows * kRows * sizeof(float));
    l.total = off;
    return l;
}

}  // namespace

extern "C" size_t moe_forward_few_workspace_size(const moe_forward_args* a) {
    return a && valid_sizes(a) && supported(a) ? layout(a).total : 0;
}

extern "C" moe_status_t moe_forward_few(const moe_forward_args* a, void* ws, size_t ws_bytes, moe_stream_t stream) {
    MOE_CHECK_ARG(a && valid_sizes(a));
    const bool fp8 = a->dtype == MOE_FP8_E4M3_B128;
    MOE_CHECK_ARG(a->x && a->W1 && a->W2 && a->out && (!fp8 || (a->W1_scales && a->W2_scales)));
    MOE_CHECK_ARG(a->logits || (a->topk_ids && a->topk_w));
    MOE_CHECK_ARG(moe::aligned16(a->x) && moe::aligned16(a->W1) && moe::aligned16(a->W2) && moe::aligned16(a->out) &&
                  moe::aligned16(a->logits) && moe::aligned16(a->topk_ids) && moe::aligned16(a->topk_w) &&
                  (!a->logits || moe::aligned16(a->expert_bias)) &&
                  (!fp8 || (moe::aligned_to(a->W1_scales, 4) && moe::aligned_to(a->W2_scales, 4))));
    if (!supported(a)) return MOE_ERR_UNSUPPORTED;
    const Layout l = layout(a);
    if (!ws || ws_bytes < l.total) return MOE_ERR_WORKSPACE;
    MOE_CHECK_ARG(moe::aligned16(ws));
    int* err = moe::device_error_word();
    if (!err) return MOE_ERR_CUDA;
    auto* base = static_cast<uint8_t*>(ws);
    const int per_vector = fp8 ? 16 : 8;
    Args a1{};
    a1.logits = a->logits;
    a1.bias = a->expert_bias;
    a1.mask = a->sentinel_mask;
    a1.ids = a->topk_ids;
    a1.w = a->topk_w;
    a1.T = a->T, a1.E = a->E, a1.k = a->k, a1.renormalize = a->renormalize;
    a1.h = reinterpret_cast<__nv_bfloat16*>(base + l.h);
    a1.part = reinterpret_cast<float*>(base + l.part);
    a1.out = static_cast<__nv_bfloat16*>(a->out);
    a1.arrived = reinterpret_cast<int*>(base + l.arrived);
    a1.columns = (a->H + kRows - 1) / kRows;
    a1.err = err;
    Args a2 = a1;
    a1.x = static_cast<const uint4*>(a->x);
    a1.W = static_cast<const uint4*>(a->W1);
    a1.scales = a->W1_scales;
    a1.nv = a->H / per_vector, a1.nx = a->H / 8, a1.F = a->I;
    a2.x = reinterpret_cast<const uint4*>(a1.h);
    a2.W = static_cast<const uint4*>(a->W2);
    a2.scales = a->W2_scales;
    a2.nv = a->I / per_vector, a2.nx = a->I / 8, a2.F = a->H;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return fp8 ? launch_for<true>(a1, a2, s) : launch_for<false>(a1, a2, s);
}
