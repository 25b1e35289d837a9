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
// features) of one expert against up to 32 of its rows of x; the units lie in
// expert order and every block takes a run of them.  A producer warp brings the
// weights 512 columns at a time into a ring in shared memory by TMA tiles of 128
// bytes by 16 rows, so that the loads in flight do not depend on what the other
// warps do.  Eight warps take 64 of the columns each (m16n8k16 MMAs; the order of
// the contraction's elements within a step is the lanes' own, the same for both
// operands), with their columns of the expert's rows of x in shared memory for as
// long as the expert lasts.  Two more warps take turns at adding the eight partial
// sums in warp order and finishing a unit while the others go on to the next.
//
// FP8 weights are converted to bf16 on the way (exact) and the partial sum of a
// warp's 64 columns is multiplied by their block's scale in fp32.  x and h stay
// bf16: quantising them would save no weight bytes, and cost accuracy.
//
// The first kernel writes h, rounded to bf16 (the type of the MMA's operand).  The
// second one is launched programmatically, beside the first if their shared memory
// allows it, and has its ring full of weights when it waits for h.  It writes fp32
// rows y; the block that brings the last of a 16-feature column's units sums each
// token's rows in slot order and rounds once.
#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"
#include "route.cuh"

namespace {

constexpr int kProduct = 8;                     // warps that multiply
constexpr int kThreads = 32 * (kProduct + 3);   // two that finish units, and the producer
constexpr int kRows = 16;                       // weight rows of a unit
constexpr int kColumns = 512;                   // columns of a stage
constexpr int kRowBytes = 128;                  // of a tile's row: 64 columns in bf16, 128 in e4m3
constexpr int kTileBytes = kRows * kRowBytes;
template <bool FP8>
constexpr int kTiles = kColumns * (FP8 ? 1 : 2) / kRowBytes;   // of a stage
constexpr int kMaxStages = 16;
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr int kMaxT = 64;                       // tokens: the bits of a mask
constexpr int kMaxSlots = 1024;
constexpr int kMaxE = 256;
constexpr int kMaxK = 32768;                     // columns of a product: a row of x takes 2 bytes each of a block

struct Args {
    // routing
    const float* logits;
    const float* bias;
    const uint8_t* mask;
    int32_t* ids;
    float* w;
    int T, E, k, renormalize;
    // product
    const uint4* x;           // GATED: x [T, K], else h [T*k, K]
    const float* scales;      // FP8: a scale per 128 x 128 block of W
    int K, F;                 // columns and features of W: [E, 2F, K] (GATED) or [E, F, K]
    int xrows, stages;        // the most rows of a unit; depth of the ring
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
    short chunk_expert[kMaxSlots];     // up to a.xrows rows of an expert each
    short chunk_row[kMaxSlots];        // the first of them, counted from the expert's
    uint8_t token[kMaxSlots];           // a row's token
    short slot_id[kMaxSlots];
    float slot_w[kMaxSlots];
    int chunks;
};

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
        for (int t = warp; t < a.T; t += kProduct + 3) {
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
            const int c = (n + a.xrows - 1) / a.xrows;
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
                    P.chunk_row[chunks + first - c + i] = static_cast<short>(i * a.xrows);
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

// Named barriers between the warps that multiply and those that finish, two of
// each kind for the two buffers of partial sums.
constexpr int kFull = 1, kEmpty = 3, kBarThreads = 32 * (kProduct + 1);
__device__ __forceinline__ void bar_sync(int id) { asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(kBarThreads) : "memory"); }
__device__ __forceinline__ void bar_arrive(int id) { asm volatile("bar.arrive %0, %1;" ::"r"(id), "n"(kBarThreads) : "memory"); }

struct Ring {
    uint64_t full[kMaxStages], empty[kMaxStages];
    int abort_flag;
};

// Where a unit is: rows p to p + rows - 1 of expert e, and its first feature.
struct Unit {
    int chunk, e, f0, p, rows;
};
template <bool GATED>
__device__ __forceinline__ Unit unit_at(const Args& a, const Plan& P, int unit, int per) {
    Unit u;
    u.chunk = unit / per;
    u.f0 = (unit - u.chunk * per) * (GATED ? kRows / 2 : kRows);
    u.e = P.chunk_expert[u.chunk];
    u.p = P.base[u.e] + P.chunk_row[u.chunk];
    u.rows = min(a.xrows, rows_of(P, u.e) - P.chunk_row[u.chunk]);
    return u;
}

// A warp's 64 columns of a stage.  Tiles are swizzled: vector j of row r is at
// j ^ (r mod 8).  bf16: the tile's 8 vectors, lane l taking 2 (l mod 4) and the one
// after it of rows l / 4 and l / 4 + 8: the 8 lanes that are served together find
// theirs in different banks.  e4m3: two warps share a tile, one with the even
// vectors, one with the odd.  x: [row][8 vectors], swizzled alike; rows past the
// last one read the last (their sums are not used).
template <int NB>
__device__ __forceinline__ void multiply(const uint8_t* tile, const uint8_t* xs, int rows, float (&d)[NB][4]) {
    const int g = (threadIdx.x & 31) >> 2, c = threadIdx.x & 3;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int at = ((2 * c + i) ^ g) * 16;
        const uint4 r0 = *reinterpret_cast<const uint4*>(tile + g * kRowBytes + at);
        const uint4 r1 = *reinterpret_cast<const uint4*>(tile + (g + 8) * kRowBytes + at);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int r = min(8 * b + g, rows - 1);
            const uint4 xv = *reinterpret_cast<const uint4*>(xs + r * kRowBytes + ((2 * c + i) ^ (r & 7)) * 16);
            mma(d[b], r0.x, r1.x, r0.y, r1.y, xv.x, xv.y);
            mma(d[b], r0.z, r1.z, r0.w, r1.w, xv.z, xv.w);
        }
    }
}
template <int NB>
__device__ __forceinline__ void multiply_fp8(const uint8_t* tile, int odd, const uint8_t* xs, int rows, float s0, float s1,
                                             float (&d)[NB][4]) {
    const int g = (threadIdx.x & 31) >> 2, c = threadIdx.x & 3;
    const int at = ((2 * c + odd) ^ g) * 16;
    const uint4 q0 = *reinterpret_cast<const uint4*>(tile + g * kRowBytes + at);
    const uint4 q1 = *reinterpret_cast<const uint4*>(tile + (g + 8) * kRowBytes + at);
    const uint32_t a0[4] = {q0.x, q0.y, q0.z, q0.w}, a1[4] = {q1.x, q1.y, q1.z, q1.w};
    float t[NB][4];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) t[b][i] = 0.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint4 xv[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int r = min(8 * b + g, rows - 1);
            xv[b] = *reinterpret_cast<const uint4*>(xs + r * kRowBytes + ((2 * c + i) ^ (r & 7)) * 16);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t m0 = bf16x2_of_e4m3x2(a0[2 * i + j] & 0xFFFF), m2 = bf16x2_of_e4m3x2(a0[2 * i + j] >> 16);
            const uint32_t m1 = bf16x2_of_e4m3x2(a1[2 * i + j] & 0xFFFF), m3 = bf16x2_of_e4m3x2(a1[2 * i + j] >> 16);
#pragma unroll
            for (int b = 0; b < NB; ++b) mma(t[b], m0, m1, m2, m3, j ? xv[b].z : xv[b].x, j ? xv[b].w : xv[b].y);
        }
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        d[b][0] = fmaf(s0, t[b][0], d[b][0]);
        d[b][1] = fmaf(s0, t[b][1], d[b][1]);
        d[b][2] = fmaf(s1, t[b][2], d[b][2]);
        d[b][3] = fmaf(s1, t[b][3], d[b][3]);
    }
}

// One warp sums every token's rows of 16 features, in slot order: 4 lanes a token,
// TP of 8 tokens each at a time with 4 slots' loads in flight.  (A block that falls
// behind brings its columns' last units and has to sum them too: at 11 us for 64
// tokens, one load at a time, it fell ever further behind, and the second kernel
// took 211 us instead of 100.)
template <int TP>
__device__ __forceinline__ void sum_rows(const Args& a, const Plan& P, const float* y, int f0) {
    const int lane = threadIdx.x & 31, f = 4 * (lane & 3);
    for (int t0 = lane >> 2; t0 < a.T; t0 += 8 * TP) {
        float4 sum[TP];
#pragma unroll
        for (int i = 0; i < TP; ++i) sum[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int j0 = 0; j0 < a.k; j0 += 4) {
            float4 v[TP][4];
            float w[TP][4];
#pragma unroll
            for (int i = 0; i < TP; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int t = t0 + 8 * i, s = t * a.k + j0 + j;
                    const bool in = t < a.T && j0 + j < a.k && P.slot_id[s] != a.E;
                    v[i][j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    w[i][j] = 0.0f;
                    if (in) {
                        v[i][j] = __ldcg(reinterpret_cast<const float4*>(y + row_of(P, P.slot_id[s], t) * kRows + f));
                        w[i][j] = P.slot_w[s];
                    }
                }
#pragma unroll
            for (int i = 0; i < TP; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    sum[i].x = fmaf(w[i][j], v[i][j].x, sum[i].x);
                    sum[i].y = fmaf(w[i][j], v[i][j].y, sum[i].y);
                    sum[i].z = fmaf(w[i][j], v[i][j].z, sum[i].z);
                    sum[i].w = fmaf(w[i][j], v[i][j].w, sum[i].w);
                }
        }
#pragma unroll
        for (int i = 0; i < TP; ++i) {
            const int t = t0 + 8 * i;
            if (t < a.T && f0 + f < a.F)
                *reinterpret_cast<uint2*>(a.out + static_cast<int64_t>(t) * a.F + f0 + f) =
                    make_uint2(moe::pack_bf16x2(sum[i].x, sum[i].y), moe::pack_bf16x2(sum[i].z, sum[i].w));
        }
    }
}

// R: the most rows of a unit (8, 16 or 32; a.xrows <= R).  Dynamic shared memory:
// the ring (tiles want 1024-byte boundaries), two buffers of partial sums, and
// every product warp's columns of x, [warp][step][row][8 vectors].
template <bool FP8, bool GATED, int R>
__global__ void __launch_bounds__(kThreads, R == 8 ? 2 : 1)
few_tokens_kernel(const __grid_constant__ CUtensorMap map, const Args a) {
    extern __shared__ __align__(16) uint8_t smem[];
    using Sums = float4[R / 8][kProduct][32];   // group of 8 rows, warp, lane
    constexpr int kStageBytes = kTiles<FP8> * kTileBytes;
    uint8_t* ring = smem + (-moe::smem_u32(smem) & 1023u);
    Sums* red = reinterpret_cast<Sums*>(ring + a.stages * kStageBytes);
    uint8_t* xcols = ring + a.stages * kStageBytes + 2 * sizeof(Sums);
    __shared__ Plan P;
    __shared__ Ring S;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2;
    if (GATED) {
        if (blockIdx.x == 0)
            for (int i = threadIdx.x; i < a.columns; i += kThreads) a.arrived[i] = 0;
        moe::launch_dependents();   // the second product may take its place beside this one
    }
    if (threadIdx.x == 0) {
        S.abort_flag = 0;
        for (int i = 0; i < a.stages; ++i) {
            moe::mbar_init(moe::smem_u32(&S.full[i]), 1);
            moe::mbar_init(moe::smem_u32(&S.empty[i]), kProduct);
        }
        moe::fence_barrier_init();
        moe::prefetch_tensormap(&map);
    }
    make_plan(a, P, GATED && blockIdx.x == 0);
    constexpr int kFeatures = GATED ? kRows / 2 : kRows;
    const int per = (a.F + kFeatures - 1) / kFeatures;   // units of a chunk
    const int64_t units = static_cast<int64_t>(P.chunks) * per;
    const int begin = static_cast<int>(units * blockIdx.x / gridDim.x), end = static_cast<int>(units * (blockIdx.x + 1) / gridDim.x);
    const int steps = (a.K + kColumns - 1) / kColumns;   // stages of a unit
    constexpr int kTileColumns = kRowBytes / (FP8 ? 1 : 2);
    if (warp == kProduct + 2) {
        // ---- producer
        int slot = 0;
        uint32_t turn = 0;
        int64_t filled = 0;
        bool gave_up = false;
        for (int unit = begin; unit < end && !gave_up; ++unit) {
            const int c = unit / per, f0 = (unit - c * per) * kFeatures, e = P.chunk_expert[c];
            for (int k0 = 0; k0 < a.K; k0 += kColumns, ++filled) {
                if (filled >= a.stages && !moe::mbar_wait(moe::smem_u32(&S.empty[slot]), turn ^ 1u, &S.abort_flag, kWaitNs)) {
                    gave_up = true;
                    break;
                }
                const int tiles = min(kTiles<FP8>, (a.K - k0 + kTileColumns - 1) / kTileColumns);
                const uint32_t bar = moe::smem_u32(&S.full[slot]), dst = moe::smem_u32(ring) + slot * kStageBytes;
                if (moe::elect_one()) {
                    moe::mbar_arrive_expect_tx(bar, tiles * kTileBytes);
                    for (int i = 0; i < tiles; ++i) {
                        if (GATED) moe::tma_load_4d(dst + i * kTileBytes, &map, bar, k0 + i * kTileColumns, f0, 0, e);
                        else moe::tma_load_3d(dst + i * kTileBytes, &map, bar, k0 + i * kTileColumns, f0, e);
                    }
                }
                __syncwarp();
                if (++slot == a.stages) {
                    slot = 0;
                    turn ^= 1u;
                }
            }
        }
        if (gave_up) {   // no copy may land after the block has ended
            if (lane == 0 && !S.abort_flag) moe::raise_device_error(a.err, MOE_DEVERR_TIMEOUT);
            S.abort_flag = 1;
            int never = 0;
            for (int i = 0; i < a.stages && i < filled; ++i)
                moe::mbar_wait(moe::smem_u32(&S.full[i]), static_cast<uint32_t>((filled - 1 - i) / a.stages) & 1u, &never, kWaitNs / 16);
        }
    } else if (warp < kProduct) {
        // ---- this warp's 64 columns of every stage
        int turn = 0, slot = 0, held = -1;
        uint32_t phase = 0;
        uint8_t* const mine = xcols + static_cast<size_t>(warp) * steps * a.xrows * kRowBytes;
        // vector q of a step's 64 columns, counted from the step's first
        const auto column = [&](int q) { return FP8 ? 128 * (warp / 2) + 16 * ((q & ~1) + (warp & 1)) + 8 * (q & 1) : 64 * warp + 8 * q; };
        const int blocks_k = a.K / 128, block0 = warp / 2;   // FP8: scales of a row, and of this warp's first columns
        const int64_t blocks_n = ((GATED ? 2 : 1) * static_cast<int64_t>(a.F) + 127) / 128;
        // lane i's scales of step i, fetched a unit ahead
        float s0 = 0.0f, s1 = 0.0f;
        const auto scales_of = [&](int unit, int step, float& v0, float& v1) {
            const int c = unit / per, f0 = (unit - c * per) * kFeatures;
            const float* row = a.scales + P.chunk_expert[c] * blocks_n * blocks_k;
            const int k = (step + lane) * (kColumns / 128) + block0;
            if (k < blocks_k) {
                v0 = __ldg(row + static_cast<int64_t>(f0 / 128) * blocks_k + k);
                v1 = GATED ? __ldg(row + static_cast<int64_t>((a.F + f0) / 128) * blocks_k + k) : v0;
            }
        };
        if (FP8 && begin < end) scales_of(begin, 0, s0, s1);
        for (int unit = begin; unit < end; ++unit, turn ^= 1) {
            const Unit u = unit_at<GATED>(a, P, unit, per);
            float n0 = 0.0f, n1 = 0.0f;
            if (FP8 && unit + 1 < end) scales_of(unit + 1, 0, n0, n1);
            if (u.chunk != held) {   // this warp's columns of the next rows of x
                if (!GATED && held < 0) moe::wait_for_primary();
                held = u.chunk;
                __syncwarp();
                const int vectors = steps * u.rows * 8;
                for (int v0 = 0; v0 < vectors; v0 += 32 * 8) {
                    uint4 v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int at = v0 + 32 * i + lane, q = at & 7, step = (at >> 3) / u.rows, r = (at >> 3) - step * u.rows;
                        const int k = step * kColumns + column(q);
                        v[i] = make_uint4(0, 0, 0, 0);
                        if (at < vectors && k < a.K)
                            v[i] = a.x[(static_cast<int64_t>(GATED ? P.token[u.p + r] : u.p + r) * a.K + k) / 8];
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int at = v0 + 32 * i + lane, q = at & 7, step = (at >> 3) / u.rows, r = (at >> 3) - step * u.rows;
                        if (at < vectors)
                            *reinterpret_cast<uint4*>(mine + (step * a.xrows + r) * kRowBytes + (q ^ (r & 7)) * 16) = v[i];
                    }
                }
                __syncwarp();
            }
            const auto go = [&](auto nb) {
                constexpr int NB = decltype(nb)::value;
                float d[NB][4];
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int i = 0; i < 4; ++i) d[b][i] = 0.0f;
                for (int step = 0; step < steps; ++step) {
                    if (FP8 && step > 0 && step % 32 == 0) scales_of(unit, step, s0, s1);
                    if (!moe::mbar_wait(moe::smem_u32(&S.full[slot]), phase, &S.abort_flag, kWaitNs)) {
                        if (lane == 0 && !S.abort_flag) moe::raise_device_error(a.err, MOE_DEVERR_TIMEOUT);
                        S.abort_flag = 1;   // what follows is not waited for as long
                    }
                    const uint8_t* tile = ring + slot * kStageBytes + (FP8 ? warp / 2 : warp) * kTileBytes;
                    const uint8_t* xs = mine + step * a.xrows * kRowBytes;
                    if (step * kColumns + (FP8 ? 128 * (warp / 2) : 64 * warp) < a.K) {
                        if (FP8)
                            multiply_fp8<NB>(tile, warp & 1, xs, u.rows, __shfl_sync(0xffffffffu, s0, step & 31),
                                             __shfl_sync(0xffffffffu, s1, step & 31), d);
                        else multiply<NB>(tile, xs, u.rows, d);
                    }
                    __syncwarp();
                    if (lane == 0) moe::mbar_arrive(moe::smem_u32(&S.empty[slot]));
                    if (++slot == a.stages) {
                        slot = 0;
                        phase ^= 1u;
                    }
                }
                if (unit - begin >= 2) bar_sync(kEmpty + turn);
#pragma unroll
                for (int b = 0; b < NB; ++b) red[turn][b][warp][lane] = make_float4(d[b][0], d[b][1], d[b][2], d[b][3]);
            };
            if (R == 8 || u.rows <= 8) go(std::integral_constant<int, 1>());
            else if (R == 16 || u.rows <= 16) go(std::integral_constant<int, (R >= 16 ? 2 : 1)>());
            else go(std::integral_constant<int, R / 8>());
            bar_arrive(kFull + turn);
            s0 = n0;
            s1 = n1;
        }
        // the finishing warps arrive once for every unit: take the last two as well
        for (int i = max(0, end - begin - 2); i < end - begin; ++i) bar_sync(kEmpty + (i & 1));
    } else {
        // ---- finishing: every other unit
        if (!GATED) moe::wait_for_primary();
        const int turn = warp - kProduct, rows_all = a.T * a.k;
        for (int unit = begin + turn; unit < end; unit += 2) {
            const Unit u = unit_at<GATED>(a, P, unit, per);
            bar_sync(kFull + turn);
            for (int b = 0; 8 * b < u.rows; ++b) {
                float4 s = red[turn][b][0][lane];
#pragma unroll
                for (int i = 1; i < kProduct; ++i) {
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
                    if (row >= u.rows) continue;
                    if (GATED) {
                        if (u.f0 + g < a.F)
                            a.h[static_cast<int64_t>(u.p + row) * a.F + u.f0 + g] =
                                __float2bfloat16_rn(top[j] / (1.0f + expf(-top[j])) * bottom[j]);
                    } else {
                        float* y = a.part + (static_cast<int64_t>(u.f0 / kRows) * rows_all + u.p + row) * kRows;
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
            if (lane == 0) before = atomicAdd(&a.arrived[u.f0 / kRows], 1);
            if (__shfl_sync(0xffffffffu, before, 0) != P.chunks - 1) continue;
            __threadfence();
            sum_rows<R == 8 ? 1 : 4>(a, P, a.part + static_cast<int64_t>(u.f0 / kRows) * rows_all * kRows, u.f0);
        }
    }
    if (!GATED && P.chunks == 0) {   // no token has an expert
        moe::wait_for_primary();
        for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < static_cast<int64_t>(a.T) * a.F;
             i += static_cast<int64_t>(gridDim.x) * kThreads)
            a.out[i] = __float2bfloat16_rn(0.0f);
    }
}

// The kernel may take that much dynamic shared memory; remembered per device.
bool allow_smem(const void* kernel, std::atomic<int> (&cache)[moe::kMaxDevices], size_t smem) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= moe::kMaxDevices) return false;
    if (cache[dev].load(std::memory_order_relaxed) >= static_cast<int>(smem)) return true;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess) {
        (void)cudaGetLastError();
        return false;
    }
    cache[dev].store(static_cast<int>(smem), std::memory_order_relaxed);
    return true;
}

constexpr size_t kHalf = 113 * 1024, kWhole = 227 * 1024;   // shared memory of a block, with another one beside it or not
constexpr size_t kLeastRing = 64 * 1024;

// Shared memory of a product of K columns and at most T rows an expert: R, a.xrows
// and a.stages.  Room for a block of the other kernel beside this one if the ring
// is still deep enough; else the whole SM, with as many rows of x as leave the ring
// that depth.
template <bool FP8>
size_t shape(Args& a, int& R) {
    const size_t row = static_cast<size_t>((a.K + kColumns - 1) / kColumns) * kProduct * kRowBytes, stage = kTiles<FP8> * kTileBytes;
    const size_t fixed = sizeof(Plan) + sizeof(Ring) + 64 + 1024;   // with what alignment takes
    const auto sums = [](int r) { return static_cast<size_t>(2 * r / 8) * kProduct * 32 * sizeof(float4); };
    size_t all = kWhole;
    R = a.T <= 8 ? 8 : a.T <= 16 ? 16 : 32;
    if (R == 8 && fixed + sums(8) + a.T * row + kLeastRing <= kHalf) {
        all = kHalf;
        a.xrows = a.T;
    } else {
        while (R > 8 && fixed + sums(R) + (a.T < R ? a.T : R) * row + kLeastRing > kWhole) R /= 2;
        const size_t most = (kWhole - fixed - sums(R) - kLeastRing) / row;
        a.xrows = a.T < R ? a.T : R;
        if (most < static_cast<size_t>(a.xrows)) a.xrows = static_cast<int>(most);
    }
    const size_t n = (all - fixed - sums(R) - a.xrows * row) / stage;
    a.stages = static_cast<int>(n < kMaxStages ? n : kMaxStages);
    return 1024 + a.stages * stage + sums(R) + a.xrows * row;
}

// x and W of 16 rows by 128 bytes; GATED: 8 gate rows and the same 8 up rows.
bool weight_map(CUtensorMap* map, bool fp8, bool gated, const void* W, int E, int F, int K) {
    const cuuint64_t e = fp8 ? 1 : 2, k = K, f = F;
    const cuuint32_t columns = fp8 ? kRowBytes : kRowBytes / 2;
    if (gated) {
        const cuuint64_t dims[4] = {k, f, 2, static_cast<cuuint64_t>(E)}, strides[3] = {k * e, f * k * e, 2 * f * k * e};
        const cuuint32_t box[4] = {columns, kRows / 2, 2, 1};
        return moe::encode_tile_map(map, fp8, W, 4, dims, strides, box);
    }
    const cuuint64_t dims[3] = {k, f, static_cast<cuuint64_t>(E)}, strides[2] = {k * e, f * k * e};
    const cuuint32_t box[3] = {columns, kRows, 1};
    return moe::encode_tile_map(map, fp8, W, 3, dims, strides, box);
}

template <bool FP8, bool GATED, int R>
moe_status_t launch(const CUtensorMap& map, const Args& a, size_t smem, cudaStream_t s) {
    static std::atomic<int> allowed[moe::kMaxDevices];
    const int sms = moe::sm_count();
    if (sms <= 0 || !allow_smem(reinterpret_cast<const void*>(few_tokens_kernel<FP8, GATED, R>), allowed, smem)) return MOE_ERR_CUDA;
    // a block per SM, if every slot has an expert of its own
    const int chunks = a.T * a.k < a.E ? a.T * a.k : a.E, features = GATED ? kRows / 2 : kRows;
    const int64_t units = static_cast<int64_t>((a.F + features - 1) / features) * chunks;
    const int blocks = static_cast<int>(units < sms ? units : sms);
    if (!GATED) return moe::launch_after(few_tokens_kernel<FP8, GATED, R>, dim3(blocks), kThreads, smem, s, map, a);
    few_tokens_kernel<FP8, GATED, R><<<blocks, kThreads, smem, s>>>(map, a);
    MOE_CHECK_LAUNCH();
    return MOE_OK;
}

template <bool FP8, bool GATED>
moe_status_t product(Args a, const void* W, cudaStream_t s) {
    CUtensorMap map;
    if (!weight_map(&map, FP8, GATED, W, a.E, a.F, a.K)) return MOE_ERR_CUDA;
    int R;
    const size_t smem = shape<FP8>(a, R);
    if (R == 8) return launch<FP8, GATED, 8>(map, a, smem, s);
    if (R == 16) return launch<FP8, GATED, 16>(map, a, smem, s);
    return launch<FP8, GATED, 32>(map, a, smem, s);
}

template <bool FP8>
moe_status_t both(const Args& a1, const void* W1, const Args& a2, const void* W2, cudaStream_t s) {
    const moe_status_t st = product<FP8, true>(a1, W1, s);
    return st != MOE_OK ? st : product<FP8, false>(a2, W2, s);
}

bool valid_sizes(const moe_forward_args* a) {
    if (a->T < 1 || a->E < 1 || a->E > kMaxE || a->k < 1 || a->k > a->E || a->k > 32) return false;
    if (a->H < 8 || a->H % 8 || a->I < 8 || a->I % 8) return false;
    if (a->dtype == MOE_FP8_E4M3_B128) return a->H % 128 == 0 && a->I % 128 == 0;
    return a->dtype == MOE_BF16;
}

// Not more tokens than a mask has bits, more slots or longer rows than a block keeps, nor what only moe_forward does.
bool supported(const moe_forward_args* a) {
    return a->T <= kMaxT && a->T * a->k <= kMaxSlots && a->H <= kMaxK && a->I <= kMaxK && a->flags == 0;
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
    a1.scales = a->W1_scales;
    a1.K = a->H, a1.F = a->I;
    a2.x = reinterpret_cast<const uint4*>(a1.h);
    a2.scales = a->W2_scales;
    a2.K = a->I, a2.F = a->H;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return fp8 ? both<true>(a1, a->W1, a2, a->W2, s) : both<false>(a1, a->W1, a2, a->W2, s);
}
