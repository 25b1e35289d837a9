// Softmax cross entropy of T tokens against a vocabulary matrix, without the
// logits ever being stored: the loss behind the layer when a model with it is
// trained or its text is scored.
//
//   z[t, v] = sum_c x[t, c] W[v, c],   lse[t] = log sum_v exp z[t, v],
//   loss[t] = lse[t] - z[t, label[t]]
//   G[t, v] = exp(z[t, v] - lse[t]) - [v = label[t]]   (the label's from the fp32 dot product below)
//   dx[t] = dloss[t] sum_v G[t, v] W[v],   dW[v] = sum_t G[t, v] dloss[t] x[t]
//
// Forward: the logits kernel below computes z tile by tile in tensor memory
// and reduces each tile to a running maximum and sum of exponentials a row,
// without the label's column.  The label's logit z_l comes from a dot product
// of its own, in fp32 arithmetic that rounds to nearest, by warps that have
// nothing else to do: the tensor cores' sums, which cut off, are off by some
// 2e-6 of z_l, which the difference lse - z_l would keep.  (lse has the other
// logits' share of that: over 1 to 64 tokens and H up to 7168 it is off by 7e-8 in
// the median and by 7e-6 at most, one token at H = 7032, and loss by 1.5e-5; fp32
// products: 4e-8 and 8e-7.)  A second, small
// kernel joins the vocabulary tiles' pairs (m, s) and the label:
//   M = max m,  S = sum s exp(m - M),  lse = log(S exp M + exp z_l),
//   loss = log(1 + S exp(M - z_l)),
// which keeps its precision where the label is all but certain.
// 2 T H V operations, W read once: bound by the tensor pipe for many tokens
// and by reading W for few.
//
// Backward, a piece of the vocabulary at a time (6 T H V operations, as the
// logits are computed again): the logits kernel writes the piece's G in bf16,
// the grouped GEMM's data gradient adds G W to dx in fp32, and its weight
// gradient computes the piece's rows of dW.  G's entries are probabilities and
// label entries near -1, each rounded by at most a relative 2^-8,
// independently; dloss stays out of G, so that the label entries, which carry
// most of the gradient, are not all off by the same rounding of dloss.  It
// multiplies dx in fp32; for dW its largest magnitude d does, and x is scaled by
// dloss / d, which changes nothing where all tokens weigh the same (a mean) and
// rounds x to bf16 once more elsewhere.
//
// The logits kernel: CTA pairs (clusters of two), tcgen05 cta_group::2 MMAs of
// 256 tokens (128 per CTA) x up to 256 vocabulary rows (half staged by each
// CTA) x 64 columns a stage, seven stages, accumulators double-buffered in
// tensor memory.  A lane of tensor memory is a token, so a row's maximum and
// sum run along a thread's own columns.  Tiles are walked vocabulary-major
// with the token tiles inside, so the pairs that run together read the same
// rows of W, once from HBM, while x stays in L2.  At most 128 tokens take
// M = 128 MMAs (64 tokens staged per CTA, half the tensor time), whose
// accumulator holds token l % 64 in lane l, columns (l / 64) N/2 .. + N/2.  The tile's width in
// vocabulary rows is 256 or, where the tiles do not fill whole rounds of the
// pairs, the smallest multiple of 16 that takes as many rounds.
//
// Roles in a CTA (384 threads): warp 0 loads (TMA), warp 1 of the even CTA
// issues the MMAs, warps 4-11 are the epilogue (warp w: lanes 32 (w % 4)..,
// half (w - 4) / 4 of the columns), and in the forward pass warps 2 and 3 take
// the labels' logits.  Every wait is bounded; on expiry the CTA
// records MOE_DEVERR_TIMEOUT, waits for its loads and MMAs and leaves.
#include <climits>

#include "common.cuh"
#include "internal.h"

namespace {

constexpr int kMaxStages = 7;
// Backward gives one stage to the warps' transposes of G.
template <bool BACK>
constexpr int kStagesOf = BACK ? 6 : kMaxStages;
constexpr int kStageA = 128 * 128;   // 128 tokens x 64 bf16
constexpr int kStageB = 128 * 128;   // up to 128 vocabulary rows x 64 bf16
constexpr int kStageBytes = kStageA + kStageB;
constexpr int BT = 256, BV = 256;    // tokens and vocabulary rows of a pair's tile
constexpr int kEpiThreads = 256;
constexpr int kThreads = 128 + kEpiThreads;
constexpr uint32_t kTmemCols = 512;
constexpr uint64_t kWaitNs = 2000000000ull, kDrainNs = 100000000ull;
constexpr float kLog2e = 1.4426950408889634f;

struct Params {
    const int32_t* labels;
    int* err;
    int T, k_blocks;
    int bt;               // tokens of a tile: BT, or 128 for at most 128 tokens
    int v0, cols;         // the launch's vocabulary rows: [v0, v0 + cols)
    int bv;               // vocabulary rows of a tile (multiple of 16, <= BV)
    int tok_tiles, voc_tiles;
    int ignore, V;
    moe::After after;
    // forward
    float2* part;         // [shares * voc_tiles, T]: maximum and sum of each share of a tile's columns
    int shares;           // 2, or 4 for tiles of 128 tokens
    float* at_label;      // [T]: the label's logit
    const uint4 *x, *W;
    int row_vecs;
    // backward
    const float* lse;
    const float* g_label;   // [T]: the label's entry of G
    __nv_bfloat16* G;     // [T, ldg]; columns from cols on are never read
    int ldg;
};

struct alignas(16) Shared {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t mma_done;
    uint32_t tmem_base;
    int abort_flag;
};
constexpr int kTransposeBytes = 32 * 128;   // a warp's 32 tokens x 64 columns of G
static_assert(8 * kTransposeBytes <= kStageBytes, "the transposes take the stage they were given");
constexpr size_t kSmemBytes = 1024 + static_cast<size_t>(kMaxStages) * kStageBytes + sizeof(Shared);
static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");

__device__ __forceinline__ uint32_t bar(uint64_t& b) { return moe::smem_u32(&b); }

__device__ __forceinline__ void fail(Shared& S, const Params& p) {
    S.abort_flag = 1;
    moe::raise_device_error(p.err, MOE_DEVERR_TIMEOUT);
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <int kStages>
__device__ void producer(const CUtensorMap* tmX, const CUtensorMap* tmW, uint8_t* stages, Shared& S, const Params& p,
                         int total, uint32_t rank) {
    int stage = 0;
    uint32_t phase = 0, issued = 0, issued_par = 0;
    bool ok = true;
    const int half = p.bv / 2;
    const auto load_w = [&](int st, int kb, int voc) {   // one lane
        if (rank == 0) moe::mbar_arrive_expect_tx(bar(S.full[st]), (p.bt + p.bv) * 128);   // both CTAs' rows
        moe::tma_load_2d_pair(moe::smem_u32(stages + st * kStageBytes) + kStageA, tmW, moe::map_to_cta(bar(S.full[st]), 0),
                              kb * 64, voc);
    };
    // behind the kernel that writes x or reads G: the ring's first rows of W are on
    // their way while it drains
    bool waiting = p.after == moe::After::kPrimary;
    int early = 0;
    for (int t = blockIdx.x >> 1; ok && t < total; t += gridDim.x >> 1) {
        const int row = (t % p.tok_tiles) * BT + static_cast<int>(rank) * (p.bt / 2);
        const int voc = p.v0 + (t / p.tok_tiles) * p.bv + static_cast<int>(rank) * half;
        if (waiting) {
            early = min(p.k_blocks, kStages);
            for (int kb = 0; kb < early; ++kb) {
                if (moe::elect_one()) load_w(kb, kb, voc);
                __syncwarp();
            }
            issued |= (1u << early) - 1;   // in flight from here on (phase 0)
            moe::wait_for_primary();
            waiting = false;
        }
        for (int kb = 0; kb < p.k_blocks; ++kb) {
            const bool got = moe::mbar_wait(bar(S.empty[stage]), phase ^ 1u, &S.abort_flag, kWaitNs);
            if (!__all_sync(0xffffffffu, got)) {
                ok = false;
                break;
            }
            if (moe::elect_one()) {
                if (early == 0) load_w(stage, kb, voc);
                moe::tma_load_2d_pair(moe::smem_u32(stages + stage * kStageBytes), tmX,
                                      moe::map_to_cta(bar(S.full[stage]), 0), kb * 64, row);
            }
            if (early > 0) --early;
            __syncwarp();
            issued |= 1u << stage;
            issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
            if (++stage == kStages) { stage = 0; phase ^= 1u; }
        }
    }
    if (waiting) moe::wait_for_primary();
    if (!ok && moe::elect_one()) {
        fail(S, p);
        int zero = 0;
        if (rank == 0) {
            for (int s = 0; s < kStages; ++s)
                if ((issued >> s) & 1u) moe::mbar_wait(bar(S.full[s]), (issued_par >> s) & 1u, &zero, kDrainNs);
        } else {
            // the peer's loads complete on the leader's barrier: give them time to land
            const uint64_t t0 = moe::global_timer_ns();
            while (moe::global_timer_ns() - t0 < 1000000ull) __nanosleep(1000);
        }
    }
    __syncwarp();
}

template <int kStages>
__device__ void mma_issuer(uint8_t* stages, Shared& S, const Params& p, int total, uint32_t tmem) {
    const uint32_t idesc = moe::make_idesc(1u, p.bt, p.bv);
    int stage = 0, acc = 0;
    uint32_t phase = 0, acc_phase = 0;
    bool ok = true, issued = false;
    for (int t = blockIdx.x >> 1; ok && t < total; t += gridDim.x >> 1) {
        bool got = moe::mbar_wait_cluster(bar(S.acc_empty[acc]), acc_phase ^ 1u, &S.abort_flag, kWaitNs);
        if (!__all_sync(0xffffffffu, got)) { ok = false; break; }
        moe::tc_fence_after();
        const uint32_t d = tmem + static_cast<uint32_t>(acc * BV);
        for (int kb = 0; kb < p.k_blocks; ++kb) {
            got = moe::mbar_wait(bar(S.full[stage]), phase, &S.abort_flag, kWaitNs);
            if (!__all_sync(0xffffffffu, got)) { ok = false; break; }
            moe::tc_fence_after();
            const uint32_t sa = moe::smem_u32(stages + stage * kStageBytes);
            const uint64_t adesc = moe::smem_desc_sw128(sa), bdesc = moe::smem_desc_sw128(sa + kStageA);
            if (moe::elect_one()) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    moe::mma_bf16_pair(d, adesc + 2 * k, bdesc + 2 * k, idesc, (kb | k) != 0);
                moe::tc_commit_pair(bar(S.empty[stage]), 0x3);
            }
            __syncwarp();
            issued = true;
            if (++stage == kStages) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        if (moe::elect_one()) moe::tc_commit_pair(bar(S.acc_full[acc]), 0x3);
        __syncwarp();
        acc ^= 1;
        if (!acc) acc_phase ^= 1u;
    }
    if (!ok && moe::elect_one()) fail(S, p);
    __syncwarp();
    if (issued) {   // every MMA has finished before tensor memory is freed
        int zero = 0;
        if (moe::elect_one()) moe::tc_commit_pair(bar(S.mma_done), 0x1);
        __syncwarp();
        moe::mbar_wait(bar(S.mma_done), 0, &zero, kDrainNs);
    }
}

template <bool BACK>
__device__ void epilogue(uint8_t* stages, Shared& S, const Params& p, int total, uint32_t tmem, uint32_t rank) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int q = warp & 3, hsel = (warp - 4) >> 2;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(q * 32) << 16);
    // backward: the warp's transpose buffer, rows of 128 bytes whose 16-byte
    // pieces are permuted by the row, so that neither side conflicts on banks
    uint4* buf = reinterpret_cast<uint4*>(stages + kStagesOf<BACK> * kStageBytes + (warp - 4) * kTransposeBytes);
    int acc = 0;
    uint32_t acc_phase = 0;
    const uint32_t leader[2] = {moe::map_to_cta(bar(S.acc_empty[0]), 0), moe::map_to_cta(bar(S.acc_empty[1]), 0)};
    // this thread's token within the CTA's, and its accumulator columns: the
    // tile's, or for M = 128 the half of them that its lanes hold
    const bool small = p.bt == 128;
    const int trow = small ? (q & 1) * 32 + lane : q * 32 + lane;
    const int shift = small ? (q >> 1) * (p.bv / 2) : 0, width = small ? p.bv / 2 : p.bv;
    const int chunks = (width + 31) / 32, c_lo = hsel ? (chunks + 1) / 2 : 0, c_hi = hsel ? chunks : (chunks + 1) / 2;
    const int share = small ? 2 * (q >> 1) + hsel : hsel;   // which part of a row's tile this thread reduces
    for (int t = blockIdx.x >> 1; t < total; t += gridDim.x >> 1) {
        const int vt = t / p.tok_tiles;
        const int row = (t % p.tok_tiles) * BT + static_cast<int>(rank) * (p.bt / 2) + trow;
        const int col0 = vt * p.bv + shift;                  // first of its columns within the launch's
        const int ncols = min(width, p.cols - col0);         // those that exist
        const int label = row < p.T ? p.labels[row] : p.ignore;
        const bool counts = label != p.ignore && label >= 0 && label < p.V;
        const int rel = counts ? label - p.v0 - col0 : -1;   // the label's column, in the tile if 0 <= rel < ncols
        float neg_lse = 0.0f, g_label = 0.0f;
        if (BACK && row < p.T) {
            neg_lse = -p.lse[row] * kLog2e;
            g_label = p.g_label[row];
        }
        if (!moe::mbar_wait(bar(S.acc_full[acc]), acc_phase, &S.abort_flag, kWaitNs)) { fail(S, p); return; }
        moe::tc_fence_after();
        const uint32_t ta = lane_base + static_cast<uint32_t>(acc * BV);
        float m = -INFINITY, s = 0.0f;
#pragma unroll 1
        for (int c = c_lo; c < c_hi; ++c) {
            const int col = c * 32;
            uint32_t u[32];
            moe::tmem_ld32(ta + col, u);
            moe::tmem_ld_wait();
            float z[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) z[j] = __uint_as_float(u[j]);
            if (!BACK) {
                if (counts && rel >= col && rel < min(col + 32, ncols))   // the join adds it
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (rel == col + j) z[j] = -INFINITY;
                if (col + 32 > ncols)
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (col + j >= ncols) z[j] = -INFINITY;
                float cm = z[0];
#pragma unroll
                for (int j = 1; j < 32; ++j) cm = fmaxf(cm, z[j]);
                const float nm = fmaxf(m, cm);
                // a piece without any column, or of -inf alone, adds nothing
                const float base = nm == -INFINITY ? 0.0f : nm * kLog2e;
                s *= exp2_approx(fmaf(m, kLog2e, -base));
                m = nm;
#pragma unroll
                for (int j = 0; j < 32; ++j) s += exp2_approx(fmaf(z[j], kLog2e, -base));
            } else {
                float g[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) g[j] = exp2_approx(fmaf(z[j], kLog2e, neg_lse));
                if (counts && rel >= col && rel < min(col + 32, ncols))
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (rel == col + j) g[j] = g_label;
                if (!counts || col + 32 > ncols)
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (!counts || col + j >= ncols) g[j] = 0.0f;
                const int half = (c - c_lo) & 1;   // two chunks fill the buffer
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    buf[lane * 8 + ((4 * half + i) ^ (lane & 7))] =
                        make_uint4(moe::pack_bf16x2(g[8 * i], g[8 * i + 1]), moe::pack_bf16x2(g[8 * i + 2], g[8 * i + 3]),
                                   moe::pack_bf16x2(g[8 * i + 4], g[8 * i + 5]),
                                   moe::pack_bf16x2(g[8 * i + 6], g[8 * i + 7]));
                if (half == 0 && c + 1 < c_hi) continue;
                // eight lanes a token: 128 contiguous bytes of its row of G
                __syncwarp();
                const int first = col - 32 * half, piece = lane & 7;
                const bool in = piece < 4 * (half + 1) && first + 8 * piece < width && col0 + first + 8 * piece < p.ldg;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int r = 4 * i + (lane >> 3), token = row - lane + r;
                    const uint4 v = buf[r * 8 + (piece ^ (r & 7))];
                    if (in && token < p.T)
                        *reinterpret_cast<uint4*>(p.G + static_cast<int64_t>(token) * p.ldg + col0 + first + 8 * piece) = v;
                }
                __syncwarp();
            }
        }
        moe::tc_fence_before();
        if (rank != 0) moe::mbar_arrive_cluster(leader[acc]);
        else moe::mbar_arrive(bar(S.acc_empty[acc]));
        acc ^= 1;
        if (!acc) acc_phase ^= 1u;
        if (!BACK && row < p.T) p.part[static_cast<int64_t>(p.shares * vt + share) * p.T + row] = make_float2(m, s);
    }
}

// A label's logit, by a warp, from x[t] and W[label] in fp32: the same bits in
// both passes.
__device__ __forceinline__ float label_dot(const uint4* __restrict__ x, const uint4* __restrict__ w, int vecs) {
    float dot = 0.0f;
#pragma unroll 4
    for (int c = threadIdx.x & 31; c < vecs; c += 32) {
        const uint4 a = __ldg(x + c), b = __ldg(w + c);
        const uint32_t a4[4] = {a.x, a.y, a.z, a.w}, b4[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            dot = fmaf(moe::bf16_lo(a4[i]), moe::bf16_lo(b4[i]), dot);
            dot = fmaf(moe::bf16_hi(a4[i]), moe::bf16_hi(b4[i]), dot);
        }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
    return dot;
}

// The labels' logits, a warp a token.
__device__ void label_logits(const Params& p, int warp) {
    for (int64_t t = blockIdx.x * 2 + warp; t < p.T; t += gridDim.x * 2) {   // T goes up to INT_MAX - BT
        const int label = p.labels[t];
        if (label == p.ignore || label < 0 || label >= p.V) continue;
        const float dot = label_dot(p.x + t * p.row_vecs,
                                    p.W + static_cast<int64_t>(label) * p.row_vecs, p.row_vecs);
        if ((threadIdx.x & 31) == 0) p.at_label[t] = dot;
    }
}

template <bool BACK>
__global__ void __launch_bounds__(kThreads, 1)
logits_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW, const Params p) {
    const uint32_t rank = moe::cluster_ctarank();   // 0 leads the pair
    extern __shared__ uint8_t smem_raw[];
    uint8_t* stages = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Shared& S = *reinterpret_cast<Shared*>(stages + kMaxStages * kStageBytes);
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kMaxStages; ++s) {
            moe::mbar_init(bar(S.full[s]), 1);
            moe::mbar_init(bar(S.empty[s]), 1);
        }
        for (int a = 0; a < 2; ++a) {
            moe::mbar_init(bar(S.acc_full[a]), 1);
            moe::mbar_init(bar(S.acc_empty[a]), 2 * kEpiThreads);
        }
        moe::mbar_init(bar(S.mma_done), 1);
        S.abort_flag = 0;
        moe::fence_barrier_init();
        moe::prefetch_tensormap(&tmX);
        moe::prefetch_tensormap(&tmW);
    }
    __syncthreads();
    if (warp == 1) {
        moe::tmem_alloc_pair(moe::smem_u32(&S.tmem_base), kTmemCols);
        moe::tmem_relinquish_pair();
    }
    moe::tc_fence_before();
    moe::cluster_sync();   // the peer's barriers exist before anyone signals them
    moe::tc_fence_after();
    const uint32_t tmem = S.tmem_base;
    // the producers wait themselves, behind the first rows of W
    if (BACK && warp != 0) moe::begin_after(p.after);
    const int total = p.tok_tiles * p.voc_tiles;
    if (warp >= 4) epilogue<BACK>(stages, S, p, total, tmem, rank);
    else if (warp == 0) producer<kStagesOf<BACK>>(&tmX, &tmW, stages, S, p, total, rank);
    else if (warp == 1 && rank == 0) mma_issuer<kStagesOf<BACK>>(stages, S, p, total, tmem);
    else if (!BACK && warp >= 2) label_logits(p, warp - 2);
    if (!BACK) moe::launch_dependents();
    moe::tc_fence_before();
    moe::cluster_sync();   // no CTA of the pair leaves while its peer may still signal it
    if (warp == 1) {
        moe::tc_fence_after();
        moe::tmem_dealloc_pair(tmem, kTmemCols);
    }
}

// Joins the vocabulary tiles' (m, s): TOKENS tokens a block, 256 / TOKENS
// threads each, whose shares are merged in a fixed tree.  An ignored or invalid
// label gets loss 0 (the latter is reported).
__device__ __forceinline__ float2 merge(float2 a, float2 b) {
    const float m = fmaxf(a.x, b.x), base = m == -INFINITY ? 0.0f : m;
    return make_float2(m, a.y * expf(a.x - base) + b.y * expf(b.x - base));
}
template <int TOKENS>
__global__ void __launch_bounds__(256)
join_kernel(const float2* part, int parts, const float* at_label,
            const int32_t* __restrict__ labels, int T, int V, int ignore, float* __restrict__ loss,
            float* __restrict__ lse, int* err) {
    constexpr int kShares = 256 / TOKENS;
    __shared__ float2 share[kShares][TOKENS];
    moe::wait_for_primary();
    const int tok = threadIdx.x % TOKENS, g = threadIdx.x / TOKENS;
    const int t = blockIdx.x * TOKENS + tok;
    float2 v = make_float2(-INFINITY, 0.0f);
    if (t < T) {
#pragma unroll 4
        for (int i = g; i < parts; i += kShares) v = merge(v, part[static_cast<int64_t>(i) * T + t]);
    }
    share[g][tok] = v;
    for (int n = kShares / 2; n > 0; n >>= 1) {
        __syncthreads();
        if (g < n) share[g][tok] = merge(share[g][tok], share[g + n][tok]);
    }
    if (g != 0 || t >= T) return;
    const float m = share[0][tok].x, s = share[0][tok].y;
    const int label = labels[t];
    float out = 0.0f, l;
    if (label != ignore && label >= 0 && label < V) {
        const float z = at_label[t], top = fmaxf(m, z);
        const float rest = s * expf(m - top), sum = rest + expf(z - top);
        l = top + logf(sum);
        out = z >= m ? log1pf(rest) : (m - z) + logf(sum);
    } else {
        l = m + logf(s);
        if (label != ignore) moe::raise_device_error(err, MOE_DEVERR_LABEL);
    }
    loss[t] = out;
    lse[t] = l;
}

// Backward's per-token factors: scale[t] = dloss[t], 0 where the label is
// ignored or invalid (the latter is reported), scale[T] = the largest
// magnitude among them; offsets = {0, T}.  One block.
__global__ void __launch_bounds__(1024)
scale_kernel(const float* __restrict__ dloss, const int32_t* __restrict__ labels, int T, int V, int ignore,
             float* __restrict__ scale, int32_t* __restrict__ offsets, int* err) {
    __shared__ float part[32];
    moe::launch_dependents();
    float top = 0.0f;
    bool bad = false;
    for (int64_t t = threadIdx.x; t < T; t += 1024) {   // T goes up to INT_MAX - BT
        const int label = labels[t];
        const bool counts = label != ignore && label >= 0 && label < V;
        const float d = counts ? dloss[t] : 0.0f;
        bad |= !counts && label != ignore;
        scale[t] = d;
        top = fmaxf(top, fabsf(d));
    }
    if (bad) moe::raise_device_error(err, MOE_DEVERR_LABEL);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = top;
    __syncthreads();
    if (threadIdx.x < 32) {
        top = part[threadIdx.x];
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        if (threadIdx.x == 0) {
            scale[T] = top;
            offsets[0] = 0;
            offsets[1] = T;
        }
    }
}

// A warp a token:  g_label[t] = exp(z_l - lse[t]) - 1 with the label's logit as in
// the forward pass (the tensor cores' would be off by more than a nearly certain
// label's entry);  xs[t] = bf16(scale[t] / scale[T] * x[t]), zeros where scale[t] is
// 0, and a copy xa of x (either may be NULL), rows ld_vecs vectors apart: whole
// 128-byte lines, so that no box of the products that read them straddles two.
__global__ void __launch_bounds__(256)
token_rows_kernel(const uint4* __restrict__ x, const uint4* __restrict__ W, const int32_t* __restrict__ labels,
                  const float* __restrict__ lse, const float* scale, int T, int V, int ignore, int row_vecs, int ld_vecs,
                  float* __restrict__ g_label, uint4* __restrict__ xs, uint4* __restrict__ xa) {
    moe::begin_after(moe::After::kPrimary);
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (t >= T) return;
    const int label = labels[t];
    if (label != ignore && label >= 0 && label < V) {   // the same for the whole warp
        const float z = label_dot(x + static_cast<int64_t>(t) * row_vecs, W + static_cast<int64_t>(label) * row_vecs, row_vecs);
        if (lane == 0) g_label[t] = expm1f(z - lse[t]);
    }
    if (!xs && !xa) return;
    const float d = scale[t], r = d == 0.0f ? 0.0f : __fdiv_rn(d, scale[T]);
    for (int c = lane; c < row_vecs; c += 32) {
        const uint4 v = __ldg(x + static_cast<int64_t>(t) * row_vecs + c);
        if (xa) xa[static_cast<int64_t>(t) * ld_vecs + c] = v;
        if (!xs) continue;
        const uint32_t a[4] = {v.x, v.y, v.z, v.w};
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o[i] = d == 0.0f ? 0u : moe::pack_bf16x2(r * moe::bf16_lo(a[i]), r * moe::bf16_hi(a[i]));
        xs[static_cast<int64_t>(t) * ld_vecs + c] = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

// dx[t] = scale[t] * (the ranges' sums, in range order), four columns a thread.
__global__ void __launch_bounds__(256)
finish_kernel(const float4* sum, int splits, int64_t n, int row_quads, const float* scale, uint2* dx) {
    moe::wait_for_primary();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= n) return;
    float4 a = sum[i];
#pragma unroll 4
    for (int r = 1; r < splits; ++r) {
        const float4 b = sum[r * n + i];
        a.x += b.x;
        a.y += b.y;
        a.z += b.z;
        a.w += b.w;
    }
    const float d = scale[i / row_quads];
    dx[i] = make_uint2(moe::pack_bf16x2(d * a.x, d * a.y), moe::pack_bf16x2(d * a.z, d * a.w));
}

// ---------------------------------------------------------------- host side
bool valid_sizes(int T, int H, int V) {
    return T >= 1 && V >= 1 && H >= 8 && H % 8 == 0 && V <= INT_MAX - BV && T <= INT_MAX - BT &&
           (static_cast<int64_t>(T) / BT + 1) * (static_cast<int64_t>(V) / 16 + 1) < INT_MAX;
}

// Vocabulary rows of a tile for `cols` of them and T tokens: a multiple of 16,
// or of 32 for M = 128 MMAs.
int tile_width(int cols, int T) {
    const int tok_tiles = (T + BT - 1) / BT, step = T <= 128 ? 32 : 16;
    const int pairs = moe::sm_count() / 2 > 0 ? moe::sm_count() / 2 : 76;
    const auto rounds = [&](int bv) {
        return (static_cast<int64_t>((cols + bv - 1) / bv) * tok_tiles + pairs - 1) / pairs;
    };
    const int64_t least = rounds(BV);
    int bv = BV;
    while (bv > 32 && rounds(bv - step) == least) bv -= step;
    return bv;
}

// x's rows start ldx elements apart.
template <bool BACK>
moe_status_t launch_logits(const void* x, int ldx, const void* W, int H, int V, Params p, cudaStream_t s) {
    CUtensorMap tmX, tmW;
    const cuuint64_t stride[1] = {static_cast<cuuint64_t>(H) * 2}, stride_x[1] = {static_cast<cuuint64_t>(ldx) * 2};
    const cuuint64_t dx[2] = {static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(p.T)};
    const cuuint64_t dw[2] = {static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(V)};
    const cuuint32_t bx[2] = {64, static_cast<cuuint32_t>(p.bt / 2)}, bw[2] = {64, static_cast<cuuint32_t>(p.bv / 2)};
    if (!moe::encode_tile_map(&tmX, false, x, 2, dx, stride_x, bx) ||
        !moe::encode_tile_map(&tmW, false, W, 2, dw, stride, bw))
        return MOE_ERR_CUDA;
    auto kern = logits_kernel<BACK>;
    static std::atomic<int> configured[moe::kMaxDevices];
    int dev = 0;
    MOE_CHECK_CUDA(cudaGetDevice(&dev));
    if (dev < 0 || dev >= moe::kMaxDevices) return MOE_ERR_CUDA;
    if (!configured[dev].load(std::memory_order_relaxed)) {
        MOE_CHECK_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                            static_cast<int>(kSmemBytes)));
        configured[dev].store(1, std::memory_order_relaxed);
    }
    const int64_t tiles = static_cast<int64_t>(p.tok_tiles) * p.voc_tiles;
    int pairs = moe::sm_count() / 2;
    if (pairs <= 0) return MOE_ERR_CUDA;
    if (tiles < pairs) pairs = static_cast<int>(tiles);
    return moe::launch_pairs(kern, 2 * pairs, kThreads, kSmemBytes, s, p.after, tmX, tmW, p);
}

struct Carver {
    size_t off = 0;
    size_t take(size_t bytes) {
        const size_t at = off;
        off += (bytes + 255) & ~static_cast<size_t>(255);
        return at;
    }
};

struct ForwardLayout {
    int tok_tiles, bv, voc_tiles;
    size_t part, at_label, total;
};
ForwardLayout forward_layout(int T, int V) {
    ForwardLayout l{};
    l.tok_tiles = (T + BT - 1) / BT;
    l.bv = tile_width(V, T);
    l.voc_tiles = (V + l.bv - 1) / l.bv;
    Carver c;
    l.part = c.take(static_cast<size_t>(T <= 128 ? 4 : 2) * l.voc_tiles * T * sizeof(float2));
    l.at_label = c.take(static_cast<size_t>(T) * sizeof(float));
    l.total = c.off;
    return l;
}

// A piece's G takes up to kPieceBytes, but a piece has at least kPieceMin
// vocabulary rows, whatever G takes then (more than 65536 tokens): every piece
// but the last reads and writes dx's fp32 sum.
constexpr int64_t kPieceBytes = 256ll << 20;
constexpr int kPieceMin = 2048;

struct BackwardLayout {
    int piece, pieces, ldg, splits, ldx;
    size_t G, xs, xa, g_label, scale, offsets, sum, total;
};
BackwardLayout backward_layout(int T, int H, int V) {
    BackwardLayout l{};
    int64_t piece = kPieceBytes / 2 / T / BV * BV;
    if (piece < kPieceMin) piece = kPieceMin;
    if (piece > V) piece = V;
    const int64_t pieces = (V + piece - 1) / piece;   // V goes up to INT_MAX - BV: sums with it in 64 bits
    l.piece = pieces == 1 ? V : static_cast<int>(((V + pieces - 1) / pieces + BV - 1) / BV * BV);
    l.pieces = (V - 1) / l.piece + 1;
    l.ldg = (l.piece + 63) / 64 * 64;   // rows of whole 128-byte lines
    Carver c;
    l.G = c.take(static_cast<size_t>(T) * l.ldg * 2);
    l.ldx = (H + 63) / 64 * 64;
    l.xs = c.take(static_cast<size_t>(T) * l.ldx * 2);
    l.xa = c.take(l.ldx == H ? 0 : static_cast<size_t>(T) * l.ldx * 2);
    l.g_label = c.take(static_cast<size_t>(T) * sizeof(float));
    l.scale = c.take((static_cast<size_t>(T) + 1) * sizeof(float));
    l.offsets = c.take(2 * sizeof(int32_t));
    l.splits = moe::dgrad_sum_splits(T, l.piece, H);
    l.sum = c.take(l.pieces > 1 || l.splits > 1 ? static_cast<size_t>(l.splits) * T * H * sizeof(float) : 0);
    l.total = c.off;
    return l;
}

}  // namespace

extern "C" size_t moe_cross_entropy_forward_workspace_size(int T, int H, int V) {
    return valid_sizes(T, H, V) ? forward_layout(T, V).total : 0;
}

extern "C" moe_status_t moe_cross_entropy_forward(const void* x, const void* W, const int32_t* labels, int T, int H,
                                                  int V, int ignore_index, float* loss, float* lse, void* ws,
                                                  size_t ws_bytes, moe_stream_t stream) {
    MOE_CHECK_ARG(x && W && labels && loss && lse && valid_sizes(T, H, V));
    MOE_CHECK_ARG(moe::aligned16(x) && moe::aligned16(W) && moe::aligned16(labels) && moe::aligned16(loss) &&
                  moe::aligned16(lse));
    const ForwardLayout l = forward_layout(T, V);
    if (!ws || ws_bytes < l.total) return MOE_ERR_WORKSPACE;
    MOE_CHECK_ARG(moe::aligned16(ws));
    int* err = moe::device_error_word();
    if (!err) return MOE_ERR_CUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    auto* base = static_cast<uint8_t*>(ws);
    Params p{};
    p.labels = labels;
    p.err = err;
    p.T = T;
    p.k_blocks = (H + 63) / 64;
    p.cols = V;
    p.bt = T <= 128 ? 128 : BT;
    p.shares = T <= 128 ? 4 : 2;
    p.bv = l.bv;
    p.tok_tiles = l.tok_tiles;
    p.voc_tiles = l.voc_tiles;
    p.ignore = ignore_index;
    p.part = reinterpret_cast<float2*>(base + l.part);
    p.at_label = reinterpret_cast<float*>(base + l.at_label);
    p.x = static_cast<const uint4*>(x);
    p.W = static_cast<const uint4*>(W);
    p.V = V;
    p.row_vecs = H / 8;
    const moe_status_t st = launch_logits<false>(x, H, W, H, V, p, s);
    if (st != MOE_OK) return st;
    // neighbouring tokens' pairs share a sector; with few tokens the latency of
    // a token's own pairs counts
    const bool few = T < 8 * moe::sm_count();
    return moe::launch_after(few ? join_kernel<1> : join_kernel<8>, dim3(few ? T : (T + 7) / 8), 256, 0, s,
                             static_cast<const float2*>(p.part), p.shares * l.voc_tiles,
                             static_cast<const float*>(p.at_label), labels, T, V, ignore_index, loss, lse, err);
}

extern "C" size_t moe_cross_entropy_backward_workspace_size(int T, int H, int V) {
    return valid_sizes(T, H, V) ? backward_layout(T, H, V).total : 0;
}

extern "C" moe_status_t moe_cross_entropy_backward(const void* x, const void* W, const int32_t* labels,
                                                   const float* lse, const float* dloss, int T, int H, int V,
                                                   int ignore_index, void* dx, void* dW, void* ws, size_t ws_bytes,
                                                   moe_stream_t stream) {
    MOE_CHECK_ARG(x && W && labels && lse && dloss && (dx || dW) && valid_sizes(T, H, V));
    MOE_CHECK_ARG(moe::aligned16(x) && moe::aligned16(W) && moe::aligned16(labels) && moe::aligned16(lse) &&
                  moe::aligned16(dloss) && moe::aligned16(dx) && moe::aligned16(dW));
    const BackwardLayout l = backward_layout(T, H, V);
    if (!ws || ws_bytes < l.total) return MOE_ERR_WORKSPACE;
    MOE_CHECK_ARG(moe::aligned16(ws));
    int* err = moe::device_error_word();
    if (!err) return MOE_ERR_CUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    auto* base = static_cast<uint8_t*>(ws);
    auto* G = reinterpret_cast<__nv_bfloat16*>(base + l.G);
    void* xs = base + l.xs;
    void* xa = l.ldx == H ? nullptr : base + l.xa;   // x in whole lines (1021 x 1000, V = 50257: 283 -> 275 us)
    auto* g_label = reinterpret_cast<float*>(base + l.g_label);
    auto* scale = reinterpret_cast<float*>(base + l.scale);
    auto* offsets = reinterpret_cast<int32_t*>(base + l.offsets);
    auto* sum = l.pieces > 1 || l.splits > 1 ? reinterpret_cast<float*>(base + l.sum) : nullptr;
    scale_kernel<<<1, 1024, 0, s>>>(dloss, labels, T, V, ignore_index, scale, offsets, err);
    MOE_CHECK_LAUNCH();
    moe_status_t st = moe::launch_after(
        token_rows_kernel, dim3((T + 7) / 8), 256, 0, s, static_cast<const uint4*>(x), static_cast<const uint4*>(W), labels,
        lse, static_cast<const float*>(scale), T, V, ignore_index, H / 8, l.ldx / 8, g_label,
        static_cast<uint4*>(dW ? xs : nullptr), static_cast<uint4*>(xa));
    if (st != MOE_OK) return st;
    for (int i = 0; i < l.pieces; ++i) {
        Params p{};
        p.labels = labels;
        p.err = err;
        p.T = T;
        p.k_blocks = (H + 63) / 64;
        p.v0 = i * l.piece;
        p.cols = V - p.v0 < l.piece ? V - p.v0 : l.piece;
        p.tok_tiles = (T + BT - 1) / BT;
        p.bt = T <= 128 ? 128 : BT;
        p.bv = tile_width(p.cols, T);
        p.voc_tiles = (p.cols + p.bv - 1) / p.bv;
        p.ignore = ignore_index;
        p.V = V;
        p.lse = lse;
        p.G = G;
        p.ldg = l.ldg;
        p.g_label = g_label;
        p.after = moe::After::kPrimary;
        st = launch_logits<true>(xa ? xa : x, l.ldx, W, H, V, p, s);
        if (st != MOE_OK) return st;
        const auto* Wp = static_cast<const __nv_bfloat16*>(W) + static_cast<int64_t>(p.v0) * H;
        if (dx && (st = moe::dgrad_sum_gemm(G, l.ldg, Wp, offsets, T, p.cols, H, sum, l.splits, i == 0,
                                            l.splits == 1 && i == l.pieces - 1, scale, dx, s,
                                            moe::After::kPrimary)) != MOE_OK)
            return st;
        if (dW) {
            auto* dWp = static_cast<__nv_bfloat16*>(dW) + static_cast<int64_t>(p.v0) * H;
            // needs nothing of dx's product: takes the SMs that it frees (1021 x 1000: 264 -> 261 us)
            st = moe::wgrad_gemm(G, l.ldg, xs, l.ldx, nullptr, nullptr, offsets, 1, T, p.cols, H, dWp, s,
                                 dx ? moe::After::kBeside : moe::After::kPrimary, scale + T);
            if (st != MOE_OK) return st;
        }
    }
    if (dx && l.splits > 1) {
        const int64_t n = static_cast<int64_t>(T) * (H / 4);
        return moe::launch_after(finish_kernel, dim3(static_cast<unsigned>((n + 255) / 256)), 256, 0, s,
                                 reinterpret_cast<const float4*>(sum), l.splits, n, H / 4,
                                 static_cast<const float*>(scale), static_cast<uint2*>(dx));
    }
    return MOE_OK;
}
