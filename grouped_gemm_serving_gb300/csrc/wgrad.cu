// The weight-gradient GEMM of the grouped GEMM C[p, n] = sum_c A[p, c] B[e, n, c]:
//   dB[e, n, c] = sum over expert e's rows p of dC[p, n] A[p, c].
// The contraction runs over an expert's own rows, some hundreds of them, and
// the output is every weight, so a tile has few k-blocks and its epilogue's
// stores matter as much as its MMAs.
//
// CTA pairs (clusters of two, tcgen05 cta_group::2): a tile is 256 output rows
// (128 per CTA, the MMA's M rows, from dC's columns) x up to 256 output columns
// (half staged by each CTA, the MMA's N, from A's columns; the last tile's N is
// what is left, rounded up to 16).
// Both operands are read in place, MN-major, as 64-column x 64-row boxes of
// 128-byte swizzled rows: four boxes (32 KB) a CTA and k-block, six stages.  A
// lane of the accumulator is an output row, so a warp's 32 rows x 64 columns
// go through a 4 KB transpose and leave as whole 128-byte lines.  (With the
// roles of dC and A exchanged a warp store covered 64 bytes of one output row:
// the path from the SM to L2 was busy for 56 % of the time with the requests
// and a tile's stores took as long as its MMAs.)
//
// An expert's last, partial k-block (cnt mod 64 rows) comes from a copy of its
// rows, zero-padded to a multiple of 16 (the tails), so that no MMA reaches
// into the next expert's rows; the 16-row steps that hold no row are skipped.
// Tiles are walked column tile first: the pairs that run together share dC's
// columns.  Every wait is bounded (2 s); on expiry the CTA records
// MOE_DEVERR_TIMEOUT, waits for its loads and MMAs and leaves.
#include <climits>

#include "common.cuh"
#include "internal.h"

namespace {

constexpr int kStages = 6;
constexpr int kOperand = 2 * 64 * 128;          // two 64-column x 64-row boxes
constexpr int kStageBytes = 2 * kOperand;
constexpr int kTransposeBytes = 32 * 128;       // a warp's 32 output rows x 64 columns
constexpr int BR = 256, BC = 256;               // output rows and columns of a pair's tile
constexpr int kEpiThreads = 256;
constexpr int kThreads = 128 + kEpiThreads;     // warp 0 loads, warp 1 issues MMAs, warps 4-11 store
constexpr uint32_t kTmemCols = 512;
constexpr uint64_t kWaitNs = 2000000000ull, kDrainNs = 100000000ull;
constexpr int kMaxE = 256;

struct Params {
    const int32_t* offsets;
    __nv_bfloat16* out;    // [E, N, K]
    const float* scale;    // one factor for all of it, or NULL
    int* err;
    int E, M_cap, N, K;
    int row_tiles, col_tiles;
    moe::After after;
    int tails;             // 0: rows past offsets[E] lie outside the tensor maps (zeros)
};

struct alignas(16) Shared {
    uint64_t full[kStages], empty[kStages];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t mma_done;
    uint32_t tmem_base;
    int abort_flag;
};
constexpr size_t kSmemBytes = 1024 + static_cast<size_t>(kStages) * kStageBytes + 8 * kTransposeBytes + sizeof(Shared);
static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");

struct Maps {
    CUtensorMap c, a, tail_c, tail_a;
};

struct Tile {
    int e, row0, col0;
    int first, rows;   // the expert's rows
    int nkb, last;     // its k-blocks, and the 16-row steps of the last one
    int bc;            // the tile's columns, rounded up to 16
};

__device__ __forceinline__ Tile decode(int t, const Params& p) {
    const int per = p.row_tiles * p.col_tiles;
    Tile ti;
    ti.e = t / per;
    t -= ti.e * per;
    ti.row0 = t / p.col_tiles * BR;
    ti.col0 = t % p.col_tiles * BC;
    ti.bc = min(BC, (p.K - ti.col0 + 15) & ~15);
    ti.first = p.offsets[ti.e];
    ti.rows = p.offsets[ti.e + 1] - ti.first;
    ti.nkb = (ti.rows + 63) / 64;
    ti.last = (ti.rows - (ti.nkb - 1) * 64 + 15) / 16;
    return ti;
}

__device__ __forceinline__ uint32_t bar(uint64_t& b) { return moe::smem_u32(&b); }

__device__ __forceinline__ void fail(Shared& S, const Params& p) {
    S.abort_flag = 1;
    moe::raise_device_error(p.err, MOE_DEVERR_TIMEOUT);
}

__device__ void producer(const Maps& maps, uint8_t* stages, Shared& S, const Params& p, int total, uint32_t rank) {
    int stage = 0;
    uint32_t phase = 0, issued = 0, issued_par = 0;
    bool ok = true;
    for (int t = blockIdx.x >> 1; ok && t < total; t += gridDim.x >> 1) {
        const Tile ti = decode(t, p);
        const int half = ti.bc / 2, boxes = half > 64 ? 2 : 1;   // this CTA's columns of A
        const int n0 = ti.row0 + static_cast<int>(rank) * 128, c0 = ti.col0 + static_cast<int>(rank) * half;
        const int whole = p.tails ? ti.rows / 64 : ti.nkb;   // k-blocks read in place
        for (int kb = 0; kb < ti.nkb; ++kb) {
            const bool got = moe::mbar_wait(bar(S.empty[stage]), phase ^ 1u, &S.abort_flag, kWaitNs);
            if (!__all_sync(0xffffffffu, got)) {
                ok = false;
                break;
            }
            const uint32_t fb = moe::map_to_cta(bar(S.full[stage]), 0);
            const uint32_t sc = moe::smem_u32(stages + stage * kStageBytes), sa = sc + kOperand;
            if (moe::elect_one()) {
                if (rank == 0) moe::mbar_arrive_expect_tx(bar(S.full[stage]), 2 * (2 + boxes) * 8192);
                const CUtensorMap* mc = kb < whole ? &maps.c : &maps.tail_c;
                const CUtensorMap* ma = kb < whole ? &maps.a : &maps.tail_a;
                const int row = kb < whole ? ti.first + kb * 64 : ti.e * 64;
                moe::tma_load_2d_pair(sc, mc, fb, n0, row);
                moe::tma_load_2d_pair(sc + 8192, mc, fb, n0 + 64, row);
                moe::tma_load_2d_pair(sa, ma, fb, c0, row);
                if (boxes > 1) moe::tma_load_2d_pair(sa + 8192, ma, fb, c0 + 64, row);
            }
            __syncwarp();
            issued |= 1u << stage;
            issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
            if (++stage == kStages) { stage = 0; phase ^= 1u; }
        }
    }
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

__device__ void mma_issuer(uint8_t* stages, Shared& S, const Params& p, int total, uint32_t tmem) {
    int stage = 0, acc = 0;
    uint32_t phase = 0, acc_phase = 0;
    bool ok = true, issued = false;
    for (int t = blockIdx.x >> 1; ok && t < total; t += gridDim.x >> 1) {
        const Tile ti = decode(t, p);
        const uint32_t idesc = moe::make_idesc_ab_mn(1u, BR, ti.bc);
        bool got = moe::mbar_wait_cluster(bar(S.acc_empty[acc]), acc_phase ^ 1u, &S.abort_flag, kWaitNs);
        if (!__all_sync(0xffffffffu, got)) { ok = false; break; }
        moe::tc_fence_after();
        const uint32_t d = tmem + static_cast<uint32_t>(acc * BC);
        // an expert without rows has no k-blocks: its accumulator is committed
        // untouched and the epilogue writes zeros
        for (int kb = 0; kb < ti.nkb; ++kb) {
            got = moe::mbar_wait(bar(S.full[stage]), phase, &S.abort_flag, kWaitNs);
            if (!__all_sync(0xffffffffu, got)) { ok = false; break; }
            moe::tc_fence_after();
            const uint32_t sc = moe::smem_u32(stages + stage * kStageBytes);
            // 64-column atoms 8 KB apart; a step of 16 rows is 2 KB further on
            const uint64_t cdesc = moe::smem_desc_sw128_mn(sc, 8192);
            const uint64_t adesc = moe::smem_desc_sw128_mn(sc + kOperand, 8192);
            const int steps = kb + 1 < ti.nkb ? 4 : ti.last;
            if (moe::elect_one()) {
                for (int k = 0; k < steps; ++k)
                    moe::mma_bf16_pair(d, cdesc + (2048 >> 4) * k, adesc + (2048 >> 4) * k, idesc, (kb | k) != 0);
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

__device__ void epilogue(uint8_t* transposes, Shared& S, const Params& p, int total, uint32_t tmem, uint32_t rank) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int q = warp & 3, hsel = (warp - 4) >> 2;   // lanes 32 q.., columns 128 hsel.. of the tile
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(q * 32) << 16);
    uint4* buf = reinterpret_cast<uint4*>(transposes + (warp - 4) * kTransposeBytes);
    int acc = 0;
    uint32_t acc_phase = 0;
    const uint32_t leader[2] = {moe::map_to_cta(bar(S.acc_empty[0]), 0), moe::map_to_cta(bar(S.acc_empty[1]), 0)};
    const float scale = p.scale ? *p.scale : 1.0f;
    const int piece = lane & 7;
    for (int t = blockIdx.x >> 1; t < total; t += gridDim.x >> 1) {
        const Tile ti = decode(t, p);
        const int n0 = ti.row0 + static_cast<int>(rank) * 128 + q * 32;   // the warp's first output row
        const int col0 = ti.col0 + hsel * 128;
        const int ncols = min(128, p.K - col0);   // its columns that exist
        if (!moe::mbar_wait(bar(S.acc_full[acc]), acc_phase, &S.abort_flag, kWaitNs)) { fail(S, p); return; }
        moe::tc_fence_after();
        // the whole share is packed into registers at once, so that the
        // accumulator goes back to the MMAs before anything is stored
        uint32_t w[2][32];
        const uint32_t ta = lane_base + static_cast<uint32_t>(acc * BC + hsel * 128);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            uint32_t v[2][32];
            moe::tmem_ld32(ta + c * 64, v[0]);
            moe::tmem_ld32(ta + c * 64 + 32, v[1]);
            moe::tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j)
                w[c][j] = moe::pack_bf16x2(scale * __uint_as_float(v[j / 16][2 * (j % 16)]),
                                           scale * __uint_as_float(v[j / 16][2 * (j % 16) + 1]));
        }
        moe::tc_fence_before();
        if (rank != 0) moe::mbar_arrive_cluster(leader[acc]);
        else moe::mbar_arrive(bar(S.acc_empty[acc]));
        acc ^= 1;
        if (!acc) acc_phase ^= 1u;
        if (ti.nkb == 0)   // an expert without rows has an accumulator that nothing wrote
#pragma unroll
            for (int j = 0; j < 32; ++j) w[0][j] = w[1][j] = 0u;
        __nv_bfloat16* out = p.out + (static_cast<int64_t>(ti.e) * p.N + n0) * p.K + col0 + 8 * piece;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            if (c * 64 >= ncols) break;   // the same for the whole warp
#pragma unroll
            for (int i = 0; i < 8; ++i)
                buf[lane * 8 + (i ^ (lane & 7))] = make_uint4(w[c][4 * i], w[c][4 * i + 1], w[c][4 * i + 2], w[c][4 * i + 3]);
            __syncwarp();
            // eight lanes an output row: 128 contiguous bytes of it
            const bool in = c * 64 + 8 * piece < ncols;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = 4 * i + (lane >> 3);
                const uint4 o = buf[r * 8 + (piece ^ (r & 7))];
                if (in && n0 + r < p.N) *reinterpret_cast<uint4*>(out + static_cast<int64_t>(r) * p.K + c * 64) = o;
            }
            __syncwarp();
        }
    }
}

__global__ void __launch_bounds__(kThreads, 1)
wgrad_kernel(const __grid_constant__ Maps maps, const Params p) {
    const uint32_t rank = moe::cluster_ctarank();   // 0 leads the pair
    extern __shared__ uint8_t smem_raw[];
    uint8_t* stages = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* transposes = stages + kStages * kStageBytes;
    Shared& S = *reinterpret_cast<Shared*>(transposes + 8 * kTransposeBytes);
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
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
        moe::prefetch_tensormap(&maps.c);
        moe::prefetch_tensormap(&maps.a);
    }
    int bad = 0;
    for (int i = threadIdx.x; i < p.E; i += kThreads) bad |= p.offsets[i + 1] < p.offsets[i];
    if (threadIdx.x == 0) bad |= p.offsets[0] != 0 || p.offsets[p.E] > p.M_cap;
    if (__syncthreads_or(bad)) {   // both CTAs of a pair read the same offsets and leave together
        if (threadIdx.x == 0) moe::raise_device_error(p.err, MOE_DEVERR_OFFSETS);
        return;
    }
    if (warp == 1) {
        moe::tmem_alloc_pair(moe::smem_u32(&S.tmem_base), kTmemCols);
        moe::tmem_relinquish_pair();
    }
    moe::tc_fence_before();
    moe::cluster_sync();   // the peer's barriers exist before anyone signals them
    moe::tc_fence_after();
    const uint32_t tmem = S.tmem_base;
    moe::begin_after(p.after);
    const int total = p.E * p.row_tiles * p.col_tiles;
    if (warp >= 4) epilogue(transposes, S, p, total, tmem, rank);
    else if (warp == 0) producer(maps, stages, S, p, total, rank);
    else if (warp == 1 && rank == 0) mma_issuer(stages, S, p, total, tmem);
    moe::end_after(p.after);
    moe::tc_fence_before();
    moe::cluster_sync();   // no CTA of the pair leaves while its peer may still signal it
    if (warp == 1) {
        moe::tc_fence_after();
        moe::tmem_dealloc_pair(tmem, kTmemCols);
    }
}

bool encode_operand(CUtensorMap* map, const void* base, int cols, int ld, int64_t rows) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
    const cuuint32_t box[2] = {64, 64};
    return moe::encode_tile_map(map, false, base, 2, dims, strides, box);
}

}  // namespace

moe_status_t moe::wgrad_gemm(const void* dC, int ldc, const void* A, int lda, const void* tail_c, const void* tail_a,
                             const int32_t* offsets, int E, int M_cap, int N, int K, void* dB, cudaStream_t s,
                             After after, const float* scale) {
    MOE_CHECK_ARG(dC && A && (tail_c && tail_a ? true : E == 1) && offsets && dB && E >= 1 && E <= kMaxE && M_cap >= 1);
    MOE_CHECK_ARG(N >= 1 && ldc >= N && ldc % 8 == 0 && K >= 8 && K % 8 == 0 && lda >= K && lda % 8 == 0);
    MOE_CHECK_ARG(moe::aligned16(dC) && moe::aligned16(A) && moe::aligned16(tail_c) && moe::aligned16(tail_a) &&
                  moe::aligned16(dB));
    Params p{};
    p.offsets = offsets;
    p.out = static_cast<__nv_bfloat16*>(dB);
    p.scale = scale;
    p.after = after;
    p.err = moe::device_error_word();
    if (!p.err) return MOE_ERR_CUDA;
    p.E = E;
    p.M_cap = M_cap;
    p.N = N;
    p.K = K;
    p.row_tiles = (N - 1) / BR + 1;
    p.col_tiles = (K - 1) / BC + 1;
    p.tails = tail_c && tail_a;
    const int64_t tiles = static_cast<int64_t>(E) * p.row_tiles * p.col_tiles;
    MOE_CHECK_ARG(tiles < INT_MAX);
    Maps maps;
    if (!encode_operand(&maps.c, dC, N, ldc, M_cap) || !encode_operand(&maps.a, A, K, lda, M_cap)) return MOE_ERR_CUDA;
    maps.tail_c = maps.c;
    maps.tail_a = maps.a;
    if (p.tails && (!encode_operand(&maps.tail_c, tail_c, N, N, 64ll * E) || !encode_operand(&maps.tail_a, tail_a, K, K, 64ll * E)))
        return MOE_ERR_CUDA;
    static std::atomic<int> configured[moe::kMaxDevices];
    int dev = 0;
    MOE_CHECK_CUDA(cudaGetDevice(&dev));
    if (dev < 0 || dev >= moe::kMaxDevices) return MOE_ERR_CUDA;
    if (!configured[dev].load(std::memory_order_relaxed)) {
        MOE_CHECK_CUDA(cudaFuncSetAttribute(wgrad_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                            static_cast<int>(kSmemBytes)));
        configured[dev].store(1, std::memory_order_relaxed);
    }
    int pairs = moe::sm_count() / 2;
    if (pairs <= 0) return MOE_ERR_CUDA;
    if (tiles < pairs) pairs = static_cast<int>(tiles);
    return moe::launch_pairs(wgrad_kernel, 2 * pairs, kThreads, kSmemBytes, s, p.after, maps, p);
}
