// moe_layer_norm_backward: with xh = (x - mean) * rstd and g = dy * weight,
//   dx = rstd * (g - sum(g) / H - xh * sum(g * xh) / H)      per row,
//   dweight = sum over rows of dy * xh,   dbias = sum over rows of dy.
//
// One pass: a row's x and dy are read once, held in registers while the two
// row sums are taken, and dx is written; bound by HBM.  Blocks are persistent
// and a thread owns the same columns in every row, so it sums its share of
// dweight and dbias in fp32 registers as it goes.  Each block then writes one
// partial row of each to the workspace, and a second small kernel adds the
// partial rows in block order: no atomics, the same bits every time.
//
// Wide rows that start on 16-byte boundaries come through shared memory: one
// thread keeps a ring of rows in flight with bulk copies (TMA), so that the
// loads of the next rows run under the present row's sums and barrier without
// taking registers.  All others are loaded straight into registers.
#include <climits>

#include "norm.cuh"

namespace {

using namespace moe::norm;

// Adds a thread's columns to the block's partial row of dweight and dbias.
template <int VEC, int TEAM, int EPT>
__device__ __forceinline__ void store_partial(float* pw, int H, int lane, const float (&dw)[EPT],
                                              const float (&db)[EPT]) {
#pragma unroll
    for (int i = 0; i < EPT / VEC; ++i) {
        const int c = (i * TEAM + lane) * VEC;
        if (c < H)
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                pw[c + j] = dw[i * VEC + j];
                pw[H + c + j] = db[i * VEC + j];
            }
    }
}

template <typename T, typename W, int VEC, int TEAM, int EPT>
__global__ void __launch_bounds__(TEAM <= 32 ? 256 : TEAM)
norm_backward_kernel(const T* dy, int64_t lddy, const T* x, int64_t ldx, int rows, int H,
                     const W* __restrict__ weight, const float* __restrict__ mean_in,
                     const float* __restrict__ rstd_in, T* dx, int64_t lddx,
                     float* __restrict__ partial) {
    constexpr int NV = EPT / VEC;
    constexpr int kTeams = TEAM <= 32 ? 256 / TEAM : 1;
    __shared__ float slots[TEAM <= 32 ? 1 : 128];
    const int lane = threadIdx.x % TEAM, team = threadIdx.x / TEAM;
    const float inv_h = 1.0f / static_cast<float>(H);
    const int step = gridDim.x * kTeams;
    int turn = 0;
    Raw<W, VEC> w[NV];
    float dw[EPT], db[EPT];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TEAM + lane) * VEC;
        if (c < H && weight) w[i] = load_raw<W, VEC>(weight + c);
    }
#pragma unroll
    for (int i = 0; i < EPT; ++i) dw[i] = db[i] = 0.0f;
    Raw<T, VEC> xn[NV], gn[NV];
    float mean_n = 0.0f, rstd_n = 0.0f;
    const auto fetch = [&](int64_t row) {   // the next row's loads run under the present row's sums
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TEAM + lane) * VEC;
            if (c < H) {
                xn[i] = load_raw<T, VEC>(x + row * ldx + c);
                gn[i] = load_raw<T, VEC>(dy + row * lddy + c);
            }
        }
        mean_n = mean_in[row];
        rstd_n = rstd_in[row];
    };
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kTeams;   // the block's first row of a step
    if (row0 + team < rows) fetch(row0 + team);
    // teams of a warp or less share its shuffles: the trip count is the block's
    for (int64_t at = row0; at < rows; at += step) {
        const int64_t row = at + team;
        const bool live = row < rows;
        Raw<T, VEC> xr[NV], gr[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) { xr[i] = xn[i]; gr[i] = gn[i]; }
        const float mean = mean_n, rstd = rstd_n;
        if (row + step < rows) fetch(row + step);
        float s[2] = {0.0f, 0.0f};   // sum of g, sum of g * xh
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (live && (i * TEAM + lane) * VEC < H)
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const float d = get<T, VEC>(gr[i], j), xh = (get<T, VEC>(xr[i], j) - mean) * rstd;
                    const float g = weight ? d * get<W, VEC>(w[i], j) : d;
                    s[0] += g;
                    s[1] = fmaf(g, xh, s[1]);
                    dw[i * VEC + j] = fmaf(d, xh, dw[i * VEC + j]);
                    db[i * VEC + j] += d;
                }
        }
        team_sum<TEAM, 2>(s, slots, turn);
        const float c0 = s[0] * inv_h, c1 = s[1] * inv_h;
        if (dx && live) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * TEAM + lane) * VEC;
                if (c < H) {
                    float o[VEC];
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        const float d = get<T, VEC>(gr[i], j), xh = (get<T, VEC>(xr[i], j) - mean) * rstd;
                        const float g = weight ? d * get<W, VEC>(w[i], j) : d;
                        o[j] = rstd * (g - c0 - xh * c1);
                    }
                    store_vec<T, VEC>(dx + row * lddx + c, o);
                }
            }
        }
    }
    if (!partial) return;
    moe::launch_dependents();
    float* pw = partial + static_cast<int64_t>(blockIdx.x) * 2 * H;
    if constexpr (TEAM <= 32) {
        // the block's teams add their columns in team order
        __shared__ float sum[2 * TEAM * EPT];
        for (int t = 0; t < kTeams; ++t) {
            if (team == t)
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        const int c = (i * TEAM + lane) * VEC + j;
                        sum[c] = (t ? sum[c] : 0.0f) + dw[i * VEC + j];
                        sum[TEAM * EPT + c] = (t ? sum[TEAM * EPT + c] : 0.0f) + db[i * VEC + j];
                    }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < H; c += 256) {
            pw[c] = sum[c];
            pw[H + c] = sum[TEAM * EPT + c];
        }
    } else {
        store_partial<VEC, TEAM, EPT>(pw, H, lane, dw, db);
    }
}

// 16384 x 7168 bf16 rows with fp32 weights: 0.127 ms, 5.6 TB/s of the three
// tensors (0.82 of the measured copy bandwidth); 0.215 ms with the loads in
// registers, and 0.162 ms with 1024 threads of 8 elements, whose sums over the
// row took as many instructions as the rest.
//
// The same for rows of 16-byte vectors, one block per row at a time, through a
// ring of `depth` rows of x and dy in shared memory.  A stage is read into
// registers before the row's barrier (in team_sum), so after that barrier
// thread 0 can fill it again.  At two bytes an element the arithmetic is as
// long as the memory traffic: it runs on pairs of elements, with xh and g held
// from the sums to dx.
constexpr int kMaxDepth = 8;
constexpr size_t kRingBytes = 208 * 1024;

template <typename T, typename W, int TEAM, int EPT, int BLOCKS>
__global__ void __launch_bounds__(TEAM, BLOCKS)
norm_backward_ring_kernel(const T* dy, int64_t lddy, const T* x, int64_t ldx, int rows, int H,
                          const W* __restrict__ weight, const float* __restrict__ mean_in,
                          const float* __restrict__ rstd_in, T* dx, int64_t lddx, float* __restrict__ partial,
                          int depth, int* err) {
    constexpr int VEC = Elem<T>::kVec, NV = EPT / VEC;
    constexpr bool kHold = EPT <= 16;   // xh and g stay in registers; else they are computed again
    extern __shared__ __align__(128) uint8_t ring[];   // depth x (x row, dy row)
    __shared__ uint64_t full[kMaxDepth];
    __shared__ float slots[64];
    __shared__ int abort_flag;
    const int tid = threadIdx.x;
    const uint32_t row_bytes = static_cast<uint32_t>(H) * sizeof(T);
    const float inv_h = 1.0f / static_cast<float>(H);
    int turn = 0;
    if (tid == 0) {
        abort_flag = 0;
        for (int d = 0; d < depth; ++d) moe::mbar_init(moe::smem_u32(&full[d]), 1);
        moe::fence_barrier_init();
    }
    __syncthreads();
    const auto fill = [&](int stage, int64_t row) {
        const uint32_t dst = moe::smem_u32(ring) + stage * 2 * row_bytes, b = moe::smem_u32(&full[stage]);
        moe::mbar_arrive_expect_tx(b, 2 * row_bytes);
        moe::bulk_load(dst, x + row * ldx, row_bytes, b);
        moe::bulk_load(dst + row_bytes, dy + row * lddy, row_bytes, b);
    };
    if (tid == 0)
        for (int d = 0; d < depth; ++d) {
            const int64_t row = blockIdx.x + static_cast<int64_t>(d) * gridDim.x;
            if (row < rows) fill(d, row);
        }
    Raw<W, VEC> w[NV];
    uint64_t dw[EPT / 2], db[EPT / 2];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TEAM + tid) * VEC;
        w[i] = c < H && weight ? load_raw<W, VEC>(weight + c) : ones<W, VEC>();
    }
#pragma unroll
    for (int i = 0; i < EPT / 2; ++i) dw[i] = db[i] = 0;
    int stage = 0;
    uint32_t phase = 0;
    // a row's mean and rstd are fetched a row ahead
    float mean_n = mean_in[blockIdx.x], rstd_n = rstd_in[blockIdx.x];
    const int step = gridDim.x;
    for (int row = blockIdx.x; row < rows; row += step) {
        const float rstd = rstd_n;
        const uint64_t neg_mean = pair(-mean_n, -mean_n), rstd2 = pair(rstd, rstd);
        if (rows - row > step) {
            mean_n = mean_in[row + step];
            rstd_n = rstd_in[row + step];
        }
        if (!moe::mbar_wait(moe::smem_u32(&full[stage]), phase, &abort_flag, 2000000000ull)) {
            abort_flag = 1;   // the rows that follow are not waited for as long
            moe::raise_device_error(err, MOE_DEVERR_TIMEOUT);
        }
        const T* xs = reinterpret_cast<const T*>(ring + static_cast<size_t>(stage) * 2 * row_bytes);
        const T* gs = xs + H;
        Raw<T, VEC> xr[NV], gr[NV];
        uint64_t xh[kHold ? EPT / 2 : 1], g[kHold ? EPT / 2 : 1];
        uint64_t s0 = 0, s1 = 0;   // sum of g, sum of g * xh
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TEAM + tid) * VEC;
            if (c < H) {
                xr[i] = load_raw<T, VEC>(xs + c);
                gr[i] = load_raw<T, VEC>(gs + c);
#pragma unroll
                for (int j = 0; j < VEC / 2; ++j) {
                    const int e = i * (VEC / 2) + j;
                    const uint64_t d = get2<T, VEC>(gr[i], j);
                    const uint64_t xe = mul2(add2(get2<T, VEC>(xr[i], j), neg_mean), rstd2);
                    const uint64_t ge = mul2(d, get2<W, VEC>(w[i], j));
                    s0 = add2(s0, ge);
                    s1 = fma2(ge, xe, s1);
                    dw[e] = fma2(d, xe, dw[e]);
                    db[e] = add2(db[e], d);
                    if (kHold) {
                        xh[kHold ? e : 0] = xe;
                        g[kHold ? e : 0] = ge;
                    }
                }
            }
        }
        float s[2], hi;
        split(s0, s[0], hi);
        s[0] += hi;
        split(s1, s[1], hi);
        s[1] += hi;
        block_sum2<TEAM>(s[0], s[1], slots, turn);
        if (tid == 0 && row + static_cast<int64_t>(depth) * step < rows)
            fill(stage, row + static_cast<int64_t>(depth) * step);
        if (++stage == depth) { stage = 0; phase ^= 1u; }
        if (dx) {
            const float c0 = -s[0] * inv_h, c1 = -s[1] * inv_h;
            T* dx_row = dx + static_cast<int64_t>(row) * lddx;
            const uint64_t c02 = pair(c0, c0), c12 = pair(c1, c1);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * TEAM + tid) * VEC;
                if (c < H) {
                    float o[VEC];
#pragma unroll
                    for (int j = 0; j < VEC / 2; ++j) {
                        const int e = kHold ? i * (VEC / 2) + j : 0;
                        const uint64_t d = get2<T, VEC>(gr[i], j);
                        const uint64_t xe = kHold ? xh[e] : mul2(add2(get2<T, VEC>(xr[i], j), neg_mean), rstd2);
                        const uint64_t ge = kHold ? g[e] : mul2(d, get2<W, VEC>(w[i], j));
                        split(mul2(fma2(xe, c12, add2(ge, c02)), rstd2), o[2 * j], o[2 * j + 1]);
                    }
                    store_vec<T, VEC>(dx_row + c, o);
                }
            }
        }
    }
    moe::launch_dependents();
    if (partial) {
        float a[EPT], b[EPT];
#pragma unroll
        for (int i = 0; i < EPT / 2; ++i) {
            split(dw[i], a[2 * i], a[2 * i + 1]);
            split(db[i], b[2 * i], b[2 * i + 1]);
        }
        store_partial<VEC, TEAM, EPT>(partial + static_cast<int64_t>(blockIdx.x) * 2 * H, H, tid, a, b);
    }
}

// Rows of more elements than a team holds: x and dy are read twice, and a
// block sums its dweight and dbias in its partial row itself.
template <typename T, typename W>
__global__ void __launch_bounds__(kWide)
norm_backward_wide_kernel(const T* dy, int64_t lddy, const T* x, int64_t ldx, int rows,
                          int H, const W* __restrict__ weight, const float* __restrict__ mean_in,
                          const float* __restrict__ rstd_in, T* dx, int64_t lddx, float* partial) {
    __shared__ float slots[128];
    int turn = 0;
    float* pw = partial ? partial + static_cast<int64_t>(blockIdx.x) * 2 * H : nullptr;
    bool first = true;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const float mean = mean_in[row], rstd = rstd_in[row];
        float s[2] = {0.0f, 0.0f};
        for (int c = threadIdx.x; c < H; c += kWide) {
            const float d = to_f32(dy[row * lddy + c]), xh = (to_f32(x[row * ldx + c]) - mean) * rstd;
            const float g = weight ? d * to_f32(weight[c]) : d;
            s[0] += g;
            s[1] = fmaf(g, xh, s[1]);
            if (pw) {   // the same thread's columns in every row
                pw[c] = fmaf(d, xh, first ? 0.0f : pw[c]);
                pw[H + c] = d + (first ? 0.0f : pw[H + c]);
            }
        }
        first = false;
        team_sum<kWide, 2>(s, slots, turn);
        const float c0 = s[0] / static_cast<float>(H), c1 = s[1] / static_cast<float>(H);
        if (dx)
            for (int c = threadIdx.x; c < H; c += kWide) {
                const float d = to_f32(dy[row * lddy + c]), xh = (to_f32(x[row * ldx + c]) - mean) * rstd;
                const float o = rstd * ((weight ? d * to_f32(weight[c]) : d) - c0 - xh * c1);
                store_vec<T, 1>(dx + row * lddx + c, &o);
            }
    }
}

// out[c] = sum of the blocks' partial rows, in order within each of 64
// interleaved shares, then over the shares in a fixed tree; 16 columns (whole
// sectors of a partial row) a block.  blockIdx.y: 0 dweight, 1 dbias.
constexpr int kShares = 64, kCols = 16;
template <typename W>
__global__ void __launch_bounds__(kCols * kShares)
norm_reduce_kernel(const float* partial, int blocks, int H, W* __restrict__ dweight, W* __restrict__ dbias) {
    __shared__ float share[kCols][kShares + 1];
    W* out = blockIdx.y == 0 ? dweight : dbias;
    moe::wait_for_primary();   // this grid may start while the blocks' last stores are under way
    if (!out) return;
    const int col = threadIdx.x % kCols, part = threadIdx.x / kCols;
    const int c = blockIdx.x * kCols + col;
    float s = 0.0f;
    if (c < H) {
        const float* p = partial + static_cast<int64_t>(blockIdx.y) * H + c;
#pragma unroll 4
        for (int b = part; b < blocks; b += kShares) s += p[static_cast<int64_t>(b) * 2 * H];
    }
    share[col][part] = s;
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp >= kCols) return;
    float v = share[warp][lane] + share[warp][lane + 32];   // warp i: column i of the block
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if (lane == 0 && blockIdx.x * kCols + warp < H) store_vec<W, 1>(out + blockIdx.x * kCols + warp, &v);
}

// Blocks of a launch, each of which writes a partial row: as many as the GPU
// holds, but (past one an SM) with at least four rows each.
int partial_rows(int rows, int H) {
    const int sm = moe::sm_count() > 0 ? moe::sm_count() : 152;
    const int per_sm = H <= 1024 ? 8 : H <= 2048 ? 4 : H <= 4096 ? 2 : 1;
    const int64_t most = static_cast<int64_t>(sm) * per_sm;
    int64_t n = rows / 4 > sm ? rows / 4 : sm;
    if (n > most) n = most;
    return static_cast<int>(n < rows ? n : rows);
}

struct Args {
    const void *dy, *x, *weight;
    int64_t lddy, ldx, lddx;
    int rows, H;
    const float *mean, *rstd;
    void* dx;
    float* partial;   // NULL: neither dweight nor dbias is wanted
    int* err;
    cudaStream_t stream;
};

template <typename T, typename W, int VEC, int TEAM, int EPT>
int launch(const Args& a) {   // the blocks launched, 0 on failure
    auto kern = norm_backward_kernel<T, W, VEC, TEAM, EPT>;
    constexpr int kThreads = TEAM <= 32 ? 256 : TEAM, kTeams = TEAM <= 32 ? 256 / TEAM : 1;
    static std::atomic<int> resident[moe::kMaxDevices];
    int grid = moe::resident_blocks(reinterpret_cast<const void*>(kern), kThreads, 0, resident);
    if (grid <= 0) return 0;
    const int room = partial_rows(a.rows, a.H), need = (a.rows - 1) / kTeams + 1;
    if (room < grid) grid = room;
    if (need < grid) grid = need;
    kern<<<grid, kThreads, 0, a.stream>>>(
        static_cast<const T*>(a.dy), a.lddy, static_cast<const T*>(a.x), a.ldx, a.rows, a.H,
        static_cast<const W*>(a.weight), a.mean, a.rstd, static_cast<T*>(a.dx), a.lddx, a.partial);
    return grid;
}

template <typename T, typename W, int TEAM, int EPT, int BLOCKS>
int launch_ring(const Args& a) {
    auto kern = norm_backward_ring_kernel<T, W, TEAM, EPT, BLOCKS>;
    constexpr size_t kBytes = kRingBytes / BLOCKS;
    static std::atomic<int> configured[moe::kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= moe::kMaxDevices) return 0;
    if (!configured[dev].load(std::memory_order_relaxed)) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kBytes)) != cudaSuccess) return 0;
        configured[dev].store(1, std::memory_order_relaxed);
    }
    const size_t stage = static_cast<size_t>(a.H) * sizeof(T) * 2;
    int depth = static_cast<int>(kBytes / stage);
    if (depth > kMaxDepth) depth = kMaxDepth;
    const int grid = partial_rows(a.rows, a.H);
    kern<<<grid, TEAM, depth * stage, a.stream>>>(
        static_cast<const T*>(a.dy), a.lddy, static_cast<const T*>(a.x), a.ldx, a.rows, a.H,
        static_cast<const W*>(a.weight), a.mean, a.rstd, static_cast<T*>(a.dx), a.lddx, a.partial, depth, a.err);
    return grid;
}

// Rows of vectors go through the ring from 257 elements on: 16 a thread, 512
// threads an SM.  Narrower ones, and rows that are no vectors, do not.
template <typename T, typename W>
int pick_ring(const Args& a) {
    if (a.H <= 64 * 16) return launch_ring<T, W, 64, 16, 8>(a);
    if (a.H <= 128 * 16) return launch_ring<T, W, 128, 16, 4>(a);
    if (a.H <= 256 * 16) return launch_ring<T, W, 256, 16, 2>(a);
    if (a.H <= 512 * 16) return launch_ring<T, W, 512, 16, 1>(a);
    return launch_ring<T, W, 512, 32, 1>(a);
}
template <typename T, typename W, int VEC>
int pick(const Args& a) {
    if (a.H <= 8 * 8) return launch<T, W, VEC, 8, 8>(a);
    if (a.H <= 32 * 8) return launch<T, W, VEC, 32, 8>(a);
    if constexpr (VEC == 1) {
        if (a.H <= 128 * 8) return launch<T, W, VEC, 128, 8>(a);
        if (a.H <= 256 * 8) return launch<T, W, VEC, 256, 8>(a);
        if (a.H <= 512 * 8) return launch<T, W, VEC, 512, 8>(a);
        if (a.H <= 512 * 16) return launch<T, W, VEC, 512, 16>(a);   // 4099 bf16: 0.29 ms, 0.38 as 1024 x 8
        return launch<T, W, VEC, 1024, 16>(a);                       // 12289 bf16: 0.6 ms, 1.2 as 512 x 32
    } else {
        return pick_ring<T, W>(a);
    }
}

template <typename T, typename W>
moe_status_t run(const Args& a, void* dweight, void* dbias) {
    int blocks;
    if (a.H > kTeamMax) {
        blocks = partial_rows(a.rows, a.H);
        norm_backward_wide_kernel<T, W><<<blocks, kWide, 0, a.stream>>>(
            static_cast<const T*>(a.dy), a.lddy, static_cast<const T*>(a.x), a.ldx, a.rows, a.H,
            static_cast<const W*>(a.weight), a.mean, a.rstd, static_cast<T*>(a.dx), a.lddx, a.partial);
    } else {
        constexpr int V = Elem<T>::kVec;
        const bool vec = a.H % V == 0 && a.ldx % V == 0 && a.lddy % V == 0 && a.lddx % V == 0 &&
                         moe::aligned16(a.x) && moe::aligned16(a.dy) && moe::aligned16(a.dx);
        blocks = vec ? pick<T, W, V>(a) : pick<T, W, 1>(a);
        if (blocks <= 0) return MOE_ERR_CUDA;
    }
    MOE_CHECK_LAUNCH();
    if (a.partial) {
        return moe::launch_after(norm_reduce_kernel<W>, dim3((a.H + kCols - 1) / kCols, 2), kCols * kShares, 0, a.stream,
                                 static_cast<const float*>(a.partial), blocks, a.H, static_cast<W*>(dweight),
                                 static_cast<W*>(dbias));
    }
    return MOE_OK;
}

}  // namespace

extern "C" size_t moe_layer_norm_backward_workspace_size(int rows, int H) {
    if (rows < 1 || H < 1) return 0;
    return static_cast<size_t>(partial_rows(rows, H)) * 2 * H * sizeof(float);
}

extern "C" moe_status_t moe_layer_norm_backward(moe_dtype_t dtype, const void* dy, int64_t lddy, const void* x,
                                                int64_t ldx, int rows, int H, moe_dtype_t w_dtype,
                                                const void* weight, const float* mean, const float* rstd, void* dx,
                                                int64_t lddx, void* dweight, void* dbias, void* ws,
                                                size_t ws_bytes, moe_stream_t stream) {
    MOE_CHECK_ARG(dy && x && mean && rstd && rows >= 1 && H >= 1 && lddy >= H && ldx >= H && (!dx || lddx >= H));
    MOE_CHECK_ARG((dtype == MOE_BF16 || dtype == MOE_F32) && (w_dtype == dtype || w_dtype == MOE_F32));
    MOE_CHECK_ARG(moe::aligned16(weight) && moe::aligned16(mean) && moe::aligned16(rstd));
    MOE_CHECK_ARG(moe::aligned16(dweight) && moe::aligned16(dbias));
    const unsigned e = dtype == MOE_BF16 ? 2 : 4;
    MOE_CHECK_ARG(moe::aligned_to(x, e) && moe::aligned_to(dy, e) && moe::aligned_to(dx, e));
    const bool sums = dweight || dbias;
    MOE_CHECK_ARG(sums || dx);
    if (sums) {
        if (!ws || ws_bytes < moe_layer_norm_backward_workspace_size(rows, H)) return MOE_ERR_WORKSPACE;
        MOE_CHECK_ARG(moe::aligned16(ws));
    }
    int* err = moe::device_error_word();
    if (!err) return MOE_ERR_CUDA;
    const Args a{dy, x, weight, lddy, ldx, dx ? lddx : 0, rows, H, mean, rstd, dx,
                 sums ? static_cast<float*>(ws) : nullptr, err, reinterpret_cast<cudaStream_t>(stream)};
    if (dtype == MOE_F32) return run<float, float>(a, dweight, dbias);
    if (w_dtype == MOE_F32) return run<__nv_bfloat16, float>(a, dweight, dbias);
    return run<__nv_bfloat16, __nv_bfloat16>(a, dweight, dbias);
}
