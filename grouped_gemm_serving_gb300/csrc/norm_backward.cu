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
#include <climits>

#include "norm.cuh"

namespace {

using namespace moe::norm;

template <typename T, typename W, int VEC, int TEAM, int EPT>
__global__ void __launch_bounds__(TEAM == 32 ? 256 : TEAM)
norm_backward_kernel(const T* dy, int64_t lddy, const T* x, int64_t ldx, int rows, int H,
                     const W* __restrict__ weight, const float* __restrict__ mean_in,
                     const float* __restrict__ rstd_in, T* dx, int64_t lddx,
                     float* __restrict__ partial) {
    constexpr int NV = EPT / VEC;
    constexpr int kTeams = TEAM == 32 ? 8 : 1;
    __shared__ float slots[TEAM == 32 ? 1 : 128];
    const int lane = TEAM == 32 ? threadIdx.x & 31 : threadIdx.x;
    const int team = TEAM == 32 ? threadIdx.x >> 5 : 0;
    const float inv_h = 1.0f / static_cast<float>(H);
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
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * kTeams + team; row < rows; row += gridDim.x * kTeams) {
        Raw<T, VEC> xr[NV], gr[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TEAM + lane) * VEC;
            if (c < H) {
                xr[i] = load_raw<T, VEC>(x + row * ldx + c);
                gr[i] = load_raw<T, VEC>(dy + row * lddy + c);
            }
        }
        const float mean = mean_in[row], rstd = rstd_in[row];
        float s[2] = {0.0f, 0.0f};   // sum of g, sum of g * xh
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if ((i * TEAM + lane) * VEC < H)
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
        if (dx) {
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
    float* pw = partial + static_cast<int64_t>(blockIdx.x) * 2 * H;
    if constexpr (TEAM == 32) {
        // the block's eight warps add their columns in warp order
        __shared__ float sum[2 * 32 * EPT];
        for (int t = 0; t < kTeams; ++t) {
            if (team == t)
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        const int c = (i * TEAM + lane) * VEC + j;
                        sum[c] = (t ? sum[c] : 0.0f) + dw[i * VEC + j];
                        sum[32 * EPT + c] = (t ? sum[32 * EPT + c] : 0.0f) + db[i * VEC + j];
                    }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < H; c += 256) {
            pw[c] = sum[c];
            pw[H + c] = sum[32 * EPT + c];
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TEAM + lane) * VEC;
            if (c < H)
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    pw[c + j] = dw[i * VEC + j];
                    pw[H + c + j] = db[i * VEC + j];
                }
        }
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

// out[c] = sum of the blocks' partial rows, block order within each of eight
// interleaved shares, then the shares in order.  blockIdx.y: 0 dweight, 1 dbias.
template <typename W>
__global__ void __launch_bounds__(256)
norm_reduce_kernel(const float* __restrict__ partial, int blocks, int H, W* __restrict__ dweight,
                   W* __restrict__ dbias) {
    __shared__ float share[8][32];
    W* out = blockIdx.y == 0 ? dweight : dbias;
    if (!out) return;
    const int lane = threadIdx.x & 31, part = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float s = 0.0f;
    if (c < H) {
        const float* p = partial + static_cast<int64_t>(blockIdx.y) * H + c;
#pragma unroll 8
        for (int b = part; b < blocks; b += 8) s += p[static_cast<int64_t>(b) * 2 * H];
    }
    share[part][lane] = s;
    __syncthreads();
    if (part == 0 && c < H) {
        float v = share[0][lane];
#pragma unroll
        for (int i = 1; i < 8; ++i) v += share[i][lane];
        store_vec<W, 1>(out + c, &v);
    }
}

// Blocks whose partial rows the workspace has room for.
int partial_rows(int rows, int H) {
    const int sm = moe::sm_count() > 0 ? moe::sm_count() : 152;
    const int64_t teams = H <= 1024 ? (static_cast<int64_t>(rows) + 7) / 8 : rows;
    const int64_t cap = static_cast<int64_t>(sm) * (H <= 1024 ? 4 : 2);
    return static_cast<int>(teams < cap ? teams : cap);
}

struct Args {
    const void *dy, *x, *weight;
    int64_t lddy, ldx, lddx;
    int rows, H;
    const float *mean, *rstd;
    void* dx;
    float* partial;   // NULL: neither dweight nor dbias is wanted
    cudaStream_t stream;
};

template <typename T, typename W, int VEC, int TEAM, int EPT>
int launch(const Args& a) {   // the blocks launched, 0 on failure
    auto kern = norm_backward_kernel<T, W, VEC, TEAM, EPT>;
    constexpr int kThreads = TEAM == 32 ? 256 : TEAM;
    static std::atomic<int> resident[moe::kMaxDevices];
    int grid = moe::resident_blocks(reinterpret_cast<const void*>(kern), kThreads, 0, resident);
    if (grid <= 0) return 0;
    const int room = partial_rows(a.rows, a.H);
    if (room < grid) grid = room;
    kern<<<grid, kThreads, 0, a.stream>>>(
        static_cast<const T*>(a.dy), a.lddy, static_cast<const T*>(a.x), a.ldx, a.rows, a.H,
        static_cast<const W*>(a.weight), a.mean, a.rstd, static_cast<T*>(a.dx), a.lddx, a.partial);
    return grid;
}

template <typename T, typename W, int VEC>
int pick(const Args& a) {
    if (a.H <= 32 * 8) return launch<T, W, VEC, 32, 8>(a);
    if (a.H <= 32 * 32) return launch<T, W, VEC, 32, 32>(a);
    if (a.H <= 128 * 16) return launch<T, W, VEC, 128, 16>(a);
    if (a.H <= 256 * 16) return launch<T, W, VEC, 256, 16>(a);
    if (a.H <= 512 * 16) return launch<T, W, VEC, 512, 16>(a);
    return launch<T, W, VEC, 512, 32>(a);
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
        norm_reduce_kernel<W><<<dim3((a.H + 31) / 32, 2), 256, 0, a.stream>>>(
            a.partial, blocks, a.H, static_cast<W*>(dweight), static_cast<W*>(dbias));
        MOE_CHECK_LAUNCH();
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
    const Args a{dy, x, weight, lddy, ldx, lddx, rows, H, mean, rstd, dx, sums ? static_cast<float*>(ws) : nullptr,
                 reinterpret_cast<cudaStream_t>(stream)};
    if (dtype == MOE_F32) return run<float, float>(a, dweight, dbias);
    if (w_dtype == MOE_F32) return run<__nv_bfloat16, float>(a, dweight, dbias);
    return run<__nv_bfloat16, __nv_bfloat16>(a, dweight, dbias);
}
