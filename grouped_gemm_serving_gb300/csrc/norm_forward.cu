// moe_layer_norm_forward: y = (x - mean) * rstd * weight + bias per row.
//
// A row is read once and stays in registers while its mean and then the mean
// square of x - mean are summed (two passes over registers: no cancellation
// between large sums), so the kernel moves each element once in and once out
// and is bound by HBM.  Blocks are persistent: a thread keeps its columns'
// weights in registers over all its rows and has the next row's loads in
// flight while it sums the present one.
#include <climits>

#include "norm.cuh"

namespace {

using namespace moe::norm;

template <typename T, typename W, int VEC, int TEAM, int EPT>
__global__ void __launch_bounds__(TEAM <= 32 ? 256 : TEAM)
norm_forward_kernel(const T* x, int64_t ldx, int rows, int H, const W* __restrict__ weight,
                    const W* __restrict__ bias, float eps, T* y, int64_t ldy,
                    float* __restrict__ mean_out, float* __restrict__ rstd_out) {
    constexpr int NV = EPT / VEC;
    constexpr int kTeams = TEAM <= 32 ? 256 / TEAM : 1;   // rows in flight in a block
    __shared__ float slots[TEAM <= 32 ? 1 : 64];
    const int lane = threadIdx.x % TEAM, team = threadIdx.x / TEAM;
    const int step = gridDim.x * kTeams;
    const float inv_h = 1.0f / static_cast<float>(H);
    int turn = 0;
    Raw<W, VEC> w[NV], b[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TEAM + lane) * VEC;
        if (c < H && weight) w[i] = load_raw<W, VEC>(weight + c);
        if (c < H && bias) b[i] = load_raw<W, VEC>(bias + c);
    }
    Raw<T, VEC> cur[NV], next[NV];
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kTeams;   // the block's first row of a step
    if (row0 + team < rows) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TEAM + lane) * VEC;
            if (c < H) next[i] = load_raw<T, VEC>(x + (row0 + team) * ldx + c);
        }
    }
    // teams of a warp or less share its shuffles: the trip count is the block's
    for (int64_t at = row0; at < rows; at += step) {
        const int64_t row = at + team;
        const bool live = row < rows;
#pragma unroll
        for (int i = 0; i < NV; ++i) cur[i] = next[i];
        if (row + step < rows) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (i * TEAM + lane) * VEC;
                if (c < H) next[i] = load_raw<T, VEC>(x + (row + step) * ldx + c);
            }
        }
        float s[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (live && (i * TEAM + lane) * VEC < H)
#pragma unroll
                for (int j = 0; j < VEC; ++j) s[0] += get<T, VEC>(cur[i], j);
        team_sum<TEAM, 1>(s, slots, turn);
        const float mean = s[0] * inv_h;
        float q[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (live && (i * TEAM + lane) * VEC < H)
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const float d = get<T, VEC>(cur[i], j) - mean;
                    q[0] = fmaf(d, d, q[0]);
                }
        team_sum<TEAM, 1>(q, slots, turn);
        const float rstd = rsqrtf(fmaf(q[0], inv_h, eps));
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TEAM + lane) * VEC;
            if (live && c < H) {
                float o[VEC];
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const float n = (get<T, VEC>(cur[i], j) - mean) * rstd;
                    o[j] = fmaf(n, weight ? get<W, VEC>(w[i], j) : 1.0f, bias ? get<W, VEC>(b[i], j) : 0.0f);
                }
                store_vec<T, VEC>(y + row * ldy + c, o);
            }
        }
        if (live && lane == 0) {
            if (mean_out) mean_out[row] = mean;
            if (rstd_out) rstd_out[row] = rstd;
        }
    }
}

// Rows of more elements than a team holds: read three times (the second and
// third time from L2).
template <typename T, typename W>
__global__ void __launch_bounds__(kWide)
norm_forward_wide_kernel(const T* x, int64_t ldx, int rows, int H, const W* __restrict__ weight,
                         const W* __restrict__ bias, float eps, T* y, int64_t ldy,
                         float* __restrict__ mean_out, float* __restrict__ rstd_out) {
    __shared__ float slots[64];
    int turn = 0;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const T* xr = x + row * ldx;
        float s[1] = {0.0f};
        for (int c = threadIdx.x; c < H; c += kWide) s[0] += to_f32(xr[c]);
        team_sum<kWide, 1>(s, slots, turn);
        const float mean = s[0] / static_cast<float>(H);
        float q[1] = {0.0f};
        for (int c = threadIdx.x; c < H; c += kWide) {
            const float d = to_f32(xr[c]) - mean;
            q[0] = fmaf(d, d, q[0]);
        }
        team_sum<kWide, 1>(q, slots, turn);
        const float rstd = rsqrtf(q[0] / static_cast<float>(H) + eps);
        for (int c = threadIdx.x; c < H; c += kWide) {
            const float o = fmaf((to_f32(xr[c]) - mean) * rstd, weight ? to_f32(weight[c]) : 1.0f,
                                 bias ? to_f32(bias[c]) : 0.0f);
            store_vec<T, 1>(y + row * ldy + c, &o);
        }
        if (threadIdx.x == 0) {
            if (mean_out) mean_out[row] = mean;
            if (rstd_out) rstd_out[row] = rstd;
        }
    }
}

struct Args {
    const void *x, *weight, *bias;
    int64_t ldx, ldy;
    int rows, H;
    float eps;
    void* y;
    float *mean, *rstd;
    cudaStream_t stream;
};

template <typename T, typename W, int VEC, int TEAM, int EPT>
moe_status_t launch(const Args& a) {
    auto kern = norm_forward_kernel<T, W, VEC, TEAM, EPT>;
    constexpr int kThreads = TEAM <= 32 ? 256 : TEAM, kTeams = TEAM <= 32 ? 256 / TEAM : 1;
    static std::atomic<int> resident[moe::kMaxDevices];
    const int grid = moe::resident_blocks(reinterpret_cast<const void*>(kern), kThreads, 0, resident);
    if (grid <= 0) return MOE_ERR_CUDA;
    const int64_t want = (static_cast<int64_t>(a.rows) + kTeams - 1) / kTeams;
    kern<<<static_cast<int>(want < grid ? want : grid), kThreads, 0, a.stream>>>(
        static_cast<const T*>(a.x), a.ldx, a.rows, a.H, static_cast<const W*>(a.weight),
        static_cast<const W*>(a.bias), a.eps, static_cast<T*>(a.y), a.ldy, a.mean, a.rstd);
    MOE_CHECK_LAUNCH();
    return MOE_OK;
}

template <typename T, typename W, int VEC>
moe_status_t pick(const Args& a) {
    if (a.H <= 8 * 8) return launch<T, W, VEC, 8, 8>(a);
    if (a.H <= 32 * 8) return launch<T, W, VEC, 32, 8>(a);
    if (a.H <= 32 * 32) return launch<T, W, VEC, 32, 32>(a);
    if (a.H <= 128 * 16) return launch<T, W, VEC, 128, 16>(a);
    if (a.H <= 256 * 16) return launch<T, W, VEC, 256, 16>(a);
    if (a.H <= 512 * 16) return launch<T, W, VEC, 512, 16>(a);
    return launch<T, W, VEC, 1024, 16>(a);
}

template <typename T, typename W>
moe_status_t run(const Args& a) {
    if (a.H > kTeamMax) {
        const int sm = moe::sm_count();
        if (sm <= 0) return MOE_ERR_CUDA;
        norm_forward_wide_kernel<T, W><<<a.rows < 2 * sm ? a.rows : 2 * sm, kWide, 0, a.stream>>>(
            static_cast<const T*>(a.x), a.ldx, a.rows, a.H, static_cast<const W*>(a.weight),
            static_cast<const W*>(a.bias), a.eps, static_cast<T*>(a.y), a.ldy, a.mean, a.rstd);
        MOE_CHECK_LAUNCH();
        return MOE_OK;
    }
    constexpr int V = Elem<T>::kVec;
    const bool vec = a.H % V == 0 && a.ldx % V == 0 && a.ldy % V == 0 && moe::aligned16(a.x) && moe::aligned16(a.y);
    return vec ? pick<T, W, V>(a) : pick<T, W, 1>(a);
}

}  // namespace

extern "C" moe_status_t moe_layer_norm_forward(moe_dtype_t dtype, const void* x, int64_t ldx, int rows, int H,
                                               moe_dtype_t w_dtype, const void* weight, const void* bias,
                                               float eps, void* y, int64_t ldy, float* mean, float* rstd,
                                               moe_stream_t stream) {
    MOE_CHECK_ARG(x && y && rows >= 1 && H >= 1 && ldx >= H && ldy >= H && eps >= 0.0f);
    MOE_CHECK_ARG((dtype == MOE_BF16 || dtype == MOE_F32) && (w_dtype == dtype || w_dtype == MOE_F32));
    MOE_CHECK_ARG(moe::aligned16(weight) && moe::aligned16(bias) && moe::aligned16(mean) && moe::aligned16(rstd));
    MOE_CHECK_ARG(moe::aligned_to(x, dtype == MOE_BF16 ? 2 : 4) && moe::aligned_to(y, dtype == MOE_BF16 ? 2 : 4));
    const Args a{x, weight, bias, ldx, ldy, rows, H, eps, y, mean, rstd, reinterpret_cast<cudaStream_t>(stream)};
    if (dtype == MOE_F32) return run<float, float>(a);
    if (w_dtype == MOE_F32) return run<__nv_bfloat16, float>(a);
    return run<__nv_bfloat16, __nv_bfloat16>(a);
}
