// Gradients of the routing's data path, for training the layer: of the
// combine, of the permute and of the top-k softmax.  "Mixture of Experts in
// transformers" (MoE basics: the router's weights scale the experts' outputs,
// so it learns through them).
//
// combine   out[t] = sum_j w[t, j] Y2[p], p = row_pos[t*k + j]:
//             dY2[p] = w[t, j] dout[t],   dw[t, j] = <dout[t], Y2[p]>.
//           A team of threads takes a token (or some of its slots), holds a
//           piece of dout in registers and walks the slots with it, so dout
//           is read from HBM once however many slots there are; bound by HBM
//           (dout and Y2 read, dY2 written).
// permute   xp[p] = x[t]:  dx[t] = sum_j dxp[p], the combine with unit weights.
// softmax   a warp a token:
//             renormalised  dl[e_j] = p_j (dw_j - sum_i p_i dw_i), others 0
//             full          dl[e] = p_e ([e picked as j] dw_j - sum_i p_{e_i} dw_i).
//           With the caller's ids a live slot names its expert, and only a
//           masked slot's (it is no longer in the ids) is found again from the
//           logits; without them all picks are, in moe_route_sort's order.
#include <climits>

#include "common.cuh"
#include "internal.h"

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// TEAM threads per (token, group of up to KG slots).  blockIdx.y is the group.
template <int TEAM, int KG>
__global__ void __launch_bounds__(kThreads)
combine_backward_kernel(const uint4* __restrict__ dout, const uint4* __restrict__ Y2,
                        const int32_t* __restrict__ ids, const float* __restrict__ w,
                        const int32_t* __restrict__ row_pos, int T, int k, int row_vecs, int E,
                        uint4* __restrict__ dY2, float* __restrict__ dw, int* err) {
    __shared__ float part[TEAM == 32 ? 1 : kWarps][KG];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t = TEAM == 32 ? blockIdx.x * kWarps + warp : blockIdx.x;
    if (t >= T) return;   // whole warps, or whole blocks
    const int at = TEAM == 32 ? lane : threadIdx.x;
    const int64_t R = static_cast<int64_t>(T) * k;
    const int j0 = blockIdx.y * KG;
    // lane g holds slot j0 + g: its row (-1: none) and weight (0: a sentinel)
    int my_row = -1;
    float my_w = 0.0f;
    bool my_live = false;
    if (lane < KG && j0 + lane < k) {
        const int64_t f = static_cast<int64_t>(t) * k + j0 + lane;
        const int pos = row_pos[f];
        if (pos < 0 || pos >= R) {
            if (at < 32) moe::raise_device_error(err, MOE_DEVERR_ROUTE);
        } else {
            my_row = pos;
            my_live = ids[f] != E;
            if (my_live) my_w = w[f];
        }
    }
    int row[KG];
    float wj[KG], dot[KG];
    bool live[KG];
#pragma unroll
    for (int g = 0; g < KG; ++g) {
        row[g] = __shfl_sync(0xffffffffu, my_row, g);
        wj[g] = __shfl_sync(0xffffffffu, my_w, g);
        live[g] = __shfl_sync(0xffffffffu, static_cast<int>(my_live), g) != 0;
        dot[g] = 0.0f;
    }
    const uint4* src = dout + static_cast<int64_t>(t) * row_vecs;
    for (int c = at; c < row_vecs; c += TEAM) {
        const uint4 dv = __ldg(src + c);
        uint4 v[KG];
#pragma unroll
        for (int g = 0; g < KG; ++g)
            v[g] = live[g] ? __ldg(Y2 + static_cast<int64_t>(row[g]) * row_vecs + c) : make_uint4(0, 0, 0, 0);
        const uint32_t d4[4] = {dv.x, dv.y, dv.z, dv.w};
#pragma unroll
        for (int g = 0; g < KG; ++g) {
            if (row[g] < 0) continue;
            const uint32_t v4[4] = {v[g].x, v[g].y, v[g].z, v[g].w};
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float lo = moe::bf16_lo(d4[i]), hi = moe::bf16_hi(d4[i]);
                // a sentinel's row is zero whatever dout holds
                o[i] = live[g] ? moe::pack_bf16x2(wj[g] * lo, wj[g] * hi) : 0u;
                if (live[g]) {
                    dot[g] = fmaf(lo, moe::bf16_lo(v4[i]), dot[g]);
                    dot[g] = fmaf(hi, moe::bf16_hi(v4[i]), dot[g]);
                }
            }
            dY2[static_cast<int64_t>(row[g]) * row_vecs + c] = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
#pragma unroll
    for (int g = 0; g < KG; ++g)
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) dot[g] += __shfl_xor_sync(0xffffffffu, dot[g], off);
    if constexpr (TEAM > 32) {
        if (lane == 0)
#pragma unroll
            for (int g = 0; g < KG; ++g) part[warp][g] = dot[g];
        __syncthreads();
        if (warp != 0) return;
#pragma unroll
        for (int g = 0; g < KG; ++g) {
            dot[g] = 0.0f;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) dot[g] += part[i][g];
        }
    }
#pragma unroll
    for (int g = 0; g < KG; ++g)
        if (lane == g && j0 + g < k) dw[static_cast<int64_t>(t) * k + j0 + g] = dot[g];
}

template <int NV, bool IDS>   // logits per lane: E <= 32 * NV
__global__ void __launch_bounds__(kThreads)
route_backward_kernel(const float* __restrict__ logits, const float* __restrict__ bias,
                      const int32_t* __restrict__ ids, const float* __restrict__ dw, int T, int E, int k,
                      int renormalize, float* __restrict__ dlogits, int* err) {
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (t >= T) return;
    const float* row = logits + static_cast<int64_t>(t) * E;
    float v[NV], up[NV];   // up: the gradient of the weight that this logit was picked with
    uint32_t key[NV], picked = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int e = lane + 32 * j;
        v[j] = -INFINITY;
        up[j] = 0.0f;
        if (e < E) v[j] = bias ? row[e] + bias[e] : row[e];
        key[j] = e < E ? moe::order_key(v[j]) : 0u;
    }
    const float my_dw = lane < k ? dw[static_cast<int64_t>(t) * k + lane] : 0.0f;
    const auto pick = [&](int e, float g) {
        if ((e & 31) != lane) return;
        picked |= 1u << (e >> 5);
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (j == (e >> 5)) up[j] = g;
    };
    int open = k;   // picks that are still to be found
    if (IDS) {
        // an expert belongs to the first slot that names it; an id outside [0, E] and
        // a repeated one are reported and their slots taken as masked
        const int id = lane < k ? ids[static_cast<int64_t>(t) * k + lane] : E;
        const bool names = id >= 0 && id < E;
        const unsigned same = __match_any_sync(0xffffffffu, names ? id : -1 - lane);
        const bool live = names && __ffs(same) - 1 == lane;
        if (!live && id != E) moe::raise_device_error(err, MOE_DEVERR_ROUTE);
        for (unsigned left = __ballot_sync(0xffffffffu, live); left; left &= left - 1) {
            const int r = __ffs(left) - 1;
            pick(__shfl_sync(0xffffffffu, id, r), __shfl_sync(0xffffffffu, my_dw, r));
            --open;
        }
    }
    float top = -INFINITY;
    // the picks (with ids: the masked slots'), as moe_route_sort makes them: largest
    // key, then lowest id
    for (int r = 0; r < open; ++r) {
        uint32_t bk = 0u;
        int bj = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const uint32_t kj = (picked >> j) & 1u ? 0u : key[j];
            if (kj > bk) { bk = kj; bj = j; }
        }
        const uint32_t m = __reduce_max_sync(0xffffffffu, bk);
        if (m == 0u) break;   // fewer than k numbers among the logits: the same for the whole warp
        if (!IDS && r == 0) top = moe::key_value(m);
        pick(__reduce_min_sync(0xffffffffu, bk == m ? lane + 32 * bj : INT_MAX),
             IDS ? 0.0f : __shfl_sync(0xffffffffu, my_dw, r));
    }
    if (IDS) {   // the largest logit that the softmax runs over
        uint32_t bk = 0u;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (!renormalize || ((picked >> j) & 1u)) bk = max(bk, key[j]);
        const uint32_t m = __reduce_max_sync(0xffffffffu, bk);
        if (m != 0u) top = moe::key_value(m);
    }
    float sum = 0.0f, dot = 0.0f, p[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const bool in = renormalize ? (picked >> j) & 1u : lane + 32 * j < E;
        p[j] = in ? expf(v[j] - top) : 0.0f;
        sum += p[j];
        if ((picked >> j) & 1u) dot = fmaf(p[j], up[j], dot);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, off);
        dot += __shfl_xor_sync(0xffffffffu, dot, off);
    }
    dot /= sum;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int e = lane + 32 * j;
        const bool in = renormalize ? (picked >> j) & 1u : true;
        if (e < E) dlogits[static_cast<int64_t>(t) * E + e] = in ? p[j] / sum * (up[j] - dot) : 0.0f;
    }
}

template <bool IDS>
moe_status_t route_backward(const float* logits, const float* bias, const int32_t* ids, const float* dw, int T, int E,
                            int k, int renormalize, float* dlogits, cudaStream_t s) {
    MOE_CHECK_ARG(logits && dw && dlogits && T >= 1 && E >= 1 && E <= 256 && k >= 1 && k <= 32 && k <= E);
    MOE_CHECK_ARG(static_cast<int64_t>(T) * k < INT_MAX);
    MOE_CHECK_ARG(moe::aligned16(logits) && moe::aligned16(bias) && moe::aligned16(ids) && moe::aligned16(dw) &&
                  moe::aligned16(dlogits));
    int* err = IDS ? moe::device_error_word() : nullptr;
    if (IDS && !err) return MOE_ERR_CUDA;
    const int blocks = (T - 1) / kWarps + 1;
    auto kern = E <= 32 ? route_backward_kernel<1, IDS> : E <= 64 ? route_backward_kernel<2, IDS>
              : E <= 128 ? route_backward_kernel<4, IDS> : route_backward_kernel<8, IDS>;
    kern<<<blocks, kThreads, 0, s>>>(logits, bias, ids, dw, T, E, k, renormalize, dlogits, err);
    MOE_CHECK_LAUNCH();
    return MOE_OK;
}

}  // namespace

extern "C" moe_status_t moe_combine_backward(const void* dout, const void* Y2, const int32_t* topk_ids,
                                             const float* topk_w, const int32_t* row_pos, int T, int k, int H,
                                             int E, void* dY2, float* dtopk_w, moe_stream_t stream) {
    MOE_CHECK_ARG(dout && Y2 && topk_ids && topk_w && row_pos && dY2 && dtopk_w);
    MOE_CHECK_ARG(T >= 1 && k >= 1 && k <= 32 && E >= 1 && H >= 8 && H % 8 == 0);
    MOE_CHECK_ARG(static_cast<int64_t>(T) * k < INT_MAX);
    MOE_CHECK_ARG(moe::aligned16(dout) && moe::aligned16(Y2) && moe::aligned16(topk_ids) && moe::aligned16(topk_w) &&
                  moe::aligned16(row_pos) && moe::aligned16(dY2) && moe::aligned16(dtopk_w));
    int* err = moe::device_error_word();
    const int sm = moe::sm_count();
    if (!err || sm <= 0) return MOE_ERR_CUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const auto* d = static_cast<const uint4*>(dout);
    const auto* y = static_cast<const uint4*>(Y2);
    auto* o = static_cast<uint4*>(dY2);
    if (T >= sm * kWarps) {   // a warp a token fills the GPU
        const int blocks = (T - 1) / kWarps + 1;
        if (k <= 4)
            combine_backward_kernel<32, 4><<<blocks, kThreads, 0, s>>>(d, y, topk_ids, topk_w, row_pos, T, k, H / 8, E, o, dtopk_w, err);
        else
            combine_backward_kernel<32, 8><<<dim3(blocks, (k + 7) / 8), kThreads, 0, s>>>(d, y, topk_ids, topk_w, row_pos, T, k, H / 8, E, o, dtopk_w, err);
    } else {                  // few tokens: a block for each pair of slots
        combine_backward_kernel<kThreads, 2><<<dim3(T, (k + 1) / 2), kThreads, 0, s>>>(d, y, topk_ids, topk_w, row_pos, T, k, H / 8, E, o, dtopk_w, err);
    }
    MOE_CHECK_LAUNCH();
    return MOE_OK;
}

extern "C" moe_status_t moe_permute_backward(const void* dxp, const int32_t* topk_ids, const int32_t* row_pos, int T,
                                             int k, int H, int E, void* dx, moe_stream_t stream) {
    return moe::combine_rows(dxp, topk_ids, nullptr, row_pos, T, k, H, E, dx, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" moe_status_t moe_route_backward(const float* logits, const float* expert_bias, const float* dtopk_w, int T,
                                           int E, int k, int renormalize, float* dlogits, moe_stream_t stream) {
    return route_backward<false>(logits, expert_bias, nullptr, dtopk_w, T, E, k, renormalize, dlogits,
                                 reinterpret_cast<cudaStream_t>(stream));
}

extern "C" moe_status_t moe_route_backward_ids(const float* logits, const float* expert_bias, const int32_t* topk_ids,
                                               const float* dtopk_w, int T, int E, int k, int renormalize,
                                               float* dlogits, moe_stream_t stream) {
    MOE_CHECK_ARG(topk_ids);
    return route_backward<true>(logits, expert_bias, topk_ids, dtopk_w, T, E, k, renormalize, dlogits,
                                reinterpret_cast<cudaStream_t>(stream));
}
