// The gated feed-forward block of the experts, forward and backward (training
// of the MoE layer, "Mixture of Experts in transformers"; fc1 -> silu(gate) *
// up -> fc2 of "LlamaFactory Triton fused MoE kernel", section 1).  With E = 1
// it is a dense block, such as a shared expert.
//
// Forward, per row p of expert e:  [g | u] = W1[e] x,  h = silu(g) u,
// y = W2[e] h.  Two grouped GEMMs; the first one's epilogue applies silu and
// the product to the fp32 accumulators and, for training, stores the
// pre-activations Y1 = [g | u] beside h.
//
// Backward, with s = 1 / (1 + exp(-g)):
//   dh = W2[e]^T dy
//   du = dh g s,   dg = dh u s (1 + g (1 - s))
//   dx = W1[e]^T [dg | du],   dW1[e] = sum_p [dg | du] x^T,   dW2[e] = sum_p dy h^T
// Four grouped GEMMs (two data gradients, two weight gradients) of 12 P H I
// operations in all: bound by the tensor pipe.  h is computed again from Y1
// instead of being kept.  dY1 = [dg | du] and h are rounded to bf16, the type
// of the GEMMs' operands: each rounding is at most a relative 2^-8, independent from
// element to element, and adds in a product's fp32 sum as noise of that size,
// no more than the rounding of the product itself.
#include <climits>

#include "common.cuh"
#include "internal.h"

namespace {

constexpr int kThreads = 256;

// dY1 and h from dh and Y1, eight columns a thread; rows p >= offsets[E] are
// neither read nor written (the GEMMs that follow do not read them).
__global__ void __launch_bounds__(kThreads)
swiglu_backward_kernel(const uint4* __restrict__ dh, const uint4* __restrict__ Y1,
                       const int32_t* __restrict__ offsets, int E, int M_cap, int I, uint4* __restrict__ dY1,
                       uint4* __restrict__ h) {
    const int L = offsets[E];
    if (L < 0 || L > M_cap) return;   // reported by the GEMM before this kernel
    const int cv = I / 8;
    const int64_t n = static_cast<int64_t>(L) * cv;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < n;
         i += static_cast<int64_t>(gridDim.x) * kThreads) {
        const int64_t p = i / cv;
        const int64_t at = p * 2 * cv + (i - p * cv);
        const uint4 d = __ldg(dh + i), g = __ldg(Y1 + at), u = __ldg(Y1 + at + cv);
        const uint32_t d4[4] = {d.x, d.y, d.z, d.w}, g4[4] = {g.x, g.y, g.z, g.w}, u4[4] = {u.x, u.y, u.z, u.w};
        uint32_t dg4[4], du4[4], h4[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float dg[2], du[2], hh[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const float dv = q ? moe::bf16_hi(d4[j]) : moe::bf16_lo(d4[j]);
                const float gv = q ? moe::bf16_hi(g4[j]) : moe::bf16_lo(g4[j]);
                const float uv = q ? moe::bf16_hi(u4[j]) : moe::bf16_lo(u4[j]);
                moe::swiglu_grad(dv, gv, uv, dg[q], du[q], hh[q]);
            }
            dg4[j] = moe::pack_bf16x2(dg[0], dg[1]);
            du4[j] = moe::pack_bf16x2(du[0], du[1]);
            h4[j] = moe::pack_bf16x2(hh[0], hh[1]);
        }
        dY1[at] = make_uint4(dg4[0], dg4[1], dg4[2], dg4[3]);
        dY1[at + cv] = make_uint4(du4[0], du4[1], du4[2], du4[3]);
        h[i] = make_uint4(h4[0], h4[1], h4[2], h4[3]);
    }
}

struct Layout {
    size_t dh, dY1, h, tails, total;
};

Layout layout(int E, int M_cap, int H, int I) {
    Layout l{};
    size_t off = 0;
    auto take = [&off](size_t bytes) {
        const size_t at = off;
        off += (bytes + 255) & ~static_cast<size_t>(255);
        return at;
    };
    const size_t rows = static_cast<size_t>(M_cap);
    l.dh = take(rows * I * 2);
    l.dY1 = take(rows * 2 * I * 2);
    l.h = take(rows * I * 2);
    const size_t t1 = moe_grouped_gemm_wgrad_workspace_size(E, M_cap, 2 * I, H);
    const size_t t2 = moe_grouped_gemm_wgrad_workspace_size(E, M_cap, H, I);
    l.tails = take(t1 > t2 ? t1 : t2);
    l.total = off;
    return l;
}

bool valid_sizes(int E, int M_cap, int H, int I) {
    return E >= 1 && E <= 256 && M_cap >= 1 && H >= 8 && H % 8 == 0 && I >= 8 && I % 8 == 0 && I <= INT_MAX / 2;
}

}  // namespace

extern "C" moe_status_t moe_ffn_forward(const void* x, const void* W1, const void* W2, const int32_t* offsets, int E,
                                        int M_cap, int H, int I, void* Y1, void* h, void* y, moe_stream_t stream) {
    MOE_CHECK_ARG(x && W1 && W2 && offsets && h && y && valid_sizes(E, M_cap, H, I));
    MOE_CHECK_ARG(moe::aligned16(x) && moe::aligned16(W1) && moe::aligned16(W2) && moe::aligned16(Y1) &&
                  moe::aligned16(h) && moe::aligned16(y));
    moe_status_t st;
    if (Y1)
        st = moe::swiglu_keep_gemm(x, W1, offsets, E, M_cap, 2 * I, H, Y1, h, reinterpret_cast<cudaStream_t>(stream));
    else
        st = moe_grouped_gemm(MOE_BF16, x, nullptr, W1, nullptr, offsets, E, M_cap, 2 * I, H, MOE_EPI_SWIGLU, h,
                              nullptr, stream);
    if (st != MOE_OK) return st;
    return moe_grouped_gemm(MOE_BF16, h, nullptr, W2, nullptr, offsets, E, M_cap, H, I, MOE_EPI_STORE, y, nullptr,
                            stream);
}

extern "C" size_t moe_ffn_backward_workspace_size(int E, int M_cap, int H, int I) {
    return valid_sizes(E, M_cap, H, I) ? layout(E, M_cap, H, I).total : 0;
}

extern "C" moe_status_t moe_ffn_backward(const void* x, const void* W1, const void* W2, const void* Y1,
                                         const void* dy, const int32_t* offsets, int E, int M_cap, int H, int I,
                                         void* dx, void* dW1, void* dW2, void* ws, size_t ws_bytes,
                                         moe_stream_t stream) {
    MOE_CHECK_ARG(W1 && W2 && Y1 && dy && offsets && valid_sizes(E, M_cap, H, I));
    MOE_CHECK_ARG((dx || dW1 || dW2) && (x || !dW1));
    MOE_CHECK_ARG(moe::aligned16(x) && moe::aligned16(W1) && moe::aligned16(W2) && moe::aligned16(Y1) &&
                  moe::aligned16(dy) && moe::aligned16(dx) && moe::aligned16(dW1) && moe::aligned16(dW2));
    const Layout l = layout(E, M_cap, H, I);
    if (!ws || ws_bytes < l.total) return MOE_ERR_WORKSPACE;
    MOE_CHECK_ARG(moe::aligned16(ws));
    auto* base = static_cast<uint8_t*>(ws);
    void *dh = base + l.dh, *dY1 = base + l.dY1, *h = base + l.h, *tails = base + l.tails;
    const size_t tail_bytes = l.total - l.tails;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int sm = moe::sm_count();
    if (sm <= 0) return MOE_ERR_CUDA;
    moe_status_t st = moe::dgrad_gemm(dy, W2, offsets, E, M_cap, H, I, dh, s);
    if (st != MOE_OK) return st;
    const int64_t want = (static_cast<int64_t>(M_cap) * (I / 8) + kThreads - 1) / kThreads;
    swiglu_backward_kernel<<<static_cast<int>(want < sm * 8 ? want : sm * 8), kThreads, 0, s>>>(
        static_cast<const uint4*>(dh), static_cast<const uint4*>(Y1), offsets, E, M_cap, I,
        static_cast<uint4*>(dY1), static_cast<uint4*>(h));
    MOE_CHECK_LAUNCH();
    if (dx && (st = moe::dgrad_gemm(dY1, W1, offsets, E, M_cap, 2 * I, H, dx, s)) != MOE_OK) return st;
    if (dW1 && (st = moe_grouped_gemm_wgrad(x, dY1, offsets, E, M_cap, 2 * I, H, dW1, tails, tail_bytes, stream)) != MOE_OK) return st;
    if (dW2 && (st = moe_grouped_gemm_wgrad(h, dy, offsets, E, M_cap, H, I, dW2, tails, tail_bytes, stream)) != MOE_OK) return st;
    return MOE_OK;
}
