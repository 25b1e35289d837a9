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
// operations in all: bound by the tensor pipe.  The first one's epilogue applies
// the gradient of the activation to its fp32 accumulators and computes h again
// from Y1 (not kept from the forward pass); its idle warps copy the rows that
// the weight gradients need zero-padded.  dY1 = [dg | du] and h are rounded to bf16, the type
// of the GEMMs' operands: each rounding is at most a relative 2^-8, independent from
// element to element, and adds in a product's fp32 sum as noise of that size,
// no more than the rounding of the product itself.
#include <climits>

#include "common.cuh"
#include "internal.h"

namespace {

// Up to this many rows the forward pass streams the weights past all of an
// expert's rows at once (ffn_few.cu) instead of tiling them.  Measured, weights
// from HBM, streamed / tiled, us: 32 experts H = I = 2880, a row in each of 1, 4,
// 16 experts 16.4 / 37, 37.8 / 56, 124 / 138 (reading the weights takes 7.3, 29,
// 117), and 32 rows in 32 experts 257 / 256 (234); one expert, H = 2048, I = 5632,
// 1, 16 and 32 rows 21 / 43, 25 / 43, 33 / 43 (10).
constexpr int kFewRows = 32;

struct Layout {
    size_t dY1, h, tail_dY1, tail_h, tail_x, tail_dy, total;
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
    const size_t tails = static_cast<size_t>(64) * E;
    l.dY1 = take(rows * 2 * I * 2);
    l.h = take(rows * I * 2);
    l.tail_dY1 = take(tails * 2 * I * 2);
    l.tail_h = take(tails * I * 2);
    l.tail_x = take(tails * H * 2);
    l.tail_dy = take(tails * H * 2);
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
    if (M_cap <= kFewRows)
        return moe::ffn_few_rows(x, W1, W2, offsets, E, M_cap, H, I, Y1, h, y, reinterpret_cast<cudaStream_t>(stream));
    moe_status_t st;
    if (Y1)
        st = moe::swiglu_keep_gemm(x, W1, offsets, E, M_cap, 2 * I, H, Y1, h, reinterpret_cast<cudaStream_t>(stream));
    else
        st = moe_grouped_gemm(MOE_BF16, x, nullptr, W1, nullptr, offsets, E, M_cap, 2 * I, H, MOE_EPI_SWIGLU, h,
                              nullptr, stream);
    if (st != MOE_OK) return st;
    return moe::store_gemm(h, W2, offsets, E, M_cap, H, I, y, reinterpret_cast<cudaStream_t>(stream),
                           moe::After::kPrimary);
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
    void *dY1 = base + l.dY1, *h = base + l.h;
    const moe::SwigluBack back{Y1, dY1, h, dW1 ? x : nullptr, base + l.tail_dY1, base + l.tail_h, base + l.tail_x,
                               base + l.tail_dy};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    // Each GEMM sets up, and loads its first weights, while the one before it
    // drains; dW2's, which needs only the first one's output, also starts on the
    // SMs that dW1's frees (1037 rows of 6 experts, H = 1000, I = 1368: 85 -> 72
    // us; 4096 rows of 32 experts, H = I = 2880: 814 -> 799 us).  dW1's does not
    // start beside dx's: 817 us there, and 780 instead of 738 us with 1024 rows,
    // as its pairs then no longer run in step and share less of what they read.
    moe_status_t st = moe::swiglu_back_gemm(dy, W2, offsets, E, M_cap, H, I, back, s);
    if (st == MOE_OK && dx) st = moe::dgrad_gemm(dY1, W1, offsets, E, M_cap, 2 * I, H, dx, s, moe::After::kPrimary);
    if (st == MOE_OK && dW1)
        st = moe::wgrad_gemm(dY1, 2 * I, x, H, back.tail_dY1, back.tail_x, offsets, E, M_cap, 2 * I, H, dW1, s,
                             moe::After::kPrimary);
    if (st == MOE_OK && dW2)
        st = moe::wgrad_gemm(dy, H, h, I, back.tail_dy, back.tail_h, offsets, E, M_cap, H, I, dW2, s,
                             dx || dW1 ? moe::After::kBeside : moe::After::kPrimary);
    return st;
}
