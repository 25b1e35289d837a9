// Declarations shared between translation units of libmoe.so (not exported).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "moe.h"

namespace moe {

enum class After : int;   // what a kernel's start and end wait for (common.cuh)

// C[p, n] = sum_k A[p, k] B[e, n, k]: the grouped GEMM without epilogue, bf16,
// as one of several launches.
moe_status_t store_gemm(const void* A, const void* B, const int32_t* offsets, int E, int M_cap, int N, int K, void* C,
                        cudaStream_t stream, After after);

// Launches the bf16 grouped GEMM for the data gradient (grouped_gemm.cu):
//   dA[p, c] = sum_n dC[p, n] * B[e, n, c]   (rows p of expert e)
// with B [E, N, K] read in place (MN-major); rows p >= offsets[E] of dA are
// zeros.  dC bf16 [M_cap, N], dA bf16 [M_cap, K].
moe_status_t dgrad_gemm(const void* dC, const void* B, const int32_t* offsets, int E, int M_cap, int N, int K,
                        void* dA, cudaStream_t stream, After after);

// The data gradient of fc2 with the gradient of silu(gate) * up applied to it
// in the epilogue (grouped_gemm.cu): with dh[p] = dy[p] W2[e] in fp32 and
// Y1[p] = [g | u],  dY1[p] = [dg | du] and h[p] = silu(g) u, all bf16 (M_cap rows
// of 2I, 2I and I; dy M_cap rows of H, W2 [E, H, I]).  Rows p >= offsets[E] are
// neither read nor written.  The kernel also makes the tails (see wgrad_gemm)
// of dY1, h, x (M_cap rows of H; NULL: none) and dy, 64E rows of the same widths.
struct SwigluBack {
    const void* Y1;
    void *dY1, *h;
    const void* x;
    void *tail_dY1, *tail_h, *tail_x, *tail_dy;
};
moe_status_t swiglu_back_gemm(const void* dy, const void* W2, const int32_t* offsets, int E, int M_cap, int H, int I,
                              const SwigluBack& back, cudaStream_t stream);

// Launches the weight-gradient GEMM (wgrad.cu):
//   dB[e, n, c] = sum over expert e's rows p of dC[p, n] * A[p, c]
// with dC bf16 [M_cap, N] and A bf16 [M_cap, K] (rows ldc and lda elements apart) read
// in place in 64-row k-blocks from offsets[e].  An expert's last, partial
// k-block (r = cnt_e mod 64 rows) comes instead from rows [64e, 64e + r) of the
// tails, copies of those rows of dC and A (bf16 [64E, N] and [64E, K]) with zeros
// up to the next multiple of 16.  Tails NULL: a single expert of exactly M_cap
// rows, whose last k-block reads zeros from outside the tensor maps.  dB bf16
// [E, N, K]; an expert without rows gets zeros.  scale (one float on the
// device, or NULL) multiplies dB in fp32 before it is rounded.
moe_status_t wgrad_gemm(const void* dC, int ldc, const void* A, int lda, const void* tail_c, const void* tail_a,
                        const int32_t* offsets, int E, int M_cap, int N, int K, void* dB, cudaStream_t stream,
                        After after, const float* scale = nullptr);

// The data gradient of one expert of M rows, its contraction split over
// several launches and, within one, over `splits` ranges (grouped_gemm.cu): with
// C[p, c] = sum_n dC[p, n] B[n, c] over this launch's N rows of B, cut into
// ranges, the first launch sets sum [splits, M, K] fp32 to the ranges' products
// and the others add theirs; the caller adds the ranges up.  With one range
// the last launch stores dA[p, c] = row_scale[p] * (sum + C) as bf16 instead
// (sum may be NULL if it is also the first).  dgrad_sum_splits: the number of
// ranges that fills the GPU, for the longest N of the launches.
// dC bf16 [M, N], rows ldc elements apart; B bf16 [N, K]; offsets {0, M}.
int dgrad_sum_splits(int M, int N, int K);
moe_status_t dgrad_sum_gemm(const void* dC, int ldc, const void* B, const int32_t* offsets, int M, int N, int K,
                            float* sum, int splits, bool first, bool last, const float* row_scale, void* dA,
                            cudaStream_t stream, After after);

// A tensor map for tiles staged with the 128-byte swizzle, zeros outside
// (grouped_gemm.cu): bytes for FP8, else bf16; dims and box innermost first,
// strides in bytes from the second dimension on.  False on failure.
bool encode_tile_map(CUtensorMap* map, bool fp8, const void* base, int rank, const cuuint64_t* dims,
                     const cuuint64_t* strides_bytes, const cuuint32_t* box);

// Launches the bf16 gate_up GEMM with SwiGLU that also keeps its
// pre-activations (grouped_gemm.cu): Y1 = [gate | up] bf16 [M_cap, N] rounded
// from the fp32 accumulators, h bf16 [M_cap, N/2] computed from them unrounded;
// rows p >= offsets[E] of both are zeros.
moe_status_t swiglu_keep_gemm(const void* x, const void* W1, const int32_t* offsets, int E, int M_cap, int N, int K,
                              void* Y1, void* h, cudaStream_t stream);

// moe_ffn_forward for few rows (ffn_few.cu), arguments checked by the caller.
moe_status_t ffn_few_rows(const void* x, const void* W1, const void* W2, const int32_t* offsets, int E, int M_cap,
                          int H, int I, void* Y1, void* h, void* y, cudaStream_t stream);

// The weighted combine (data.cu); topk_w NULL: unit weights.
moe_status_t combine_rows(const void* Y2, const int32_t* topk_ids, const float* topk_w, const int32_t* row_pos,
                          int T, int k, int H, int E, void* out, cudaStream_t stream);

}  // namespace moe
