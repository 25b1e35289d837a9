// A token's top-k picks and their softmax weights on one warp, for the router
// (route_sort.cu) and for the layer of a few tokens (forward_few.cu).
#pragma once

#include <climits>

#include "common.cuh"

namespace moe {

// The k largest of row[e] + bias[e] (bias may be NULL), e < E <= 32 * NV, ties to
// the lower id: lane j < k returns the id of the j-th pick and its weight in
// my_w.  A NaN is never picked; a pick that too many of them left unfilled
// returns INT_MAX.
template <int NV>   // logits per lane
__device__ __forceinline__ int top_picks(const float* __restrict__ row, const float* __restrict__ bias, int E, int k,
                                         int renormalize, float& my_w) {
    const int lane = threadIdx.x & 31;
    float v[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int e = lane + 32 * j;
        if (e < E) {
            const float l = row[e];
            v[j] = bias ? l + bias[e] : l;
        } else {
            v[j] = -INFINITY;
        }
    }
    // each pick: the largest key over the warp (one warp reduction), then
    // the lowest expert id holding it (a second one); a lane's candidate
    // is its first slot with its largest key, the lowest id of the lane
    uint32_t key[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) key[j] = lane + 32 * j < E ? order_key(v[j]) : 0u;
    uint32_t taken = 0;   // bit j: this lane's slot j was picked
    int my_id = E;
    float my_v = -INFINITY;
    for (int r = 0; r < k; ++r) {
        uint32_t bk = 0u;
        int bj = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const uint32_t kj = (taken >> j) & 1u ? 0u : key[j];
            if (kj > bk) { bk = kj; bj = j; }
        }
        const uint32_t m = __reduce_max_sync(0xffffffffu, bk);
        const int bi = __reduce_min_sync(0xffffffffu, m != 0u && bk == m ? lane + 32 * bj : INT_MAX);
        if (m != 0u && (bi & 31) == lane) taken |= 1u << (bi >> 5);
        if (lane == r) { my_v = m != 0u ? key_value(m) : -INFINITY; my_id = bi; }
    }
    const float mx = __shfl_sync(0xffffffffu, my_v, 0);  // pick 0 is the maximum
    float part = 0.0f;
    if (renormalize) {
        part = lane < k ? expf(my_v - mx) : 0.0f;
    } else {
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (lane + 32 * j < E) part += expf(v[j] - mx);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) part += __shfl_xor_sync(0xffffffffu, part, off);
    my_w = expf(my_v - mx) / part;
    return my_id;
}

}  // namespace moe
