// What the layer-norm kernels share: element types, 16-byte vectors and sums
// over the threads of a row.
#pragma once

#include "common.cuh"

namespace moe {
namespace norm {

// A row of H elements is handled by a team of TEAM threads; thread i of it
// holds EPT elements in registers: vectors i, i + TEAM, ... of VEC elements.
// VEC is 16 bytes' worth where every row starts on a 16-byte boundary and H
// fills whole vectors, and 1 otherwise (any address and stride).
template <typename T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
    static constexpr int kVec = 8;
};
template <>
struct Elem<float> {
    static constexpr int kVec = 4;
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

// VEC consecutive elements at p, as they are stored.
template <typename T, int VEC>
struct Raw {
    static constexpr int kWords = VEC * sizeof(T) / 4;
    uint32_t w[kWords];
};
template <typename T>
struct Raw<T, 1> {
    T v;
};

template <typename T, int VEC>
__device__ __forceinline__ Raw<T, VEC> load_raw(const T* p) {
    Raw<T, VEC> r;
    if constexpr (VEC == 1) {
        r.v = *p;
    } else if constexpr (Raw<T, VEC>::kWords == 8) {   // eight fp32 weights beside eight bf16 elements
        const uint4 a = *reinterpret_cast<const uint4*>(p), b = *(reinterpret_cast<const uint4*>(p) + 1);
        r.w[0] = a.x; r.w[1] = a.y; r.w[2] = a.z; r.w[3] = a.w;
        r.w[4] = b.x; r.w[5] = b.y; r.w[6] = b.z; r.w[7] = b.w;
    } else {
        const uint4 a = *reinterpret_cast<const uint4*>(p);
        r.w[0] = a.x; r.w[1] = a.y; r.w[2] = a.z; r.w[3] = a.w;
    }
    return r;
}

template <typename T, int VEC>
__device__ __forceinline__ float get(const Raw<T, VEC>& r, int j) {
    if constexpr (VEC == 1) return to_f32(r.v);
    else if constexpr (sizeof(T) == 4) return __uint_as_float(r.w[j]);
    else return (j & 1) ? moe::bf16_hi(r.w[j / 2]) : moe::bf16_lo(r.w[j / 2]);
}

template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T* p, const float* v) {
    if constexpr (VEC == 1) {
        if constexpr (sizeof(T) == 4) *p = v[0];
        else *p = __float2bfloat16_rn(v[0]);
    } else if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
        *reinterpret_cast<uint4*>(p) = make_uint4(moe::pack_bf16x2(v[0], v[1]), moe::pack_bf16x2(v[2], v[3]),
                                                  moe::pack_bf16x2(v[4], v[5]), moe::pack_bf16x2(v[6], v[7]));
    }
}

// Pairs of fp32 values: one instruction works on both.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void split(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
// Elements 2j and 2j + 1 of a vector.
template <typename T, int VEC>
__device__ __forceinline__ uint64_t get2(const Raw<T, VEC>& r, int j) {
    return pair(get<T, VEC>(r, 2 * j), get<T, VEC>(r, 2 * j + 1));
}

// Sums of N values over a team, the same in every thread.  Teams of more than
// a warp are whole blocks: `slots` holds 2 x N x 32 floats, and calls alternate
// `turn` between its halves, so that one barrier a call is enough (a half is
// written again only after every thread has passed the next call's barrier).
template <int TEAM, int N>
__device__ __forceinline__ void team_sum(float (&v)[N], float* slots, int& turn) {
    constexpr int kLanes = TEAM < 32 ? TEAM : 32;
#pragma unroll
    for (int off = kLanes / 2; off > 0; off >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], off);
    if constexpr (TEAM > 32) {
        constexpr int kWarps = TEAM / 32;
        float* s = slots + turn * (N * 32);
        turn ^= 1;
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        if (lane == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) s[i * 32 + warp] = v[i];
        __syncthreads();
        // kWarps is a power of two: lanes repeat its values, so that the sum over
        // kWarps neighbouring lanes is everybody's
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = s[i * 32 + (lane & (kWarps - 1))];
#pragma unroll
        for (int off = kWarps / 2; off > 0; off >>= 1)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], off);
    }
}

// Both sums at once over a block of TEAM <= 512 threads, with half the
// shuffles: the warp's halves trade one value each and carry on with the other.
template <int TEAM>
__device__ __forceinline__ void block_sum2(float& v0, float& v1, float* slots, int& turn) {
    constexpr int kWarps = TEAM / 32;
    static_assert(kWarps <= 16, "one slot a lane");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float a = lane < 16 ? v0 : v1;
    a += __shfl_xor_sync(0xffffffffu, lane < 16 ? v1 : v0, 16);
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) a += __shfl_xor_sync(0xffffffffu, a, off);
    float* s = slots + turn * 32;
    turn ^= 1;
    if ((lane & 15) == 0) s[lane + warp] = a;   // v0's sums at 0.., v1's at 16..
    __syncthreads();
    a = s[(lane & 16) + (lane & (kWarps - 1))];
#pragma unroll
    for (int off = kWarps / 2; off > 0; off >>= 1) a += __shfl_xor_sync(0xffffffffu, a, off);
    v0 = __shfl_sync(0xffffffffu, a, 0);
    v1 = __shfl_sync(0xffffffffu, a, 16);
}

// A weight vector of ones, for calls without weights.
template <typename T, int VEC>
__device__ __forceinline__ Raw<T, VEC> ones() {
    static_assert(VEC > 1, "vectors");
    Raw<T, VEC> r;
#pragma unroll
    for (int i = 0; i < Raw<T, VEC>::kWords; ++i) r.w[i] = sizeof(T) == 4 ? 0x3F800000u : 0x3F803F80u;
    return r;
}

constexpr int kWide = 1024;        // threads of a row that no team holds in registers
constexpr int kTeamMax = 16384;    // elements of the widest row that a team holds

}  // namespace norm
}  // namespace moe
