// The gated feed-forward block for a few rows (generating a token at a time):
// every weight of the experts that have rows is read once and meets up to 32
// rows, so the block is bound by HBM.  The grouped GEMM's tcgen05 tiles of 256
// weight rows leave CTA pairs idle when the experts' tiles do not fill them, and
// each pair's ring then has to fill from cold; fp32 FMAs on unpacked weights
// would take longer than the memory does (some 50 instructions for the 16 weights
// that two 16-byte loads bring).  Here a block takes 16 weight rows (8 features'
// gate and up rows, or 16 output features) and its eight warps split the
// contraction: a lane loads 16 bytes of rows l / 4 and l / 4 + 8 straight into
// registers, and two warp-level m16n8k16 MMAs multiply them with the same 16
// bytes of up to 8 rows of x (the order of the contraction's elements within 32
// is the lanes' own, the same for both operands).  The warps' partial sums are
// added in warp order.
//
// First product: [g | u] = W1[e] x, h = silu(g) u from the unrounded sums (and
// Y1 = [g | u] kept, if wanted).  Second product: y = W2[e] h.  The second
// kernel is launched programmatically and has its first weights under way when
// it waits for h.
//
// One token through 4 of 32 experts, H = I = 2880 (199 MB of weights): the time
// given at kFewRows in ffn.cu; with FMAs and the loads in registers 43.5 us, the
// weights by asynchronous copies 61 us, whole rows by bulk copies 66 us.
#include <climits>

#include "common.cuh"
#include "internal.h"

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = 16;    // weight rows of a block's unit
constexpr int kBatch = 6;    // 32-element steps whose loads are in flight together

struct Args {
    const uint4* x;          // [M_cap, nv]
    const uint4* W;          // GATED: [E, 2F, nv], else [E, F, nv]
    const int32_t* offsets;
    __nv_bfloat16* out;      // [M_cap, F]
    __nv_bfloat16* keep;     // GATED: [M_cap, 2F] or NULL
    int* err;
    int E, M_cap, nv, F;
};

// The experts that have rows, and the offsets.
struct Live {
    int off[257];
    short expert[256];
    int n;
};

__device__ __forceinline__ uint4 load_once(const uint4* p) {   // weights: read once, not kept in L1
    uint4 v;
    asm("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
        : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
        : "l"(__cvta_generic_to_global(p)));
    return v;
}

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// This warp's share of one unit: weight rows w0 and w1 (this lane's two) against
// NB groups of 8 rows of x from row p on, `rows` of which exist.  `wait`: the
// kernel that writes x may still run.
template <int NB, int R>
__device__ __forceinline__ void share(const Args& a, const uint4* w0, const uint4* w1, int lo, int hi, int p, int rows,
                                      bool wait, float4 (&sums)[R / 8][kWarps][32]) {
    const int lane = threadIdx.x & 31, n = lane >> 2;
    float d[NB][4];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) d[b][i] = 0.0f;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int v0 = lo + (lane & 3); v0 - (lane & 3) < hi; v0 += 4 * kBatch) {
        uint4 r0[kBatch], r1[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const bool in = v0 + 4 * i < hi;
            r0[i] = in ? load_once(w0 + v0 + 4 * i) : zero;
            r1[i] = in ? load_once(w1 + v0 + 4 * i) : zero;
        }
        if (wait) {
            moe::wait_for_primary();
            wait = false;
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                uint4 xv = zero;
                if (8 * b + n < rows && v0 + 4 * i < hi) xv = a.x[static_cast<int64_t>(p + 8 * b + n) * a.nv + v0 + 4 * i];
                mma(d[b], r0[i].x, r1[i].x, r0[i].y, r1[i].y, xv.x, xv.y);
                mma(d[b], r0[i].z, r1[i].z, r0[i].w, r1[i].w, xv.z, xv.w);
            }
        }
    }
    if (wait) moe::wait_for_primary();
#pragma unroll
    for (int b = 0; b < NB; ++b) sums[b][threadIdx.x >> 5][lane] = make_float4(d[b][0], d[b][1], d[b][2], d[b][3]);
}

// R: the most rows an expert can have, 16 or 32 (the kernel for 16 has registers
// and L1 to spare: 37.8 us for the token below that takes 41 with 32).
template <bool GATED, int R>
__global__ void __launch_bounds__(kThreads, 2)
few_rows_kernel(const Args a) {
    __shared__ Live L;
    __shared__ float4 red[2][R / 8][kWarps][32];   // turn, group of 8 rows, warp, lane
    __shared__ int bad;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (GATED) moe::launch_dependents();   // the second product may take its place beside this one
    if (threadIdx.x == 0) bad = 0;
    for (int i = threadIdx.x; i <= a.E; i += kThreads) L.off[i] = a.offsets[i];
    __syncthreads();
    if (threadIdx.x < a.E && L.off[threadIdx.x + 1] < L.off[threadIdx.x]) bad = 1;
    if (threadIdx.x == 0 && (L.off[0] != 0 || L.off[a.E] > a.M_cap)) bad = 1;
    if (warp == 0) {
        int n = 0;
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const int e = e0 + lane;
            const bool has = e < a.E && L.off[e + 1] > L.off[e];
            const unsigned m = __ballot_sync(0xffffffffu, has);
            if (has) L.expert[n + __popc(m & ((1u << lane) - 1))] = static_cast<short>(e);
            n += __popc(m);
        }
        if (lane == 0) L.n = n;
    }
    __syncthreads();
    if (bad) {
        if (blockIdx.x == 0 && threadIdx.x == 0) moe::raise_device_error(a.err, MOE_DEVERR_OFFSETS);
        return;
    }
    constexpr int kFeatures = GATED ? kRows / 2 : kRows;
    const int per = (a.F + kFeatures - 1) / kFeatures;   // units of an expert
    const int units = L.n * per;
    // this warp's vectors of every row: whole 128-byte lines
    const int slice = ((a.nv + 8 * kWarps - 1) / (8 * kWarps)) * 8;
    const int lo = min(a.nv, warp * slice), hi = min(a.nv, lo + slice);
    bool wait = !GATED;
    int turn = 0;
    for (int unit = blockIdx.x; unit < units; unit += gridDim.x, turn ^= 1) {
        const int e = L.expert[unit / per], f0 = (unit % per) * kFeatures;
        const int p = L.off[e], rows = L.off[e + 1] - p;
        // lane l's rows: features f0 + l / 4 (gate, up), or f0 + l / 4 and + 8; past the
        // last feature the last one again, whose sums are not stored
        const int g = lane >> 2;
        const int64_t first = static_cast<int64_t>(e) * (GATED ? 2 : 1) * a.F;
        const uint4* w0 = a.W + (first + min(f0 + g, a.F - 1)) * a.nv;
        const uint4* w1 = a.W + (GATED ? first + a.F + min(f0 + g, a.F - 1) : first + min(f0 + g + 8, a.F - 1)) * a.nv;
        if (rows <= 8) share<1, R>(a, w0, w1, lo, hi, p, rows, wait, red[turn]);
        else if (R == 16 || rows <= 16) share<2, R>(a, w0, w1, lo, hi, p, rows, wait, red[turn]);
        else share<R / 8, R>(a, w0, w1, lo, hi, p, rows, wait, red[turn]);
        wait = false;
        __syncthreads();
        // warp i finishes rows 8i to 8i + 7 while the others go on; this
        // buffer is written again two units on, behind the next unit's barrier
        if (8 * warp < rows) {
            float4 s = red[turn][warp][0][lane];
#pragma unroll
            for (int i = 1; i < kWarps; ++i) {
                const float4 v = red[turn][warp][i][lane];
                s.x += v.x;
                s.y += v.y;
                s.z += v.z;
                s.w += v.w;
            }
            const float top[2] = {s.x, s.y}, bottom[2] = {s.z, s.w};   // weight rows l / 4 and l / 4 + 8
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int row = 8 * warp + 2 * (lane & 3) + j;
                if (row >= rows) continue;
                const int64_t at = static_cast<int64_t>(p + row) * a.F + f0 + g;
                if (GATED) {
                    if (f0 + g >= a.F) continue;
                    a.out[at] = __float2bfloat16_rn(top[j] / (1.0f + expf(-top[j])) * bottom[j]);
                    if (a.keep) {
                        const int64_t k = static_cast<int64_t>(p + row) * 2 * a.F + f0 + g;
                        a.keep[k] = __float2bfloat16_rn(top[j]);
                        a.keep[k + a.F] = __float2bfloat16_rn(bottom[j]);
                    }
                } else {
                    if (f0 + g < a.F) a.out[at] = __float2bfloat16_rn(top[j]);
                    if (f0 + g + 8 < a.F) a.out[at + 8] = __float2bfloat16_rn(bottom[j]);
                }
            }
        }
    }
    if (wait) moe::wait_for_primary();
    // rows of no expert are zeros
    const int64_t tid = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    const int64_t all = static_cast<int64_t>(gridDim.x) * kThreads;
    const int64_t none = static_cast<int64_t>(L.off[a.E]) * a.F, end = static_cast<int64_t>(a.M_cap) * a.F;
    for (int64_t i = none + tid; i < end; i += all) a.out[i] = __float2bfloat16_rn(0.0f);
    if (GATED && a.keep)
        for (int64_t i = 2 * none + tid; i < 2 * end; i += all) a.keep[i] = __float2bfloat16_rn(0.0f);
}

template <int R>
moe_status_t launch(const Args& a1, const Args& a2, cudaStream_t s) {
    static std::atomic<int> resident[2][moe::kMaxDevices];
    const int g1 = moe::resident_blocks(reinterpret_cast<const void*>(few_rows_kernel<true, R>), kThreads, 0, resident[0]);
    const int g2 = moe::resident_blocks(reinterpret_cast<const void*>(few_rows_kernel<false, R>), kThreads, 0, resident[1]);
    if (g1 <= 0 || g2 <= 0) return MOE_ERR_CUDA;
    // As many blocks as give each the same number of units if every row has an
    // expert of its own: a last round that only some have leaves too few loads
    // in flight.
    const auto blocks = [&](int units_of_expert, int most) {
        const int64_t units = static_cast<int64_t>(units_of_expert) * (a1.M_cap < a1.E ? a1.M_cap : a1.E);
        const int64_t rounds = (units + most - 1) / most;
        return static_cast<int>((units + rounds - 1) / rounds);
    };
    few_rows_kernel<true, R><<<blocks((a1.F + 7) / 8, g1), kThreads, 0, s>>>(a1);
    MOE_CHECK_LAUNCH();
    return moe::launch_after(few_rows_kernel<false, R>, dim3(blocks((a2.F + 15) / 16, g2)), kThreads, 0, s, a2);
}

}  // namespace

moe_status_t moe::ffn_few_rows(const void* x, const void* W1, const void* W2, const int32_t* offsets, int E, int M_cap,
                               int H, int I, void* Y1, void* h, void* y, cudaStream_t s) {
    MOE_CHECK_ARG(M_cap <= 32);
    int* err = moe::device_error_word();
    if (!err) return MOE_ERR_CUDA;
    const Args a1{static_cast<const uint4*>(x), static_cast<const uint4*>(W1), offsets, static_cast<__nv_bfloat16*>(h),
                  static_cast<__nv_bfloat16*>(Y1), err, E, M_cap, H / 8, I};
    const Args a2{static_cast<const uint4*>(h), static_cast<const uint4*>(W2), offsets, static_cast<__nv_bfloat16*>(y),
                  nullptr, err, E, M_cap, I / 8, H};
    return M_cap <= 16 ? launch<16>(a1, a2, s) : launch<32>(a1, a2, s);
}
