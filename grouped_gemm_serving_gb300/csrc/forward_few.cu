// moe_forward_few: the whole expert layer for a few tokens (generating a token at
// a time for each sequence of a batch) in one kernel up to 16 tokens, in two above.
//
// With e = ids[t, j] the picks of token t and w[t, j] their weights:
//   [g | u] = W1[e] x[t],   h = silu(g) u,   out[t] = sum_j w[t, j] W2[e] h.
// Every weight of an expert that some token picked is streamed once for each chunk of
// its rows, which bounds the layer: 2 operations a weight and token against 2 bytes
// (bf16) or 1 (e4m3).  A chunk holds up to 16 rows while rows of x are short, and what
// shared memory leaves where they are long: above 16 tokens 15 of H = 2880, 7 of 5760, 6
// of 7168 in bf16, and 11 of 4096, 5 of 7168 in FP8 (the longer of H and I counts).  With
// more rows an expert than that, weights come twice or more, from L2 where chunks take
// turns (below), and moe_forward gets faster: graphs, L2 flushed before each, us of it
// and of this, 64 tokens top-4 of 32 experts, I = 2048: bf16 H = 7168 456, 577; FP8 H =
// 4096 221, 224, H = 7168 317, 490; and with 32 tokens 447, 438; 233, 171; 327, 298.
//
// Routing: per expert the set of its tokens as a mask, whose bit counts are the
// offsets, the permutation and its inverse (row r of an expert is its r-th token in
// ascending order); from it the plan, a list of chunks, up to 8 or 16 rows of an
// expert each, the rows' tokens and the slots' rows.  Above 16 tokens a kernel of one
// block makes it; up to 16 every block of the main kernel makes it for itself, which
// saves that kernel and the 3 us from it to the cooperative one (a token of 32 bf16
// experts 43.0 us instead of 45.4, of 256 e4m3 ones 70.4 instead of 73.6; 11 tokens of
// 128 experts 84.4 instead of 86.2, in one state's picks).
//
// The main kernel, a cooperative launch of a block per SM, streams the weights of
// both products.  A unit is 16 weight rows (8 features' gate and up rows, or 16
// output features) against a chunk; the units lie in expert order and every block
// takes a run of them, first of the one product, then of the other.  A producer warp
// brings the weights 16 KB at a time (1 KB of each row) into a ring in shared memory
// by TMA, as eight tiles of 128 bytes by 16 rows, without regard to what the others
// do: when the first product ends the ring is full of the second's weights.  Sixteen
// warps multiply, a tile of every other stage each (m16n8k16 MMAs; the order of the
// contraction's elements within a step is the lanes' own, the same for both
// operands), with their columns of the chunk's rows of x in shared memory for as
// long as the chunk lasts.  Two more take turns at adding the sixteen partial sums in
// warp order and finishing a unit while the others go on to the next.  Between the
// products the grid synchronises, as each block needs rows of h from many.
//
// FP8 weights are converted to fp16 on the way, one instruction for two of them
// (exact), and meet x in fp16, scaled by a power of two; the partial sum of a tile's
// 128 columns is multiplied by their block's scale in fp32.  x and h are not
// quantised: it would save no weight bytes, and cost accuracy.
//
// h is rounded once, to the MMA's operand: to bf16, or from fp32 to the scaled fp16
// (8 and 11 significant bits).  The second product leaves fp32 rows y; the grid
// synchronises again, and each block sums its share of the tokens' rows, in slot
// order, and rounds once.  (Sums by whichever block brought the last of a column's
// units fell to those that were behind already: 292 us instead of 279 for 64 tokens
// of 32 experts, 109 instead of 99 for 11 of 128.)
#include <cooperative_groups.h>
#include <cuda_fp8.h>

#include <climits>
#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace {

constexpr int kTiles = 8;                       // of a stage
constexpr int kProduct = 2 * kTiles;            // warps that multiply
constexpr int kThreads = 32 * (kProduct + 3);   // two that finish units, and the producer
constexpr int kRows = 16;                       // weight rows of a unit
constexpr int kRowBytes = 128;                  // of a tile's row
constexpr int kTileBytes = kRows * kRowBytes;
constexpr int kStageBytes = kTiles * kTileBytes;
template <bool FP8>
constexpr int kTileColumns = kRowBytes / (FP8 ? 1 : 2);
template <bool FP8>
constexpr int kColumns = kTiles * kTileColumns<FP8>;   // of a stage
constexpr int kMaxStages = 12;
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr int kMaxT = 64;                       // tokens: the bits of a mask
constexpr int kMaxSlots = 1024;
constexpr int kMaxE = 256;
constexpr int kMaxK = 32768;                    // columns of a product: a row of x takes 2 bytes each of a block
constexpr int kRouteThreads = 1024;
constexpr int kLight = 16;                      // tokens up to which the main kernel routes
constexpr int kLightSlots = kLight * 32;

// How the tokens are laid out.
template <int SLOTS>
struct PlanOf {
    int chunks;
    int pad[3];
    int4 chunk[SLOTS];        // expert, first row, rows, first row's token
    float slot_w[SLOTS];
    short slot_row[SLOTS];    // -1: a sentinel
    uint8_t token[SLOTS];     // a row's token
};
using Plan = PlanOf<kMaxSlots>;       // the routing kernel's, in the workspace
using LightPlan = PlanOf<kLightSlots>;   // a block's own, in shared memory

struct Route {
    const float* logits;
    const float* bias;
    const uint8_t* mask;
    int32_t* ids;
    float* w;
    int T, E, k, renormalize;
    int chunk_rows;
    int* err;
};

// A token's k picks on one warp, moe_route_sort's bit for bit: the largest of
// row[e], e < E (logit and bias), ties to the lower id.  Lane j < k returns the id of
// the j-th and its weight in w; a NaN is never picked, and a pick that too many of
// them left unfilled is INT_MAX.  row is in shared memory and is overwritten.  Every
// lane keeps the best of its own experts; where one is taken all lanes look for the
// next among that lane's.  Small loops on purpose: all this runs once, and
// instructions that come from L2 for one use cost more than they do.
__device__ __forceinline__ int picks(float* row, int E, int k, int renormalize, float& w) {
    const int lane = threadIdx.x & 31;
    uint32_t best = 0;
    int id = INT_MAX;
#pragma unroll 1
    for (int e = lane; e < E; e += 32) {
        const uint32_t key = moe::order_key(row[e]);
        if (key > best) {
            best = key;
            id = e;
        }
    }
    const uint32_t first = __reduce_max_sync(0xffffffffu, best);
    const float top = first ? moe::key_value(first) : -INFINITY;
    float part = 0.0f;
    if (!renormalize)
#pragma unroll 1
        for (int e = lane; e < E; e += 32) part += expf(row[e] - top);
    int my_id = INT_MAX;
    float my_v = -INFINITY;
#pragma unroll 1
    for (int r = 0; r < k; ++r) {
        const uint32_t m = __reduce_max_sync(0xffffffffu, best);
        if (m == 0) break;
        const int e = __reduce_min_sync(0xffffffffu, best == m ? id : INT_MAX);
        if (lane == r) {
            my_v = moe::key_value(m);
            my_id = e;
        }
        if (lane == (e & 31)) row[e] = NAN;   // taken
        __syncwarp();
        const int other = (e & 31) + 32 * lane;
        const uint32_t key = other < E ? moe::order_key(row[other]) : 0u;
        const uint32_t next = __reduce_max_sync(0xffffffffu, key);
        const int at = __reduce_min_sync(0xffffffffu, key == next ? other : INT_MAX);
        if (lane == (e & 31)) {
            best = next;
            id = at;
        }
    }
    if (renormalize) part = lane < k ? expf(my_v - top) : 0.0f;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) part += __shfl_xor_sync(0xffffffffu, part, off);
    w = expf(my_v - top) / part;
    return my_id;
}

// A block's threads route all tokens, a warp each at a time: the experts' masks of
// tokens, the slots' ids and weights.  logits: T * E floats of shared memory.  `record`:
// write the picks and weights out, and report invalid ones.  Between two barriers of
// the block's own.
__device__ __forceinline__ void route(const Route& a, float* logits, uint32_t (*tokens)[2], short* slot_id, float* slot_w, bool record) {
    const int tid = threadIdx.x, threads = blockDim.x, lane = tid & 31, warp = tid >> 5;
#pragma unroll 1
    for (int i = tid; i < 2 * a.E; i += threads) (&tokens[0][0])[i] = 0;
    if (a.logits) {
#pragma unroll 4
        for (int i = tid; i < a.T * a.E; i += threads) {
            const float l = a.logits[i];
            logits[i] = a.bias ? l + a.bias[i % a.E] : l;
        }
    }
    __syncthreads();
    const auto take = [&](int t, int s, int id, bool changed) {
        if (a.mask && a.mask[s]) {
            changed |= id != a.E;
            id = a.E;
        }
        if (id < 0 || id > a.E) {
            if (record) moe::raise_device_error(a.err, MOE_DEVERR_ROUTE);
            changed = true;
            id = a.E;
        }
        if (record && changed && a.ids) a.ids[s] = id;
        slot_id[s] = static_cast<short>(id);
        if (id < a.E) atomicOr(&tokens[id][t >> 5], 1u << (t & 31));
    };
    if (a.logits) {
#pragma unroll 1
        for (int t = warp; t < a.T; t += threads / 32) {
            float w;
            const int id = picks(logits + t * a.E, a.E, a.k, a.renormalize, w);
            if (lane < a.k) {
                const int s = t * a.k + lane;
                slot_w[s] = w;
                if (record && a.w) a.w[s] = w;
                take(t, s, id, true);
            }
        }
    } else {
#pragma unroll 1
        for (int s = tid; s < a.T * a.k; s += threads) {
            slot_w[s] = a.w[s];
            take(s / a.k, s, a.ids[s], false);
        }
    }
}

__device__ __forceinline__ int rows_of(const uint32_t (*tokens)[2], int e) { return __popc(tokens[e][0]) + __popc(tokens[e][1]); }

// One warp lays out the experts one behind the other: base, and the plan's chunks and
// rows' tokens.
template <int SLOTS>
__device__ __forceinline__ void lay_out(const Route& a, const uint32_t (*tokens)[2], short* base, PlanOf<SLOTS>& plan) {
    const int lane = threadIdx.x & 31;
    int before = 0;   // rows (low half) and chunks (high half) of the experts so far
#pragma unroll 1
    for (int e0 = 0; e0 < a.E; e0 += 32) {
        const int e = e0 + lane, n = e < a.E ? rows_of(tokens, e) : 0;
        const int c = n > a.chunk_rows ? (n + a.chunk_rows - 1) / a.chunk_rows : (n > 0);
        int upto = n | c << 16;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int below = __shfl_up_sync(0xffffffffu, upto, off);
            if (lane >= off) upto += below;
        }
        const int all = __shfl_sync(0xffffffffu, upto, 31);
        if (n) {
            const int row = ((before + upto) & 0xFFFF) - n;
            int chunk = ((before + upto) >> 16) - c;
            base[e] = static_cast<short>(row);
            uint64_t left = tokens[e][0] | static_cast<uint64_t>(tokens[e][1]) << 32;
            int in_chunk = 0;
#pragma unroll 1
            for (int r = 0; r < n; ++r, left &= left - 1) {
                const int t = __ffsll(left) - 1;
                plan.token[row + r] = static_cast<uint8_t>(t);
                if (in_chunk == 0) plan.chunk[chunk++] = make_int4(e, row + r, min(a.chunk_rows, n - r), t);
                if (++in_chunk == a.chunk_rows) in_chunk = 0;
            }
        }
        before += all;
    }
    if (lane == 0) plan.chunks = before >> 16;
    __syncwarp();
}

// The row of slot s among its expert's, -1 for a sentinel.
__device__ __forceinline__ short row_of_slot(const Route& a, const uint32_t (*tokens)[2], const short* base, const short* slot_id, int s) {
    const int id = slot_id[s], t = s / a.k;
    if (id >= a.E) return -1;
    const uint32_t below = (1u << (t & 31)) - 1;
    return static_cast<short>(base[id] + (t < 32 ? __popc(tokens[id][0] & below) : __popc(tokens[id][0]) + __popc(tokens[id][1] & below)));
}

// Dynamic shared memory: the logits, with their biases.
__global__ void __launch_bounds__(kRouteThreads)
few_route_kernel(const Route a, Plan* plan) {
    extern __shared__ __align__(16) float logits[];
    __shared__ uint32_t tokens[kMaxE][2];
    __shared__ short base[kMaxE], slot_id[kMaxSlots];
    moe::wait_for_primary();   // what wrote the logits or ids
    moe::launch_dependents();
    route(a, logits, tokens, slot_id, plan->slot_w, true);
    __syncthreads();
    if (threadIdx.x < 32) lay_out(a, tokens, base, *plan);
    __syncthreads();
    for (int s = threadIdx.x; s < a.T * a.k; s += kRouteThreads) plan->slot_row[s] = row_of_slot(a, tokens, base, slot_id, s);
}

template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    if (F16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four e4m3 values as two pairs of fp16 (exact).
__device__ __forceinline__ void f16x2_of_e4m3x4(uint32_t four, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(four));
}

// FP8's scaling of x: the exponent that takes the largest magnitude (bits of a
// bf16) to [2^14, 2^15), within what a float's exponent holds; 0 for zero.  Beside
// infinities and NaN every finite value has to stay finite: their exponent is one past
// the largest finite one's, and takes that to [2^13, 2^14).
__device__ __forceinline__ int scale_exponent(int bits) { return bits == 0 ? 0 : min(141 - max(bits >> 7, 1), 126); }
__device__ __forceinline__ uint32_t scaled_f16x2(float lo, float hi, float f) {
    const __half2 h = __floats2half2_rn(lo * f, hi * f);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// The largest magnitude of 8 bf16, or of 4 fp32 cut to bf16, as bits.
__device__ __forceinline__ int largest_bf16(uint4 v) {
    const uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
    return static_cast<int>(max(m & 0xFFFFu, m >> 16));
}
__device__ __forceinline__ int largest_f32(uint4 v) {
    return static_cast<int>(max(max(v.x & 0x7FFFFFFFu, v.y & 0x7FFFFFFFu), max(v.z & 0x7FFFFFFFu, v.w & 0x7FFFFFFFu)) >> 16);
}

// The weights' tiles: `whole` copies kTiles of them at once, [tile][row][128 bytes] in
// shared memory; `rest` one tile of the columns that fill none, zeros behind them (a
// stage of its own: a copy of whole tiles writes zeros where a tile is missing).
struct Maps {
    CUtensorMap whole, rest;
};

// One of the two products, y = W x, for all experts.
struct Product {
    const void* x;            // [rows, K]: x [T, K], or h [T*k, K] (FP8: fp32)
    const float* scales;      // FP8: a scale per 128 x 128 block of W
    int K, F;                 // columns and features of W: [E, 2F, K] (first) or [E, F, K]
    int whole;                // columns in whole tiles
    int whole_steps, steps;   // stages of a unit: of those, and in all, an even number (the last may be empty)
};

struct Args {
    Product p[2];
    Route route;              // up to kLight tokens
    const Plan* plan;         // above
    void* h;                  // [T*k, F of the first]
    float* part;              // y [ceil(F / 16), T*k, 16], F of the second, then summed into
    __nv_bfloat16* out;       // [T, F of the second]
    int T, E, k;
    int xrows, stages;        // the most rows of a chunk; depth of the ring
    int* err;
};

// Named barriers between the warps that multiply and those that finish, two of
// each kind for the two buffers of partial sums, and one for the block's own plan.
constexpr int kFull = 1, kEmpty = 3, kLaidOut = 5, kBarThreads = 32 * (kProduct + 1);
__device__ __forceinline__ void bar_sync(int id) { asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(kBarThreads) : "memory"); }
__device__ __forceinline__ void bar_arrive(int id) { asm volatile("bar.arrive %0, %1;" ::"r"(id), "n"(kBarThreads) : "memory"); }

struct Ring {
    uint64_t full[kMaxStages], empty[kMaxStages];
    int abort_flag;
    int sent;   // stages, once the producer has given up
    int chunks;
};

// What the plan says, within bounds whatever it says, and the number of chunks read
// once for a block: calls that share a workspace by mistake get wrong results, not
// wrong addresses, nor warps that wait for more units than others have.
template <int SLOTS>
__device__ __forceinline__ int4 chunk_of(const Args& a, const PlanOf<SLOTS>& plan, int i) {   // expert, first row, rows, first row's token
    int4 c = plan.chunk[i];
    c.x = max(0, min(c.x, a.E - 1));
    c.z = max(1, min(c.z, a.xrows));
    c.y = max(0, min(c.y, a.T * a.k - c.z));
    c.w = max(0, min(c.w, a.T - 1));
    return c;
}

// A block's run of units, in order.  An expert's chunks follow one another, or TURNS:
// take turns, with as many features at a time as a block has units, so that neighbouring
// blocks stream the same weights at the same time for two of its chunks, and one finds
// them in L2: 64 tokens of 32 bf16 experts take 265 us instead of 283.  Not for FP8, whose
// registers are full (12 and 24 bytes a thread spill in its kernels with 16 rows a chunk; us
// without turns and with them, H = 7168, I = 2048: 64 tokens top-4 of 32 experts 459, 454;
// 64 top-8 of 256 1347, 1377; 32 top-8 of 256 901, 912), nor up to kLight tokens, where an
// expert has one chunk unless rows are very long (finding out cost a token 1 to 2.6 us).
template <bool FP8, typename P>
constexpr bool kTurns = !FP8 && std::is_same_v<P, Plan>;
template <bool FIRST, bool TURNS>
struct Run {
    static constexpr int kFeatures = FIRST ? kRows / 2 : kRows;
    int chunk, f, per, left;            // feature block f of `per`
    int chunks, turn, group, members;   // of the group, an expert's chunks; features of a turn
    int begin, end;                     // feature blocks of this turn
    Run() = default;
    template <typename P>
    __device__ __forceinline__ Run(int n, const P& plan, int F) : chunks(n) {
        per = (F + kFeatures - 1) / kFeatures;
        const int64_t units = static_cast<int64_t>(chunks) * per;
        const int64_t first = units * blockIdx.x / gridDim.x;
        left = static_cast<int>(units * (blockIdx.x + 1) / gridDim.x - first);
        chunk = static_cast<int>(first / per);
        f = static_cast<int>(first - static_cast<int64_t>(chunk) * per);
        if constexpr (!TURNS) return;
        group = chunk;
        turn = max(1, static_cast<int>((units + gridDim.x - 1) / gridDim.x));
        while (group > 0 && group < chunks && plan.chunk[group - 1].x == plan.chunk[group].x) --group;
        begin = 0;
        enter(plan);
        int at = static_cast<int>(first - static_cast<int64_t>(group) * per);   // in the group
        while (at >= members * (end - begin) && end < per) {
            at -= members * (end - begin);
            begin = end;
            end = min(per, end + turn);
        }
        chunk = min(group + at / (end - begin), chunks - 1);
        f = begin + at % (end - begin);
    }
    // the group's size, and its first turn's end
    template <typename P>
    __device__ __forceinline__ void enter(const P& plan) {
        members = 1;
        while (group + members < chunks && plan.chunk[group + members].x == plan.chunk[group].x) ++members;
        end = members > 1 ? min(per, turn) : per;
    }
    __device__ __forceinline__ int f0() const { return f * kFeatures; }
    template <typename P>
    __device__ __forceinline__ void next(const P& plan) {
        --left;
        if constexpr (!TURNS) {
            if (++f == per) {
                f = 0;
                ++chunk;
            }
            return;
        }
        if (++f < end) return;
        f = begin;
        if (++chunk < group + members) return;
        if (end < per) {
            chunk = group;
            f = begin = end;
            end = min(per, end + turn);
        } else if (left > 0) {
            group = chunk = min(chunk, chunks - 1);
            f = begin = 0;
            enter(plan);
        }
    }
};

// The producer's place in its unit and in the ring.  gave_up: whether a wait of its elected
// lane, the one that waits and sends, has run out.  The warp then goes on over its stages and
// sends nothing, so that its lanes stay together (a vote on every stage took 64 tokens of 32
// experts 275 us instead of 271, one on the flag too 299).
struct Filled {
    int step, slot;
    uint32_t turn;
    int stages;     // so far
    bool gave_up;
};

// Fills the stages of run u, up to stage number `until`.
template <bool FP8, bool FIRST, bool TURNS, typename P>
__device__ __forceinline__ void produce(const Maps& maps, const Product& p, const Args& a, const P& plan, Ring& S, uint32_t ring, Run<FIRST, TURNS>& u,
                                        Filled& at, int until) {
    int chunk = -1, e = 0;
    for (; u.left > 0; u.next(plan), at.step = 0) {
        if (u.chunk != chunk) {
            chunk = u.chunk;
            e = chunk_of(a, plan, chunk).x;
        }
        const int f0 = u.f0();
        for (; at.step < p.steps; ++at.step, ++at.stages) {
            if (at.stages == until) return;
            const int step = at.step;
            const uint32_t bar = moe::smem_u32(&S.full[at.slot]), dst = ring + at.slot * kStageBytes;
            if (moe::elect_one() && !at.gave_up) {
                if (at.stages >= a.stages && !moe::mbar_wait(moe::smem_u32(&S.empty[at.slot]), at.turn ^ 1u, &S.abort_flag, kWaitNs)) {
                    if (!S.abort_flag) moe::raise_device_error(a.err, MOE_DEVERR_TIMEOUT);
                    S.abort_flag = 1;
                    S.sent = at.stages;
                    at.gave_up = true;
                } else if (step < p.whole_steps) {   // tiles past the last one come as zeros
                    moe::mbar_arrive_expect_tx(bar, kStageBytes);
                    if (FIRST) moe::tma_load_5d(dst, &maps.whole, bar, 0, f0, 0, step * kTiles, e);
                    else moe::tma_load_4d(dst, &maps.whole, bar, 0, f0, step * kTiles, e);
                } else if (step > p.whole_steps || p.whole == p.K) {
                    moe::mbar_arrive(bar);
                } else {
                    moe::mbar_arrive_expect_tx(bar, kTileBytes);
                    if (FIRST) moe::tma_load_4d(dst, &maps.rest, bar, p.whole, f0, 0, e);
                    else moe::tma_load_3d(dst, &maps.rest, bar, p.whole, f0, e);
                }
            }
            __syncwarp();
            if (++at.slot == a.stages) {
                at.slot = 0;
                at.turn ^= 1u;
            }
        }
    }
}

// Shared memory behind the ring: two buffers of partial sums, and every product
// warp's columns of x.
template <int NB>
using Sums = float4[NB][kProduct][32];   // group of 8 rows, warp, lane

// Where a product warp is in the ring.  gives_back: its first lane, until a wait of it has run
// out.  From then on the warp reads slots that may have a copy under way, and as it gives none
// back none of its slots is filled again.
struct Place {
    int stage, slot;   // the stage's number, and its slot
    uint32_t phase;
    bool gives_back;
    __device__ __forceinline__ void go_to(int to, int stages) {
        slot += to - stage;
        stage = to;
        while (slot >= stages) {
            slot -= stages;
            phase ^= 1u;
        }
    }
};

// One product on one of its warps: tile `warp mod 8` of every other stage.  Units have
// an even number of stages and so has the ring, so that a slot is always the same
// warps' turn: a wait for a phase's parity tells only neighbouring phases apart, and
// would run ahead of phases that were others' to take.  `first`: the number of the
// product's first stage; `count`: units before, whose partial sums took the buffers
// in turn.
template <bool FP8, bool FIRST, int NBMAX, typename P>
__device__ __forceinline__ void multiply(const Product& p, const Args& a, const P& plan, Ring& S, const uint8_t* ring, Sums<NBMAX>* red, uint8_t* xcols,
                                         float (&unscale)[kProduct][8 * NBMAX], Place& place, int first, int& count) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tile = warp % kTiles, half = warp / kTiles;
    const int g = lane >> 2, c = lane & 3;
    constexpr int kXRow = FP8 ? 2 * kRowBytes : kRowBytes;   // of a tile's columns of a row of x
    constexpr int kVectors = kXRow / 16;
    constexpr bool kWide = FP8 && !FIRST;   // h in fp32
    const int mine = p.steps / 2;                             // this warp's steps of a unit
    uint8_t* const xs = xcols + static_cast<size_t>(warp) * mine * a.xrows * kXRow;
    // Tiles are swizzled: vector j of row r is at j ^ (r mod 8).  Lane l takes vectors
    // 2 (l mod 4) and the one after it of rows l / 4 and l / 4 + 8: the 8 lanes that are
    // served together find theirs in different banks.
    const int w_at = tile * kTileBytes + g * kRowBytes + ((2 * c) ^ g) * 16;
    const int blocks_k = p.K / 128;   // FP8: scales of a row, one a tile
    const int64_t blocks_n = ((FIRST ? 2 : 1) * static_cast<int64_t>(p.F) + 127) / 128;
    int held = -1, rows = 0, row0 = 0, token0 = 0, e = 0;
    int x_at[NBMAX];
    float s0 = 0.0f, s1 = 0.0f;
    // lane i's scales of this warp's step i (at most 16), for rows of the first and of the second 8
    const auto scales_of = [&](int f0) {
        const int k = (2 * lane + half) * kTiles + tile;
        if (k < blocks_k) {
            const float* row = p.scales + e * blocks_n * blocks_k + k;
            s0 = __ldg(row + static_cast<int64_t>(f0 / 128) * blocks_k);
            s1 = FIRST ? __ldg(row + static_cast<int64_t>((p.F + f0) / 128) * blocks_k) : s0;
        }
    };
    // This warp's columns of the chunk's rows of x: [step][row][half][8 vectors], swizzled
    // like the tiles; an FP8 vector of weights meets two of x, the halves.  FP8: scaled
    // by a power of two per row to at most 2^15 and held in fp16, which loses nothing of
    // a bf16 within 2^29 of the largest, and of the others less than 2^-39 of that; h, in
    // fp32, is rounded to its 11 bits.  Beside infinities and NaN, which decide every sum,
    // small values become zero.  A few rows, two vectors each, on their way at a time;
    // FP8 looks at them once for the scale and once to convert them.
    const auto take_x = [&]() {
        constexpr int NW = kWide ? 2 : 1, NR = NBMAX == 1 ? 2 : 4, NV = 2 / NW;
        const int vectors = mine * kVectors;
        __syncwarp();
#pragma unroll 1
        for (int r0 = 0; r0 < rows; r0 += NR) {
            const uint4* from[NR];
            int bits[NR];   // the largest magnitude's upper half, as a bf16
            float f[NR];
#pragma unroll
            for (int j = 0; j < NR; ++j) {
                const int r = min(r0 + j, rows - 1);
                const int row = FIRST ? (r ? min(static_cast<int>(plan.token[row0 + r]), a.T - 1) : token0) : row0 + r;
                from[j] = static_cast<const uint4*>(p.x) + static_cast<int64_t>(row) * (p.K / 8) * NW;
                bits[j] = 0;
            }
#pragma unroll 1
            for (int look = FP8 ? 0 : 1; look < 2; ++look) {
                if (FP8 && look == 1)
#pragma unroll
                    for (int j = 0; j < NR; ++j) {
                        const int x = scale_exponent(__reduce_max_sync(0xffffffffu, bits[j]));
                        f[j] = moe::exp2_int(x);
                        if (lane == 0 && r0 + j < rows) unscale[warp][r0 + j] = moe::exp2_int(-x);
                    }
#pragma unroll 1
                for (int i0 = lane; i0 < vectors; i0 += 32 * NV) {
                    uint4 v[NR][NV][NW];
#pragma unroll
                    for (int i = 0; i < NV; ++i) {
                        const int at = i0 + 32 * i, step = 2 * (at / kVectors) + half;
                        const int k = (step < p.whole_steps ? step * kColumns<FP8> : p.whole) + tile * kTileColumns<FP8> + 8 * (at % kVectors);
                        const bool in = at < vectors && k < (step < p.whole_steps ? p.whole : p.K);
#pragma unroll
                        for (int j = 0; j < NR; ++j)
#pragma unroll
                            for (int w = 0; w < NW; ++w) v[j][i][w] = in ? from[j][k / 8 * NW + w] : make_uint4(0, 0, 0, 0);
                    }
#pragma unroll
                    for (int i = 0; i < NV; ++i) {
                        const int at = i0 + 32 * i, q = at % kVectors;
#pragma unroll
                        for (int j = 0; j < NR; ++j) {
                            const int r = r0 + j;
                            uint4 t = v[j][i][0];
                            if (look == 0) {
                                bits[j] = max(bits[j], kWide ? max(largest_f32(t), largest_f32(v[j][i][NW - 1])) : largest_bf16(t));
                            } else if (at < vectors && r < rows) {
                                if (kWide) {
                                    const uint4 u = v[j][i][NW - 1];
                                    t = make_uint4(scaled_f16x2(__uint_as_float(t.x), __uint_as_float(t.y), f[j]), scaled_f16x2(__uint_as_float(t.z), __uint_as_float(t.w), f[j]),
                                                   scaled_f16x2(__uint_as_float(u.x), __uint_as_float(u.y), f[j]), scaled_f16x2(__uint_as_float(u.z), __uint_as_float(u.w), f[j]));
                                } else if (FP8) {
                                    t = make_uint4(scaled_f16x2(moe::bf16_lo(t.x), moe::bf16_hi(t.x), f[j]), scaled_f16x2(moe::bf16_lo(t.y), moe::bf16_hi(t.y), f[j]),
                                                   scaled_f16x2(moe::bf16_lo(t.z), moe::bf16_hi(t.z), f[j]), scaled_f16x2(moe::bf16_lo(t.w), moe::bf16_hi(t.w), f[j]));
                                }
                                const int to = FP8 ? (q & 1) * kRowBytes + ((q / 2) ^ (r & 7)) * 16 : (q ^ (r & 7)) * 16;
                                *reinterpret_cast<uint4*>(xs + ((at / kVectors) * a.xrows + r) * kXRow + to) = t;
                            }
                        }
                    }
                }
            }
        }
        __syncwarp();
    };
    int stage = first;
    for (Run<FIRST, kTurns<FP8, P>> u(S.chunks, plan, p.F); u.left > 0; u.next(plan), stage += p.steps, ++count) {
        if (u.chunk != held) {
            held = u.chunk;
            const int4 chunk = chunk_of(a, plan, held);
            e = chunk.x;
            row0 = chunk.y;
            rows = chunk.z;
            token0 = chunk.w;
            if (FP8) scales_of(u.f0());
            take_x();
#pragma unroll
            for (int b = 0; b < NBMAX; ++b) {   // rows past the last one read the last: their sums are not used
                const int r = min(8 * b + g, rows - 1);
                x_at[b] = r * kXRow + ((2 * c) ^ (r & 7)) * 16;
            }
        } else if (FP8 && u.f0() % 128 == 0) {   // the next block of 128 weight rows
            scales_of(u.f0());
        }
        const auto unit = [&](auto nb) {
            constexpr int NB = decltype(nb)::value;
            float d[NB][4];
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) d[b][i] = 0.0f;
#pragma unroll 1
            for (int i = 0; i < mine; ++i) {
                const int step = 2 * i + half;
                place.go_to(stage + step, a.stages);
                if (!moe::mbar_wait(moe::smem_u32(&S.full[place.slot]), place.phase, &S.abort_flag, kWaitNs)) {
                    if (!S.abort_flag) moe::raise_device_error(a.err, MOE_DEVERR_TIMEOUT);
                    S.abort_flag = 1;   // what follows is not waited for as long
                    place.gives_back = false;
                }
                uint4 w[2][2];   // vector, row
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint8_t* at = ring + place.slot * kStageBytes + (w_at ^ 16 * j);
                    w[j][0] = *reinterpret_cast<const uint4*>(at);
                    w[j][1] = *reinterpret_cast<const uint4*>(at + 8 * kRowBytes);
                }
                __syncwarp();
                if (place.gives_back) moe::mbar_arrive(moe::smem_u32(&S.empty[place.slot]));
                if (step < p.whole_steps ? step * kColumns<FP8> + tile * kTileColumns<FP8> >= p.whole : step > p.whole_steps || tile > 0 || p.whole == p.K) continue;
                const uint8_t* x = xs + i * a.xrows * kXRow;
                float t[NB][4];
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int j = 0; j < 4; ++j) t[b][j] = 0.0f;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t top[4] = {w[j][0].x, w[j][0].y, w[j][0].z, w[j][0].w}, bottom[4] = {w[j][1].x, w[j][1].y, w[j][1].z, w[j][1].w};
#pragma unroll
                    for (int q = 0; q < (FP8 ? 2 : 1); ++q) {
                        uint4 v[NB];
#pragma unroll
                        for (int b = 0; b < NB; ++b) v[b] = *reinterpret_cast<const uint4*>(x + (x_at[b] ^ 16 * j) + q * kRowBytes);
#pragma unroll
                        for (int m = 0; m < 2; ++m) {
                            uint32_t a0, a1, a2, a3;
                            if (FP8) {
                                f16x2_of_e4m3x4(top[2 * q + m], a0, a2);
                                f16x2_of_e4m3x4(bottom[2 * q + m], a1, a3);
                            } else {
                                a0 = top[2 * m], a2 = top[2 * m + 1], a1 = bottom[2 * m], a3 = bottom[2 * m + 1];
                            }
#pragma unroll
                            for (int b = 0; b < NB; ++b) mma<FP8>(FP8 ? t[b] : d[b], a0, a1, a2, a3, m ? v[b].z : v[b].x, m ? v[b].w : v[b].y);
                        }
                    }
                }
                if (FP8) {
                    const float f0 = __shfl_sync(0xffffffffu, s0, i), f1 = __shfl_sync(0xffffffffu, s1, i);
#pragma unroll
                    for (int b = 0; b < NB; ++b)
#pragma unroll
                        for (int j = 0; j < 4; ++j) d[b][j] = fmaf(j < 2 ? f0 : f1, t[b][j], d[b][j]);
                }
            }
            const int turn = count & 1;
            if (count >= 2) bar_sync(kEmpty + turn);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const float f0 = FP8 ? unscale[warp][8 * b + 2 * c] : 1.0f, f1 = FP8 ? unscale[warp][8 * b + 2 * c + 1] : 1.0f;
                red[turn][b][warp][lane] = make_float4(d[b][0] * f0, d[b][1] * f1, d[b][2] * f0, d[b][3] * f1);
            }
            bar_arrive(kFull + turn);
        };
        if (NBMAX == 1 || rows <= 8) unit(std::integral_constant<int, 1>());
        else unit(std::integral_constant<int, NBMAX>());
    }
}

// This block's share of the tokens' sums: a thread takes 4 features of a token and
// adds its slots' rows in their order, four loads on their way at a time.
__device__ __forceinline__ void sum_rows(const Args& a, const float* slot_w, const short* slot_row) {
    const int F = a.p[1].F, per = F / 4;
    const int64_t rows_all = static_cast<int64_t>(a.T) * a.k, items = static_cast<int64_t>(a.T) * per;
    const int64_t begin = items * blockIdx.x / gridDim.x, end = items * (blockIdx.x + 1) / gridDim.x;
    for (int64_t i = begin + threadIdx.x; i < end; i += kThreads) {
        const int t = static_cast<int>(i / per), f = 4 * static_cast<int>(i - static_cast<int64_t>(t) * per);
        const float* y = a.part + f / kRows * rows_all * kRows + f % kRows;
        float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int j0 = 0; j0 < a.k; j0 += 4) {
            float4 v[4];
            float w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int s = t * a.k + j0 + j, row = j0 + j < a.k ? slot_row[s] : -1;
                v[j] = row >= 0 ? __ldcg(reinterpret_cast<const float4*>(y + row * kRows)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                w[j] = row >= 0 ? slot_w[s] : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                sum.x = fmaf(w[j], v[j].x, sum.x);
                sum.y = fmaf(w[j], v[j].y, sum.y);
                sum.z = fmaf(w[j], v[j].z, sum.z);
                sum.w = fmaf(w[j], v[j].w, sum.w);
            }
        }
        *reinterpret_cast<uint2*>(a.out + static_cast<int64_t>(t) * F + f) =
            make_uint2(moe::pack_bf16x2(sum.x, sum.y), moe::pack_bf16x2(sum.z, sum.w));
    }
}

// One product on one of the two finishing warps: every other unit.
template <bool FP8, bool FIRST, int NBMAX, typename P>
__device__ __forceinline__ void finish(const Product& p, const Args& a, int chunks, const P& plan, const Sums<NBMAX>* red, int& count) {
    const int lane = threadIdx.x & 31, g = lane >> 2, own = (threadIdx.x >> 5) - kProduct, rows_all = a.T * a.k;
    for (Run<FIRST, kTurns<FP8, P>> u(chunks, plan, p.F); u.left > 0; u.next(plan), ++count) {
        const int turn = count & 1, f0 = u.f0();
        if (turn != own) continue;
        const int4 chunk = chunk_of(a, plan, u.chunk);
        bar_sync(kFull + turn);
        for (int b = 0; 8 * b < chunk.z; ++b) {
            float4 s = red[turn][b][0][lane];
#pragma unroll
            for (int i = 1; i < kProduct; ++i) {
                const float4 v = red[turn][b][i][lane];
                s.x += v.x;
                s.y += v.y;
                s.z += v.z;
                s.w += v.w;
            }
            const float top[2] = {s.x, s.y}, bottom[2] = {s.z, s.w};   // weight rows l / 4 and l / 4 + 8
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int row = 8 * b + 2 * (lane & 3) + j;
                if (row >= chunk.z) continue;
                if (FIRST) {
                    const float h = top[j] / (1.0f + expf(-top[j])) * bottom[j];
                    const int64_t at = static_cast<int64_t>(chunk.y + row) * p.F + f0 + g;
                    if (f0 + g >= p.F) continue;
                    if (FP8) static_cast<float*>(a.h)[at] = h;
                    else static_cast<__nv_bfloat16*>(a.h)[at] = __float2bfloat16_rn(h);
                } else {
                    float* y = a.part + (static_cast<int64_t>(u.f) * rows_all + chunk.y + row) * kRows;
                    y[g] = top[j];
                    y[g + 8] = bottom[j];
                }
            }
        }
        bar_arrive(kEmpty + turn);
    }
}

// What every block keeps of the routing: all of it up to kLight tokens, else the slots'
// rows and weights.
template <bool ROUTES>
struct Kept {
    LightPlan plan;
    uint32_t tokens[kMaxE][2];
    short base[kMaxE], slot_id[kLightSlots];
};
template <>
struct Kept<false> {
    float slot_w[kMaxSlots];
    short slot_row[kMaxSlots];
};

// NBMAX: the most groups of 8 rows of a chunk (a.xrows <= 8 NBMAX).  ROUTES: up to
// kLight tokens.
template <bool FP8, int NBMAX, bool ROUTES>
__global__ void __launch_bounds__(kThreads, 1)
few_layer_kernel(const __grid_constant__ Maps m1, const __grid_constant__ Maps m2, const Args a) {
    extern __shared__ __align__(16) uint8_t smem[];
    uint8_t* ring = smem + (-moe::smem_u32(smem) & 1023u);   // swizzled tiles
    auto* red = reinterpret_cast<Sums<NBMAX>*>(ring + a.stages * kStageBytes);
    uint8_t* xcols = ring + a.stages * kStageBytes + 2 * sizeof(Sums<NBMAX>);
    __shared__ Ring S;
    __shared__ float unscale[kProduct][8 * NBMAX];   // FP8: of a warp's columns of a row of x
    __shared__ Kept<ROUTES> kept;
    constexpr bool kInTurns = !ROUTES && !FP8;
    __shared__ Filled parked;       // the producer's while the grid synchronises and behind
    __shared__ Run<false, kInTurns> parked_run;   // the products, out of the others' registers
    const auto grid = cooperative_groups::this_grid();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (warp == kProduct + 2 && lane == 0) {
        S.abort_flag = 0;
        S.sent = INT_MAX;
        for (int i = 0; i < a.stages; ++i) {
            moe::mbar_init(moe::smem_u32(&S.full[i]), 1);
            moe::mbar_init(moe::smem_u32(&S.empty[i]), kTiles);
        }
        moe::fence_barrier_init();
        moe::prefetch_tensormap(&m1.whole);
        moe::prefetch_tensormap(&m2.whole);
    }
    if constexpr (!ROUTES) {
        if (threadIdx.x == 0) S.chunks = max(0, min(a.plan->chunks, a.T * a.k));
    } else {
        route(a.route, reinterpret_cast<float*>(ring), kept.tokens, kept.slot_id, kept.plan.slot_w, blockIdx.x == 0);
        moe::fence_proxy_async();   // the ring's first copies follow the logits
    }
    __syncthreads();
    const auto& plan = [&]() -> const auto& {
        if constexpr (ROUTES) return kept.plan;
        else return *a.plan;
    }();
    if constexpr (ROUTES) {
        if (warp == kProduct + 2) {   // the weights wait for no more than this
            lay_out(a.route, kept.tokens, kept.base, kept.plan);
            if (lane == 0) S.chunks = kept.plan.chunks;
            __syncwarp();
            asm volatile("bar.arrive %0, %1;" ::"n"(kLaidOut), "n"(kThreads) : "memory");
        } else {
            asm volatile("bar.sync %0, %1;" ::"n"(kLaidOut), "n"(kThreads) : "memory");
        }
    }
    Place place{0, 0, 0, lane == 0};
    int count = 0;
#pragma unroll 1
    for (int part = 0; part < 2; ++part) {
        if (warp == kProduct + 2) {
            Filled at{0, 0, 0, 0, false};
            Run<false, kInTurns> second(S.chunks, plan, a.p[1].F);
            if (part == 0) {
                Run<true, kInTurns> u(S.chunks, plan, a.p[0].F);
                produce<FP8, true, kInTurns>(m1, a.p[0], a, plan, S, moe::smem_u32(ring), u, at, INT_MAX);
            } else {
                at = parked;
                second = parked_run;
            }
            // before the grid has synchronised, as much of the second product as the ring holds
            produce<FP8, false, kInTurns>(m2, a.p[1], a, plan, S, moe::smem_u32(ring), second, at, part == 0 ? at.stages + a.stages : INT_MAX);
            if (moe::elect_one()) {
                parked = at;
                if (part == 0) parked_run = second;
            }
        } else if (warp < kProduct) {
            if (part == 0) {
                multiply<FP8, true, NBMAX>(a.p[0], a, plan, S, ring, red, xcols, unscale, place, 0, count);
            } else {
                multiply<FP8, false, NBMAX>(a.p[1], a, plan, S, ring, red, xcols, unscale, place, count * a.p[0].steps, count);
                // the finishing warps arrive once for every unit: take the last two as well
                for (int i = max(0, count - 2); i < count; ++i) bar_sync(kEmpty + (i & 1));
            }
        } else if (part == 0) {
            const int own = warp - kProduct;
            for (int s = 32 * own + lane; s < a.T * a.k; s += 64) {
                if constexpr (ROUTES) {
                    kept.plan.slot_row[s] = row_of_slot(a.route, kept.tokens, kept.base, kept.slot_id, s);
                } else {
                    kept.slot_w[s] = plan.slot_w[s];
                    kept.slot_row[s] = static_cast<short>(min(static_cast<int>(plan.slot_row[s]), a.T * a.k - 1));
                }
            }
            finish<FP8, true, NBMAX>(a.p[0], a, S.chunks, plan, red, count);
        } else {
            finish<FP8, false, NBMAX>(a.p[1], a, S.chunks, plan, red, count);
        }
        // every row of h, and then of y, is written before any is read; every block comes
        // here, as its other waits have a limit
        grid.sync();
    }
    if (warp == kProduct + 2 && S.abort_flag) {   // whichever warp raised it: no copy may land after the block has ended
        int never = 0;
        const int sent = min(S.sent, parked.stages);
        for (int i = 0; i < a.stages && i < sent; ++i)
            moe::mbar_wait(moe::smem_u32(&S.full[i]), static_cast<uint32_t>((sent - 1 - i) / a.stages) & 1u, &never, kWaitNs / 16);
    }
    if constexpr (ROUTES) sum_rows(a, kept.plan.slot_w, kept.plan.slot_row);
    else sum_rows(a, kept.slot_w, kept.slot_row);
}

constexpr size_t kSmem = 227 * 1024, kLeastRing = 96 * 1024;

template <bool FP8>
Product product(const void* x, const float* scales, int K, int F) {
    Product p{x, scales, K, F, K / kTileColumns<FP8> * kTileColumns<FP8>, 0, 0};
    p.whole_steps = (p.whole + kColumns<FP8> - 1) / kColumns<FP8>;
    p.steps = (p.whole_steps + (p.whole < K) + 1) / 2 * 2;
    return p;
}

// Shared memory: as deep a ring as partial sums and rows of x leave, and no fewer
// than kLeastRing bytes: longer rows are taken fewer at a time.
template <bool FP8, int NBMAX, bool ROUTES>
size_t shape(int T, const Product (&p)[2], int& xrows, int& stages) {
    const size_t steps = p[0].steps > p[1].steps ? p[0].steps : p[1].steps;
    const size_t row = steps / 2 * kProduct * kRowBytes * (FP8 ? 2 : 1);   // of x, all warps
    const size_t fixed = sizeof(Ring) + kProduct * 8 * NBMAX * sizeof(float) + sizeof(Kept<ROUTES>) + 128 + 1024;
    const size_t sums = 2 * sizeof(Sums<NBMAX>), most = (kSmem - fixed - sums - kLeastRing) / row;
    xrows = T < 8 * NBMAX ? T : 8 * NBMAX;
    if (most < static_cast<size_t>(xrows)) xrows = static_cast<int>(most);
    const size_t n = (kSmem - fixed - sums - xrows * row) / kStageBytes;
    stages = static_cast<int>(n < kMaxStages ? n / 2 * 2 : kMaxStages);   // even, at least 4
    return 1024 + static_cast<size_t>(stages) * kStageBytes + sums + xrows * row;
}

// The kernel may take all of an SM's shared memory; remembered per device.
bool allow_smem(const void* kernel, std::atomic<int> (&cache)[moe::kMaxDevices]) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= moe::kMaxDevices) return false;
    if (cache[dev].load(std::memory_order_relaxed)) return true;
    cudaFuncAttributes at;
    if (cudaFuncGetAttributes(&at, kernel) != cudaSuccess ||
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem - at.sharedSizeBytes)) != cudaSuccess) {
        (void)cudaGetLastError();
        return false;
    }
    cache[dev].store(1, std::memory_order_relaxed);
    return true;
}

// 16 weight rows (gated: 8 gate rows and the same 8 up rows) by kTiles or one tile
// of 128 bytes.  One copy brings a stage: sixteen, one a row, took a producer 1.2 us
// of the 0.4 us that the memory takes for a stage, and eight, one a tile, 0.6 us.
// A matrix without whole tiles has no copies of them.
bool weight_maps(Maps* m, bool fp8, bool gated, const void* W, int E, int F, int K) {
    const cuuint64_t e = fp8 ? 1 : 2, k = K, f = F, n = E;
    const cuuint32_t columns = kRowBytes / (fp8 ? 1 : 2);
    const cuuint64_t tiles = K / columns;
    bool ok = true;
    if (gated) {
        const cuuint64_t dims[5] = {columns, f, 2, tiles, n}, strides[4] = {k * e, f * k * e, kRowBytes, 2 * f * k * e};
        const cuuint32_t box[5] = {columns, kRows / 2, 2, kTiles, 1};
        if (tiles) ok = moe::encode_tile_map(&m->whole, fp8, W, 5, dims, strides, box);
        const cuuint64_t rest_dims[4] = {k, f, 2, n}, rest_strides[3] = {k * e, f * k * e, 2 * f * k * e};
        const cuuint32_t rest_box[4] = {columns, kRows / 2, 2, 1};
        if (K % columns) ok = ok && moe::encode_tile_map(&m->rest, fp8, W, 4, rest_dims, rest_strides, rest_box);
    } else {
        const cuuint64_t dims[4] = {columns, f, tiles, n}, strides[3] = {k * e, kRowBytes, f * k * e};
        const cuuint32_t box[4] = {columns, kRows, kTiles, 1};
        if (tiles) ok = moe::encode_tile_map(&m->whole, fp8, W, 4, dims, strides, box);
        const cuuint64_t rest_dims[3] = {k, f, n}, rest_strides[2] = {k * e, f * k * e};
        const cuuint32_t rest_box[3] = {columns, kRows, 1};
        if (K % columns) ok = ok && moe::encode_tile_map(&m->rest, fp8, W, 3, rest_dims, rest_strides, rest_box);
    }
    if (!tiles) m->whole = m->rest;
    else if (K % columns == 0) m->rest = m->whole;
    return ok;
}

template <bool FP8, int NBMAX, bool ROUTES>
moe_status_t launch(const moe_forward_args* f, Route r, Plan* plan, Args a, const Maps& m1, const Maps& m2, cudaStream_t s) {
    static std::atomic<int> allowed[moe::kMaxDevices];
    const auto kernel = few_layer_kernel<FP8, NBMAX, ROUTES>;
    const int sms = moe::sm_count();
    if (sms <= 0 || !allow_smem(reinterpret_cast<const void*>(kernel), allowed)) return MOE_ERR_CUDA;
    const size_t smem = shape<FP8, NBMAX, ROUTES>(f->T, a.p, a.xrows, a.stages);
    r.chunk_rows = a.xrows;
    a.route = r;
    if (!ROUTES) {
        static std::atomic<int> route_allowed[moe::kMaxDevices];
        if (!allow_smem(reinterpret_cast<const void*>(few_route_kernel), route_allowed)) return MOE_ERR_CUDA;
        const size_t logits = f->logits ? static_cast<size_t>(f->T) * f->E * sizeof(float) : 0;
        const moe_status_t st = moe::launch_after(few_route_kernel, dim3(1), kRouteThreads, logits, s, r, plan);
        if (st != MOE_OK) return st;
    }
    // a block per SM, or per unit of the first product if every slot has an expert of its own
    const int64_t units = static_cast<int64_t>((a.p[0].F + kRows / 2 - 1) / (kRows / 2)) * (f->T * f->k < f->E ? f->T * f->k : f->E);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(units < sms ? units : sms));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;   // its blocks wait for one another
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, m1, m2, a) != cudaSuccess) {
        (void)cudaGetLastError();
        return MOE_ERR_CUDA;
    }
    return MOE_OK;
}

template <bool FP8>
moe_status_t run(const moe_forward_args* f, const Route& r, Plan* plan, Args a, cudaStream_t s) {
    a.p[0] = product<FP8>(f->x, f->W1_scales, f->H, f->I);
    a.p[1] = product<FP8>(a.h, f->W2_scales, f->I, f->H);
    Maps m1, m2;
    if (!weight_maps(&m1, FP8, true, f->W1, f->E, f->I, f->H) || !weight_maps(&m2, FP8, false, f->W2, f->E, f->H, f->I)) return MOE_ERR_CUDA;
    if (f->T <= 8) return launch<FP8, 1, true>(f, r, plan, a, m1, m2, s);
    return f->T <= kLight ? launch<FP8, 2, true>(f, r, plan, a, m1, m2, s) : launch<FP8, 2, false>(f, r, plan, a, m1, m2, s);
}

bool valid_sizes(const moe_forward_args* a) {
    if (a->T < 1 || a->E < 1 || a->E > kMaxE || a->k < 1 || a->k > a->E || a->k > 32) return false;
    if (a->H < 8 || a->H % 8 || a->I < 8 || a->I % 8) return false;
    if (a->dtype == MOE_FP8_E4M3_B128) return a->H % 128 == 0 && a->I % 128 == 0;
    return a->dtype == MOE_BF16;
}

// Not more tokens than a mask has bits, more slots or longer rows than a block keeps, nor what only moe_forward does.
bool supported(const moe_forward_args* a) {
    return a->T <= kMaxT && a->T * a->k <= kMaxSlots && a->H <= kMaxK && a->I <= kMaxK && a->flags == 0;
}

struct Layout {
    size_t plan, h, part, total;
};

Layout layout(const moe_forward_args* a) {
    Layout l{};
    size_t off = 0;
    const auto take = [&off](size_t bytes) {
        const size_t at = off;
        off += (bytes + 255) & ~static_cast<size_t>(255);
        return at;
    };
    const size_t rows = static_cast<size_t>(a->T) * a->k, columns = (a->H + kRows - 1) / kRows;
    l.plan = take(sizeof(Plan));
    l.h = take(rows * a->I * (a->dtype == MOE_FP8_E4M3_B128 ? 4 : 2));
    l.part = take(columns * rows * kRows * sizeof(float));
    l.total = off;
    return l;
}

}  // namespace

extern "C" size_t moe_forward_few_workspace_size(const moe_forward_args* a) {
    return a && valid_sizes(a) && supported(a) ? layout(a).total : 0;
}

extern "C" moe_status_t moe_forward_few(const moe_forward_args* a, void* ws, size_t ws_bytes, moe_stream_t stream) {
    MOE_CHECK_ARG(a && valid_sizes(a));
    const bool fp8 = a->dtype == MOE_FP8_E4M3_B128;
    MOE_CHECK_ARG(a->x && a->W1 && a->W2 && a->out && (!fp8 || (a->W1_scales && a->W2_scales)));
    MOE_CHECK_ARG(a->logits || (a->topk_ids && a->topk_w));
    MOE_CHECK_ARG(moe::aligned16(a->x) && moe::aligned16(a->W1) && moe::aligned16(a->W2) && moe::aligned16(a->out) &&
                  moe::aligned16(a->logits) && moe::aligned16(a->topk_ids) && moe::aligned16(a->topk_w) &&
                  (!a->logits || moe::aligned16(a->expert_bias)) &&
                  (!fp8 || (moe::aligned_to(a->W1_scales, 4) && moe::aligned_to(a->W2_scales, 4))));
    if (!supported(a)) return MOE_ERR_UNSUPPORTED;
    const Layout l = layout(a);
    if (!ws || ws_bytes < l.total) return MOE_ERR_WORKSPACE;
    MOE_CHECK_ARG(moe::aligned16(ws));
    int* err = moe::device_error_word();
    if (!err) return MOE_ERR_CUDA;
    auto* base = static_cast<uint8_t*>(ws);
    auto* plan = reinterpret_cast<Plan*>(base + l.plan);
    const Route r{a->logits, a->expert_bias, a->sentinel_mask, a->topk_ids, a->topk_w, a->T, a->E, a->k, a->renormalize, 0, err};
    Args args{};
    args.plan = plan;
    args.h = base + l.h;
    args.part = reinterpret_cast<float*>(base + l.part);
    args.out = static_cast<__nv_bfloat16*>(a->out);
    args.T = a->T, args.E = a->E, args.k = a->k;
    args.err = err;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return fp8 ? run<true>(a, r, plan, args, s) : run<false>(a, r, plan, args, s);
}
