// moe_sample: one token per row of logits, with temperature, top-k, top-p and min-p
// by row and a given uniform number.
//
// With L the row's largest logit and w_i = exp((l_i - L) / T), tokens in the order
// of (l descending, i ascending):
//   top-k   keeps the first k,
//   top-p   of these the shortest prefix whose weights are at least p of theirs all,
//   min-p   those with w_i >= min_p,
// and the draw takes the first token, in the order of the vocabulary, at which the
// kept weights' running sum exceeds u times their sum.
//
// The row is read once.  A cluster of blocks holds it in shared memory, a slice
// each, and goes over it there: for the largest logit; for a histogram of the
// logits' distance to it, of which only the bin where a cut falls is looked at
// closer (one block orders its tokens if they are few, else its range of values is
// divided again, down to tokens of one value, which are counted); and for the draw.
// With top-k up to 256, one block orders the few tokens that can be among the k, and
// does the rest with them alone.  No pass sorts the vocabulary.
//
// Bound by what a row's steps wait for one another, not by its bytes: 4.9 us would read
// 64 rows of 131072 fp32 logits, which top-p takes 78 to 84 us for.  Of a row's 24 to 45 us
// there, two rows to four SMs at a time, 2 go into loading it, 8 to 14 into the weights
// of all tokens and their histogram (40 and 20 issue cycles, about, for 32 tokens), the rest
// into eight rounds of the cluster and what one block does alone.  256 rows of bf16 with
// top-k: 61 us (9.9 to read), 9 to 10 a row; one row of 32000 with both: 6 us.
//
// A draw falls to another token wherever a running sum is off by more than u is from
// it.  Weights are integers, multiples of 2^-45 of the largest, whose sums are exact in
// any order (327680 of the largest fit 64 bits); each is rounded to the nearest, so it
// is off by at most 2^-46 and by 2^-35 of itself, and V of them by V 2^-46 at the very
// worst.  For logits that fall with the logarithm of a token's rank (60 rows of 131072,
// computed on the host) a draw takes another token than the definition's with
// probability 2^-21.5, 2^-17.2 in the worst row; with weights in fp32 2^-11.6 and 2^-9.7,
// cut to multiples of 2^-44 instead of rounded 2^-15.2 and 2^-13.4.
#include <cooperative_groups.h>

#include <algorithm>
#include <climits>

#include "common.cuh"

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kOctaves = 20;         // below the largest weight, which the first histogram divides
constexpr int kShare = kBins / kWarps;
constexpr int kSorted = 1024;        // tokens that one block sorts
constexpr int kCounted = kThreads;   // or whose places it counts
constexpr int kCountedFirst = 128;   // where dividing them is open too
constexpr int kMaxBlocks = 8;        // of a cluster: 8, 4, 2 or 1
constexpr int kGroups = kThreads;    // of lanes of the cluster: as many lanes each as it has blocks
constexpr int kFew = 256;            // the largest top-k whose tokens are looked for by the groups' largest
constexpr int kMaxV = 327680;        // 40960 tokens a block: 160 KB in fp32

struct Args {
    const void* logits;
    int64_t ld;
    int V, slice;                    // tokens of a block, a multiple of 8
    const float* temperature;
    const int32_t* top_k;
    const float* top_p;
    const float* min_p;
    const float* u;
    int32_t* token;
    float* logprob;
};

// 2^(j / 64) in units of 2^-62.
__constant__ uint64_t kPowers[64] = {
    0x4000000000000000ull, 0x40b268f9de0183baull, 0x4166c34c5615d0ecull, 0x421d1461d66f2023ull,
    0x42d561b3e6243d8aull, 0x438fb0cb4f468808ull, 0x444c0740496d4294ull, 0x450a6abaa4b77ecdull,
    0x45cae0f1f545eb73ull, 0x468d6fadbf2dd4f3ull, 0x47521cc5a2e6a9e0ull, 0x4818ee218a3358eeull,
    0x48e1e9b9d588e19bull, 0x49ad159789f37496ull, 0x4a7a77d47f7b84b1ull, 0x4b4a169b900c2d00ull,
    0x4c1bf828c6dc54b8ull, 0x4cf022c9905bfd32ull, 0x4dc69cdceaa72a9cull, 0x4e9f6cd3967fdba8ull,
    0x4f7a993048d088d7ull, 0x50582887dcb8a7e1ull, 0x513821818624b40cull, 0x521a8ad704f3404full,
    0x52ff6b54d8a89c75ull, 0x53e6c9da74b29ab5ull, 0x54d0ad5a753e077cull, 0x55bd1cdad49f699cull,
    0x56ac1f752150a563ull, 0x579dbc56b48521baull, 0x5891fac0e95612c8ull, 0x5988e20954889245ull,
    0x5a827999fcef3242ull, 0x5b7ec8f19468bbc9ull, 0x5c7dd7a3b17dcf75ull, 0x5d7fad59099f22feull,
    0x5e8451cfac061b5full, 0x5f8bccdb3d398841ull, 0x6096266533384a2bull, 0x61a3666d124bb204ull,
    0x62b39508aa836d6full, 0x63c6ba6455dcd8aeull, 0x64dcdec3371793d1ull, 0x65f60a7f79393e2eull,
    0x6712460a8fc24072ull, 0x683199ed779592caull, 0x69540ec8f895722dull, 0x6a79ad55e7f6fd10ull,
    0x6ba27e656b4eb57aull, 0x6cce8ae13c57ebdbull, 0x6dfddbcbed791babull, 0x6f307a412f074892ull,
    0x70666f76154a7089ull, 0x719fc4b95f452d29ull, 0x72dc8373be41a454ull, 0x741cb5281e25ee34ull,
    0x75606373ee921c97ull, 0x76a7980f6cca15c2ull, 0x77f25ccdee6d7ae6ull, 0x7940bb9e2cffd89dull,
    0x7a92be8a92436616ull, 0x7be86fb985689ddcull, 0x7d41d96db915019dull, 0x7e9f06067a4360baull,
};

// exp((l - L) / T) in units of 2^-kUnit, to the nearest, for l <= L.
constexpr int kUnit = 45;
struct Weight {
    float top;       // L
    float ch, cl;    // log2(e) / T in two parts
    const uint64_t* powers;

    // t = (l - L) c = m / 64 + r with |r| <= 1/128, and 2^t = 2^(m / 64) e^(r ln 2): a table
    // of 64 powers and four terms of the series (as in P. Tang's table-driven
    // exponentials).  t, r and the series' first term are kept in two floats each.
    // Without branches, 36 issue cycles for 32 tokens and some four for the last rounding.
    // A copy of the powers for every pair of banks and rounding by addition instead of
    // conversions took longer (37).
    __device__ __forceinline__ uint64_t operator()(float l) const {
        if (top == INFINITY) return l == top ? 1ull << kUnit : 0;   // the same for all
        const float d = l - top;
        const float p = d * ch;
        const float b = d - l, de = (l - (d - b)) + (-top - b);   // d + de = l - L
        const float pe = fmaf(d, ch, -p) + fmaf(d, cl, de * ch);
        const float big = 12582912.0f;   // 1.5 * 2^23
        const float shifted = fmaf(p, 64.0f, big);
        const int m = __float_as_int(shifted) - __float_as_int(big);
        const float rh = fmaf(shifted - big, -0.015625f, p);
        constexpr float kLn2 = 0.693147182f, kLn2Rest = -1.90465421e-9f;   // ln 2 in two floats
        const float y = rh * kLn2;
        const float ye = fmaf(rh, kLn2, -y) + fmaf(rh, kLn2Rest, pe * kLn2);
        const float rest = fmaf(y * y, fmaf(y, fmaf(y, 0.0416666679f, 0.166666672f), 0.5f), fmaf(ye, y, ye));
        // e^(r ln 2) - 1 in units of 2^-37
        const int e = __float2int_rn(y * 137438953472.0f) + __float_as_int(fmaf(rest, 137438953472.0f, big)) - __float_as_int(big);
        const uint64_t power = powers[m & 63];
        const uint64_t w = power + static_cast<uint64_t>((static_cast<int64_t>(e) * static_cast<int32_t>(power >> 32)) >> 5);
        // below half a unit, and for -infinity and the NaN of infinity times 0, nothing
        return p > -1.0f - kUnit ? ((w >> (61 - kUnit - (m >> 6))) + 1) >> 1 : 0;
    }
};

// floor(f * n), and the least integer not below f * n, for 0 < f < 1: exact.
__device__ __forceinline__ uint64_t share_below(float f, uint64_t n, bool& rest) {
    const uint32_t bits = __float_as_uint(f);
    const int e = max(static_cast<int>(bits >> 23), 1), shift = 150 - e;   // f = mantissa * 2^-shift, 24 <= shift <= 149
    const uint64_t mantissa = (bits & 0x7FFFFFu) | (bits >> 23 ? 0x800000u : 0u);
    const uint64_t lo = n * mantissa, hi = __umul64hi(n, mantissa);
    if (shift >= 128) {
        rest = true;
        return 0;
    }
    if (shift >= 64) {
        rest = lo != 0 || (shift > 64 && (hi & ((1ull << (shift - 64)) - 1)) != 0);
        return hi >> (shift - 64);
    }
    rest = (lo & ((1ull << shift) - 1)) != 0;
    return hi << (64 - shift) | lo >> shift;
}
__device__ __forceinline__ uint64_t share_reached(float f, uint64_t n) {
    if (!(f > 0.0f)) return 1;   // the first token is always kept
    bool rest;
    const uint64_t whole = share_below(f, n, rest);
    return max(whole + rest, static_cast<uint64_t>(1));
}

// A token's place in the order, larger first: its logit's key, then its index.
__device__ __forceinline__ uint64_t place_of(float l, int i) { return static_cast<uint64_t>(moe::order_key(l)) << 32 | static_cast<uint32_t>(~i); }

// Sixteen bytes of logits.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
    static constexpr int kSize = 4;
    uint4 v;
    __device__ __forceinline__ void unpack(float (&l)[4]) const {
        l[0] = __uint_as_float(v.x), l[1] = __uint_as_float(v.y), l[2] = __uint_as_float(v.z), l[3] = __uint_as_float(v.w);
    }
    __device__ __forceinline__ void clean() {   // NaN: never drawn
        v.x = __float_as_uint(fmaxf(__uint_as_float(v.x), -INFINITY));
        v.y = __float_as_uint(fmaxf(__uint_as_float(v.y), -INFINITY));
        v.z = __float_as_uint(fmaxf(__uint_as_float(v.z), -INFINITY));
        v.w = __float_as_uint(fmaxf(__uint_as_float(v.w), -INFINITY));
    }
    __device__ __forceinline__ float largest() const {
        return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
    }
    __device__ __forceinline__ void load(const float* from, int n) {   // the first n; -infinity behind them
        const uint32_t none = 0xFF800000u;
        v.x = n > 0 ? __float_as_uint(from[0]) : none;
        v.y = n > 1 ? __float_as_uint(from[1]) : none;
        v.z = n > 2 ? __float_as_uint(from[2]) : none;
        v.w = n > 3 ? __float_as_uint(from[3]) : none;
    }
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int kSize = 8;
    uint4 v;
    __device__ __forceinline__ void unpack(float (&l)[8]) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            l[2 * i] = moe::bf16_lo(w[i]);
            l[2 * i + 1] = moe::bf16_hi(w[i]);
        }
    }
    __device__ static __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
        const __nv_bfloat162 m = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
        return *reinterpret_cast<const uint32_t*>(&m);
    }
    __device__ __forceinline__ void clean() {
        const uint32_t none = 0xFF80FF80u;
        v = make_uint4(max2(v.x, none), max2(v.y, none), max2(v.z, none), max2(v.w, none));
    }
    __device__ __forceinline__ float largest() const {
        const uint32_t m = max2(max2(v.x, v.y), max2(v.z, v.w));
        return fmaxf(moe::bf16_lo(m), moe::bf16_hi(m));
    }
    __device__ __forceinline__ void load(const __nv_bfloat16* from, int n) {
        const auto* raw = reinterpret_cast<const uint16_t*>(from);
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = 2 * i < n ? raw[2 * i] : 0xFF80u, hi = 2 * i + 1 < n ? raw[2 * i + 1] : 0xFF80u;
            w[i] = lo | hi << 16;
        }
        v = make_uint4(w[0], w[1], w[2], w[3]);
    }
};

struct Shared {
    uint32_t lo[kBins], hi[kBins];   // histogram: weights, or ones, in two halves
    uint64_t list[kSorted];
    uint64_t powers[64];
    uint64_t warp[kWarps];
    uint64_t best[kMaxBlocks], total[kMaxBlocks];   // every block's, written by them
    uint64_t found[2];
    uint64_t share[kMaxBlocks][kWarps];               // every block's sums of kShare bins each, written by them
    uint32_t listed;
    uint32_t key[kGroups];                            // the groups' largest keys, this block's
    uint32_t group[kGroups];                          // every block's, written by them
    int kept;
    float ch, cl, far, far_rest;
};

// Sorts size (a power of two) places, larger first, by the whole block.
__device__ __noinline__ void sort_places(uint64_t* list, int size) {
#pragma unroll 1
    for (int block = 2; block <= size; block *= 2)   // bitonic
#pragma unroll 1
        for (int step = block / 2; step > 0; step /= 2) {
            for (int i = threadIdx.x; i < size / 2; i += kThreads) {
                const int x = 2 * i - (i & (step - 1)), y = x + step;
                const uint64_t p0 = list[x], p1 = list[y];
                if ((p0 < p1) == ((x & block) == 0)) {
                    list[x] = p1;
                    list[y] = p0;
                }
            }
            __syncthreads();
        }
}
__device__ __forceinline__ int padded(int n) { return n <= 32 ? 32 : 1 << (32 - __clz(n - 1)); }

// Running sums of two numbers a thread over the block: returns the sum up to and with
// b.  warps: kWarps words.
__device__ __noinline__ uint64_t running(uint64_t a, uint64_t b, uint64_t* warps) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint64_t sum = a + b;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint64_t o = __shfl_up_sync(0xffffffffu, sum, off);
        if (lane >= off) sum += o;
    }
    __syncthreads();
    if (lane == 31) warps[warp] = sum;
    __syncthreads();
    for (int i = 0; i < warp; ++i) sum += warps[i];
    return sum;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2)
sample_kernel(const Args a) {
    constexpr int kVec = Vec<T>::kSize;
    extern __shared__ uint4 slice[];
    __shared__ Shared sh;
    cg::cluster_group cluster = cg::this_cluster();
    cluster.barrier_arrive();   // waited for before the first write to another block's memory
    const int blocks = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int row = blockIdx.x / blocks, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int i0 = rank * a.slice;   // the slice's first token
    // a warp goes over consecutive vectors of the slice
    const int vectors = a.slice / kVec, each = (vectors + kWarps - 1) / kWarps;
    const int v_begin = min(vectors, warp * each), v_end = min(vectors, v_begin + each);
    const auto remote = [&](auto* p, int r) { return cluster.map_shared_rank(p, r); };

    // ---- the row's settings, by one thread: a double takes an SM long
    const float temperature = a.temperature ? a.temperature[row] : 1.0f;
    if (tid == kThreads - 1) {
        const double c = 1.4426950408889634 / static_cast<double>(temperature);
        sh.ch = static_cast<float>(c);
        sh.cl = static_cast<float>(c - static_cast<double>(sh.ch));
        const float least = a.min_p ? a.min_p[row] : 0.0f;
        if (least > 0.0f) {   // T ln(min-p), in two floats
            const double t = static_cast<double>(temperature) * log(fmin(static_cast<double>(least), 1.0));
            sh.far = static_cast<float>(t);
            sh.far_rest = static_cast<float>(t - static_cast<double>(sh.far));
        } else {
            sh.far = -INFINITY;
        }
    }
    // ---- the row into shared memory; the largest logit and its first place, and the
    // largest of every group of lanes
    uint64_t best;
    {
        const T* from = static_cast<const T*>(a.logits) + static_cast<int64_t>(row) * a.ld;
        const bool aligned = (reinterpret_cast<uintptr_t>(from) & 15) == 0;
        float most = -INFINITY;
        int at = v_begin + lane;   // the vector that has it first
#pragma unroll 8
        for (int v = v_begin + lane; v < v_end; v += 32) {
            const int i = i0 + v * kVec;
            Vec<T> x;
            if (aligned && i + kVec <= a.V) x.v = *reinterpret_cast<const uint4*>(from + i);
            else x.load(from + i, a.V - i);
            x.clean();
            slice[v] = x.v;
            const float m = x.largest();
            if (m > most) {
                most = m;
                at = v;
            }
        }
        uint32_t key = moe::order_key(most);
        if (tid < 64) sh.powers[tid] = kPowers[tid];
        // the warp's first token with its largest logit
        const uint32_t top_key = __reduce_max_sync(0xffffffffu, key);
        int first = INT_MAX;
        if (key == top_key && at < v_end) {
            float l[kVec];
            Vec<T>{slice[at]}.unpack(l);
#pragma unroll
            for (int j = kVec - 1; j >= 0; --j)
                if (moe::order_key(l[j]) == key) first = i0 + at * kVec + j;
        }
        first = __reduce_min_sync(0xffffffffu, first);
        if (lane == 0) sh.warp[warp] = static_cast<uint64_t>(top_key) << 32 | static_cast<uint32_t>(~first);
        for (int off = 1; off < blocks; off <<= 1) key = max(key, __shfl_xor_sync(0xffffffffu, key, off));
        if (tid % blocks == 0) sh.key[tid / blocks] = key;
        if (tid == 0) sh.listed = 0;
        __syncthreads();
        cluster.barrier_wait();   // all blocks have started: their shared memory is there
        {
            const int groups = kGroups / blocks, to = tid / groups, i = tid % groups;
            *remote(&sh.group[rank * groups + i], to) = sh.key[i];
        }
        if (tid < blocks) {
            best = sh.warp[0];
            for (int i = 1; i < kWarps; ++i) best = sh.warp[i] > best ? sh.warp[i] : best;
            *remote(&sh.best[rank], tid) = best;
        }
        cluster.sync();
        best = sh.best[0];
        for (int r = 1; r < blocks; ++r) best = sh.best[r] > best ? sh.best[r] : best;
    }
    const float top = moe::key_value(static_cast<uint32_t>(best >> 32));
    if (top == -INFINITY || !(temperature >= 1.17549435e-38f)) {   // nothing to draw from, or greedy
        if (rank == 0 && tid == 0) {
            a.token[row] = top == -INFINITY ? -1 : static_cast<int32_t>(~static_cast<uint32_t>(best));
            if (a.logprob) a.logprob[row] = top == -INFINITY ? -INFINITY : 0.0f;
        }
        cluster.sync();   // no block leaves while another may write to it
        return;
    }
    Weight weight;
    weight.top = top;
    weight.ch = sh.ch;
    weight.cl = sh.cl;
    weight.powers = sh.powers;

    // fn(l, i): a count or weight of token i, nothing below `from`.  Sums over the row:
    // every block's in sh.total, the warps' in sh.warp.
    const auto sums = [&](float from, auto fn) {
        uint64_t mine = 0;
        for (int v = v_begin + lane; v < v_end; v += 32) {
            const Vec<T> x{slice[v]};
            if (x.largest() < from) continue;
            float l[kVec];
            x.unpack(l);
#pragma unroll
            for (int j = 0; j < kVec; ++j) mine += fn(l[j], i0 + v * kVec + j);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, off);
        if (lane == 0) sh.warp[warp] = mine;
        __syncthreads();
        if (tid < blocks) {
            uint64_t all = 0;
            for (int i = 0; i < kWarps; ++i) all += sh.warp[i];
            *remote(&sh.total[rank], tid) = all;
        }
        cluster.sync();
        uint64_t all = 0;
        for (int r = 0; r < blocks; ++r) all += sh.total[r];
        return all;
    };
    // After sums of fn: calls take(l, i) on a thread that has found the first token at
    // which the running sum exceeds `target`.  Its block looks for it among the tokens
    // of its warp, two a thread at a time.
    const auto locate = [&](auto fn, uint64_t target, auto take) {
        uint64_t before = 0;
        for (int r = 0; r < rank; ++r) before += sh.total[r];
        if (target < before || target - before >= sh.total[rank]) return;
        int w = 0;
        for (; w < kWarps - 1 && target >= before + sh.warp[w]; ++w) before += sh.warp[w];
        const T* tokens = reinterpret_cast<const T*>(slice);
        const int end = min(vectors, (w + 1) * each) * kVec;
        for (int t0 = w * each * kVec; t0 < end; t0 += 2 * kThreads) {
            const int t = t0 + 2 * tid;   // and t + 1: end is even
            const float l0 = t < end ? static_cast<float>(tokens[t]) : -INFINITY, l1 = t < end ? static_cast<float>(tokens[t + 1]) : -INFINITY;
            const uint64_t w0 = t < end ? fn(l0, i0 + t) : 0, w1 = t < end ? fn(l1, i0 + t + 1) : 0;
            const uint64_t upto = before + running(w0, w1, sh.warp);
            if (target < upto && target >= upto - w1) take(l1, i0 + t + 1);
            else if (target < upto - w1 && target >= upto - w1 - w0) take(l0, i0 + t);
            for (int i = 0; i < kWarps; ++i) before += sh.warp[i];
            if (target < before) return;
        }
    };

    // whether a token is not behind the cut in the order
    const auto before_cut = [&](float l, int i, float cut_l, int cut_i) { return l >= cut_l && (l > cut_l || i <= cut_i); };
    const auto weight_at = [&](uint64_t place) { return weight(moe::key_value(static_cast<uint32_t>(place >> 32))); };
    // A block lists tokens for itself; after a cluster.sync, the number of all blocks',
    // and, if they are at most kSorted, the first block takes them together.
    const auto list = [&](float l, int i) {
        const uint32_t at = atomicAdd(&sh.listed, 1u);
        if (at < kSorted) sh.list[at] = place_of(l, i);
    };
    const auto take_listed = [&]() {
        int upto[kMaxBlocks];
#pragma unroll
        for (int r = 0; r < kMaxBlocks; ++r) upto[r] = r < blocks ? static_cast<int>(*remote(&sh.listed, r)) : 0;
#pragma unroll
        for (int r = 1; r < kMaxBlocks; ++r) upto[r] += upto[r - 1];
        const int n = upto[kMaxBlocks - 1];
        if (rank == 0 && n <= kSorted) {
            for (int i = upto[0] + tid; i < n; i += kThreads) {
                int r = 0, first = 0;
#pragma unroll
                for (int q = 0; q < kMaxBlocks - 1; ++q)
                    if (i >= upto[q]) r = q + 1, first = upto[q];
                sh.list[i] = *remote(&sh.list[i - first], r);
            }
            __syncthreads();
        }
        return n;
    };
    // n places in order, by one block: few are counted, into the histogram's place;
    // more are sorted where they are.
    const auto count_places = [&](const uint64_t* from, int n) -> const uint64_t* {
        auto* places = reinterpret_cast<uint64_t*>(sh.lo);
        if (tid < n) {
            const uint64_t place = from[tid];
            int before = 0;
#pragma unroll 4
            for (int i = 0; i < n; ++i) before += from[i] > place;
            places[before] = place;
        }
        __syncthreads();
        return places;
    };
    const auto sort_list = [&](int n) -> const uint64_t* {
        const int size = padded(n);
        for (int i = n + tid; i < size; i += kThreads) sh.list[i] = 0;
        __syncthreads();
        sort_places(sh.list, size);
        return sh.list;
    };
    // Of n listed places, by one block, those around the one that reaches a target, in
    // order, and their number and the sum before them: more than a few are divided by
    // their keys first (1000 of them: 2 us, against 7 for sorting them), unless many
    // are alike.
    const auto around = [&](int& n, bool by_weight, uint64_t target, uint64_t& above) -> const uint64_t* {
        if (n <= kCountedFirst) return count_places(sh.list, n);
        uint32_t low = 0xFFFFFFFFu, high = 0;
        for (int i = tid; i < n; i += kThreads) {
            const uint32_t key = static_cast<uint32_t>(sh.list[i] >> 32);
            low = min(low, key);
            high = max(high, key);
        }
        low = __reduce_min_sync(0xffffffffu, low);
        high = __reduce_max_sync(0xffffffffu, high);
        if (lane == 0) sh.warp[warp] = static_cast<uint64_t>(low) << 32 | high;
        sh.lo[tid] = sh.hi[tid] = 0;   // a bin a thread
        if (tid == 0) sh.kept = 0;
        __syncthreads();
        for (int i = 0; i < kWarps; ++i) {
            low = min(low, static_cast<uint32_t>(sh.warp[i] >> 32));
            high = max(high, static_cast<uint32_t>(sh.warp[i]));
        }
        const int shift = max(0, 32 - __clz(high - low) - 9);
        static_assert(kThreads == 1 << 9, "as many bins");
        const auto bin_of = [&](uint64_t place) { return static_cast<int>((high - static_cast<uint32_t>(place >> 32)) >> shift); };
        for (int i = tid; i < n; i += kThreads) {
            const uint64_t w = by_weight ? weight_at(sh.list[i]) : 1;
            const uint32_t lo = static_cast<uint32_t>(w), was = atomicAdd(&sh.lo[bin_of(sh.list[i])], lo);
            atomicAdd(&sh.hi[bin_of(sh.list[i])], static_cast<uint32_t>(w >> 32) + (was + lo < was));
        }
        __syncthreads();
        const uint64_t mine = static_cast<uint64_t>(sh.hi[tid]) << 32 | sh.lo[tid], upto = above + running(0, mine, sh.warp);
        if (upto >= target && upto - mine < target) {
            sh.found[0] = tid;
            sh.found[1] = upto - mine;
        }
        __syncthreads();
        auto* few = reinterpret_cast<uint64_t*>(sh.hi + kThreads);   // behind the bins
        static_assert(2 * kCounted <= kBins && kThreads + 2 * kCounted <= kBins, "room for both");
        for (int i = tid; i < n; i += kThreads)
            if (bin_of(sh.list[i]) == static_cast<int>(sh.found[0])) {
                const int at = atomicAdd(&sh.kept, 1);
                if (at < kCounted) few[at] = sh.list[i];
            }
        __syncthreads();
        if (sh.kept > kCounted) return sort_list(n);
        n = sh.kept;
        above = sh.found[1];
        return count_places(few, n);
    };

    // The token at which the sum in the order reaches a target: the place of the
    // last one kept.  Among the tokens at or before `cut` in the order; by_weight: the
    // target is the share p of their weights, else the number k.
    const auto cut_at = [&](uint64_t cut, bool by_weight, int k, float p) {
        uint64_t target = static_cast<uint64_t>(k), above = 0;
        uint32_t low = 0, high = 0;   // keys of the bin, once known
        int shift = -1;               // -1: the first histogram, of distances to the largest
        const float scale = sh.ch * (static_cast<float>(kBins) / kOctaves);
        const float cut_l = cut ? moe::key_value(static_cast<uint32_t>(cut >> 32)) : -INFINITY;
        const int cut_i = cut ? static_cast<int>(~static_cast<uint32_t>(cut)) : INT_MAX;
        for (;;) {
            // to the nearest; what is not a number (of an infinite largest) in the last
            const auto first_bin_of = [&](float l) { return __float_as_int(fminf((top - l) * scale, kBins - 1) + 12582912.0f) - __float_as_int(12582912.0f); };
            const auto bin_of = [&](float l) {   // -1: outside
                if (shift < 0) return first_bin_of(l);
                const uint32_t key = moe::order_key(l);
                return key >= low && key <= high ? static_cast<int>((high - key) >> shift) : -1;
            };
            for (int i = tid; i < kBins; i += kThreads) sh.lo[i] = sh.hi[i] = 0;
            __syncthreads();
            // The last bin has most of a steep row's tokens, which would wait for one
            // another (at 32 octaves below the largest 36000 cycles for a block's 16384
            // tokens instead of 16000): its sum is what the thread's tokens have beyond
            // those that it counts into the other bins.
            uint64_t last = 0;
            const bool every = shift < 0 && cut == 0;   // no token is left out
            for (int v = v_begin + lane; v < v_end; v += 32) {
                float l[kVec];
                Vec<T>{slice[v]}.unpack(l);
#pragma unroll
                for (int j0 = 0; j0 < kVec; j0 += 4) {   // four on their way at a time
                    uint64_t w[4];
                    uint32_t was[4];
                    int bin[4], least = kBins - 1;
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[j] = by_weight ? weight(l[j0 + j]) : 1;
                    if (every) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) bin[j] = first_bin_of(l[j0 + j]);
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            bin[j] = bin_of(l[j0 + j]);
                            if (bin[j] < 0 || !before_cut(l[j0 + j], i0 + v * kVec + j0 + j, cut_l, cut_i)) w[j] = 0, bin[j] = kBins - 1;
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        last += w[j];
                        least = min(least, bin[j]);
                    }
                    if (least == kBins - 1) continue;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (bin[j] == kBins - 1) w[j] = 0;
                        last -= w[j];
                        was[j] = static_cast<uint32_t>(w[j]) ? atomicAdd(&sh.lo[bin[j]], static_cast<uint32_t>(w[j])) : 0;
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t carry = was[j] + static_cast<uint32_t>(w[j]) < was[j], hi = static_cast<uint32_t>(w[j] >> 32) + carry;
                        if (hi) atomicAdd(&sh.hi[bin[j]], hi);
                    }
                }
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) last += __shfl_xor_sync(0xffffffffu, last, off);
            if (lane == 0 && last) {
                const uint32_t lo = static_cast<uint32_t>(last), was = atomicAdd(&sh.lo[kBins - 1], lo);
                atomicAdd(&sh.hi[kBins - 1], static_cast<uint32_t>(last >> 32) + (was + lo < was));
            }
            __syncthreads();
            // the sums of kShare bins each, to all blocks
            uint64_t mine = 0;
#pragma unroll
            for (int i = 0; i < kShare; i += 32) {
                const int at = warp * kShare + i + lane;
                mine += static_cast<uint64_t>(sh.hi[at]) << 32 | sh.lo[at];
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, off);
            if (lane < blocks) *remote(&sh.share[rank][warp], lane) = mine;
            if (tid == 0) sh.listed = 0;
            cluster.sync();
            // where the target is reached, the share and then the bin, every block for itself
            mine = 0;
#pragma unroll
            for (int r = 0; r < kMaxBlocks; ++r)
                if (r < blocks && lane < kWarps) mine += sh.share[r][lane];
            uint64_t upto = mine;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const uint64_t o = __shfl_up_sync(0xffffffffu, upto, off);
                if (lane >= off) upto += o;
            }
            if (by_weight && shift < 0) target = share_reached(p, __shfl_sync(0xffffffffu, upto, 31));
            const int share = min(kWarps, __ffs(__ballot_sync(0xffffffffu, above + upto >= target))) - 1;
            above += __shfl_sync(0xffffffffu, upto - mine, share);
            uint64_t sum = 0;
            if (tid < kShare) {
#pragma unroll
                for (int r = 0; r < kMaxBlocks; ++r)   // all on their way at once
                    if (r < blocks) sum += static_cast<uint64_t>(*remote(&sh.hi[share * kShare + tid], r)) << 32 | *remote(&sh.lo[share * kShare + tid], r);
            }
            upto = above + running(0, sum, sh.warp);
            if (upto >= target && upto - sum < target) {
                sh.found[0] = share * kShare + tid;
                sh.found[1] = upto - sum;
            }
            __syncthreads();
            const int bin = static_cast<int>(sh.found[0]);
            above = sh.found[1];
            const auto in_this = [&](float l, int i) {
                return bin_of(l) == bin && before_cut(l, i, cut_l, cut_i) && (!by_weight || weight(l) != 0);
            };
            const auto below = [&](float l) { return shift < 0 ? bin_of(l) > bin : moe::order_key(l) < low; };
            // those in it are listed, if they are few, and ordered by the first block
            for (int v = v_begin + lane; v < v_end; v += 32) {
                const Vec<T> x{slice[v]};
                if (below(x.largest())) continue;
                float l[kVec];
                x.unpack(l);
#pragma unroll
                for (int j = 0; j < kVec; ++j) {
                    const int i = i0 + v * kVec + j;
                    if (in_this(l[j], i)) list(l[j], i);
                }
            }
            cluster.sync();
            int n = take_listed();
            if (n <= kSorted) {
                if (rank == 0) {
                    const uint64_t* ordered = around(n, by_weight, target, above);
                    if (!by_weight) {
                        if (tid == 0) sh.found[0] = ordered[target - above - 1];
                    } else {
                        const uint64_t first = 2 * tid < n ? weight_at(ordered[2 * tid]) : 0, second = 2 * tid + 1 < n ? weight_at(ordered[2 * tid + 1]) : 0;
                        const uint64_t upto = above + running(first, second, sh.warp);
                        if (upto - second >= target && upto - second - first < target) sh.found[0] = ordered[2 * tid];
                        else if (upto >= target && upto - second < target) sh.found[0] = ordered[2 * tid + 1];
                    }
                    __syncthreads();
                    if (tid > 0 && tid < blocks) *remote(&sh.found[0], tid) = sh.found[0];
                }
                cluster.sync();
                return sh.found[0];
            }
            // the keys in the bin, or tokens of one value
            uint32_t least = 0xFFFFFFFFu, most = 0;
            for (int v = v_begin + lane; v < v_end; v += 32) {
                const Vec<T> x{slice[v]};
                if (below(x.largest())) continue;
                float l[kVec];
                x.unpack(l);
#pragma unroll
                for (int j = 0; j < kVec; ++j) {
                    if (!in_this(l[j], i0 + v * kVec + j)) continue;
                    const uint32_t key = moe::order_key(l[j]);
                    least = min(least, key);
                    most = max(most, key);
                }
            }
            least = __reduce_min_sync(0xffffffffu, least);
            most = __reduce_max_sync(0xffffffffu, most);
            if (lane == 0) sh.warp[warp] = static_cast<uint64_t>(least) << 32 | most;
            __syncthreads();
            if (tid < blocks) {
                for (int i = 0; i < kWarps; ++i) {
                    least = min(least, static_cast<uint32_t>(sh.warp[i] >> 32));
                    most = max(most, static_cast<uint32_t>(sh.warp[i]));
                }
                *remote(&sh.total[rank], tid) = static_cast<uint64_t>(least) << 32 | most;
            }
            cluster.sync();
            low = 0xFFFFFFFFu, high = 0;
            for (int r = 0; r < blocks; ++r) {
                low = min(low, static_cast<uint32_t>(sh.total[r] >> 32));
                high = max(high, static_cast<uint32_t>(sh.total[r]));
            }
            if (low == high) {
                const uint64_t one = by_weight ? weight(moe::key_value(high)) : 1;
                const uint64_t which = (target - above + one - 1) / one;   // counted from 1
                const auto tie = [&](float l, int i) { return static_cast<uint64_t>(moe::order_key(l) == high && before_cut(l, i, cut_l, cut_i)); };
                cluster.sync();   // sh.total has been read
                sums(moe::key_value(high), tie);
                locate(tie, which - 1, [&](float l, int i) {
                    for (int r = 0; r < blocks; ++r) *remote(&sh.found[0], r) = place_of(l, i);
                });
                cluster.sync();
                return sh.found[0];
            }
            shift = max(0, 32 - __clz(high - low) - 11);   // 2048 bins
            cluster.sync();   // sh.found and sh.total have been read
        }
    };

    const int k = a.top_k && a.top_k[row] > 0 && a.top_k[row] < a.V ? a.top_k[row] : 0;   // 0: all
    const float p = a.top_p ? a.top_p[row] : 1.0f, u = a.u[row];
    // min-p: the least float that is not below L + T ln(min-p)
    float least = -INFINITY;
    if (sh.far > -INFINITY) {
        const float sum = top + sh.far, b = sum - top, off = (top - (sum - b)) + (sh.far - b) + sh.far_rest;
        least = top == INFINITY || !(off > 0.0f) ? sum : nextafterf(sum, INFINITY);
    }
    const auto target_of = [&](uint64_t all) -> uint64_t {
        bool rest;
        return !(u > 0.0f) ? 0 : u < 1.0f ? share_below(u, all, rest) : all - 1;
    };
    // logarithms of neither sign's cancel: fp32 will do
    const auto drawn = [&](float l, int i, uint64_t all) {
        a.token[row] = i;
        if (a.logprob)
            a.logprob[row] = (l == top ? 0.0f : (l - top) / temperature) - log1pf(static_cast<float>(all - (1ull << kUnit)) * (1.0f / (1ull << kUnit)));
    };

    // ---- A few tokens: at least q of the row's are as large as the q-th largest of the
    // groups' largest, and hardly more.  With top-k, k = q, those are listed and sorted,
    // and all that follows is one block's.
    if (k > 0 && k <= kFew) {
        // the bound: that key's upper half, 4 bits a time, a warp for each value of them
        uint32_t mine[kGroups / 32], bound = 0;
#pragma unroll
        for (int i = 0; i < kGroups / 32; ++i) mine[i] = sh.group[lane + 32 * i];
#pragma unroll 1
        for (int bit = 28; bit >= 16; bit -= 4) {
            const uint32_t next = bound | static_cast<uint32_t>(warp) << bit;
            int n = 0;
#pragma unroll
            for (int i = 0; i < kGroups / 32; ++i) n += mine[i] >= next;
            n = __reduce_add_sync(0xffffffffu, n);
            uint32_t* enough = sh.key + (bit & 4 ? kWarps : 0);   // two in turn
            if (lane == 0) enough[warp] = n >= k;
            __syncthreads();
            // those that enough keys reach are the first ones
            bound |= (__popc(__ballot_sync(0xffffffffu, lane < kWarps && enough[lane % kWarps])) - 1) << bit;
        }
        // the smallest float that has at least this key; no bound (a row of few blocks with tokens): none
        const float from = bound > 0x007FFFFFu ? moe::key_value(bound) : -INFINITY;
        if (from > -INFINITY)
#pragma unroll 2
            for (int v = v_begin + lane; v < v_end; v += 32) {
                const Vec<T> x{slice[v]};
                if (!(x.largest() >= from)) continue;
                float l[kVec];
                x.unpack(l);
#pragma unroll
                for (int j = 0; j < kVec; ++j)
                    if (l[j] >= from) {
                        const uint32_t at = atomicAdd(remote(&sh.listed, 0), 1u);
                        if (at < kSorted) *remote(&sh.list[at], 0) = place_of(l[j], i0 + v * kVec + j);
                    }
            }
        cluster.sync();
        const int n = static_cast<int>(*remote(&sh.listed, 0));
        if (n <= kSorted && n >= k) {
            if (rank == 0 && n <= kCounted) {
                const uint64_t* places = count_places(sh.list, n);
                auto* weights = reinterpret_cast<uint64_t*>(sh.hi);
                if (tid < k) weights[tid] = weight_at(places[tid]);
                __syncthreads();
                int m = k;   // those kept are the first m
                if (p < 1.0f) {
                    const uint64_t mine = tid < m ? weights[tid] : 0, upto = running(0, mine, sh.warp);
                    uint64_t sum = 0;
                    for (int i = 0; i < kWarps; ++i) sum += sh.warp[i];
                    const uint64_t reach = share_reached(p, sum);
                    if (upto >= reach && upto - mine < reach) sh.kept = tid + 1;
                    __syncthreads();
                    m = sh.kept;
                }
                if (tid < m && moe::key_value(static_cast<uint32_t>(places[tid] >> 32)) < least) weights[tid] = 0;
                __syncthreads();
                if (tid < m) {
                    const uint64_t place = places[tid], mine = weights[tid];
                    uint64_t sum = 0, before = 0;   // all, and those with lower indexes
#pragma unroll 4
                    for (int i = 0; i < m; ++i) {
                        const uint64_t w = weights[i];
                        sum += w;
                        if (static_cast<uint32_t>(places[i]) > static_cast<uint32_t>(place)) before += w;
                    }
                    const uint64_t target = target_of(sum);
                    if (target >= before && target < before + mine)
                        drawn(moe::key_value(static_cast<uint32_t>(place >> 32)), static_cast<int>(~static_cast<uint32_t>(place)), sum);
                }
            } else if (rank == 0) {
                sort_list(n);
                int m = k;   // those kept are the first m
                uint64_t first = 2 * tid < m ? weight_at(sh.list[2 * tid]) : 0, second = 2 * tid + 1 < m ? weight_at(sh.list[2 * tid + 1]) : 0;
                if (p < 1.0f) {
                    const uint64_t upto = running(first, second, sh.warp);
                    uint64_t sum = 0;
                    for (int i = 0; i < kWarps; ++i) sum += sh.warp[i];
                    const uint64_t reach = share_reached(p, sum);
                    if (upto - second >= reach && upto - second - first < reach) sh.kept = 2 * tid + 1;
                    else if (upto >= reach && upto - second < reach) sh.kept = 2 * tid + 2;
                    __syncthreads();
                    m = sh.kept;
                }
                {   // in the order of the vocabulary
                    __syncthreads();
                    const int size2 = padded(m);
                    for (int i = tid; i < size2; i += kThreads) {
                        const uint64_t place = sh.list[i];
                        const bool in = i < m && moe::key_value(static_cast<uint32_t>(place >> 32)) >= least;
                        sh.list[i] = in ? place << 32 | place >> 32 : 0;
                    }
                    __syncthreads();
                    sort_places(sh.list, size2);
                    const auto value = [&](int i) { return moe::key_value(static_cast<uint32_t>(sh.list[i])); };
                    first = 2 * tid < size2 && sh.list[2 * tid] ? weight(value(2 * tid)) : 0;
                    second = 2 * tid + 1 < size2 && sh.list[2 * tid + 1] ? weight(value(2 * tid + 1)) : 0;
                    const uint64_t upto = running(first, second, sh.warp);
                    uint64_t sum = 0;
                    for (int i = 0; i < kWarps; ++i) sum += sh.warp[i];
                    const uint64_t target = target_of(sum);
                    if (target < upto && target >= upto - first - second) {
                        const int i = 2 * tid + (target >= upto - second ? 1 : 0);
                        drawn(value(i), static_cast<int>(~static_cast<uint32_t>(sh.list[i] >> 32)), sum);
                    }
                }
            }
            // the others leave; the first stays until they have, who read its count
            if (rank == 0) cluster.sync();
            return;
        }
        cluster.sync();
    }

    // ---- any other row
    uint64_t cut = 0;
    if (k) cut = cut_at(cut, false, k, 0.0f);
    if (p < 1.0f) cut = cut_at(cut, true, 0, p);
    const float cut_l = cut ? moe::key_value(static_cast<uint32_t>(cut >> 32)) : -INFINITY;
    const int cut_i = cut ? static_cast<int>(~static_cast<uint32_t>(cut)) : INT_MAX;
    const auto kept = [&](float l, int i) -> uint64_t { return weight(l >= least && before_cut(l, i, cut_l, cut_i) ? l : -INFINITY); };   // without a branch
    const uint64_t all = sums(fmaxf(least, cut_l), kept);
    locate(kept, target_of(all), [&](float l, int i) { drawn(l, i, all); });
    cluster.sync();   // no block leaves while another may read its sums
}

// Bytes of a row that a block may hold: an eighth of the largest vocabulary, or what lets
// two blocks share an SM (1 KB of each block's is the system's), whichever is more: in
// bf16 the latter.
constexpr size_t kTwoAnSm = 114 * 1024 - 1024 - (sizeof(Shared) + 15) / 16 * 16;
template <typename T>
constexpr size_t kMostSlice = std::max(kMaxV / kMaxBlocks * sizeof(T), kTwoAnSm);

template <typename T>
moe_status_t launch(Args a, int rows, cudaStream_t s) {
    static std::atomic<int> allowed[moe::kMaxDevices];
    int dev = 0;
    MOE_CHECK_CUDA(cudaGetDevice(&dev));
    if (dev < 0 || dev >= moe::kMaxDevices) return MOE_ERR_CUDA;
    if (!allowed[dev].load(std::memory_order_relaxed)) {
        MOE_CHECK_CUDA(cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kMostSlice<T>)));
        allowed[dev].store(1, std::memory_order_relaxed);
    }
    // Eight blocks a row, or fewer where the GPU would not hold all rows' at once, two an
    // SM, and still holds them so: every block waits for others some 5 us.  us with eight,
    // and with four, for 131072 tokens in bf16: top-k, 16 rows 17, 19; 32 rows 19, 19; 64
    // rows 27, 22; 256 rows 87, 61; top-p, 64 rows 82, 85; 256 rows 274, 244.  256 rows of
    // 32000: eight 67, four 43, the one of the rule 26.
    const int sms = moe::sm_count();
    if (sms <= 0) return MOE_ERR_CUDA;
    const auto slice_of = [&](int n) { return ((a.V + n - 1) / n + 7) / 8 * 8; };
    int blocks = kMaxBlocks;
    while (blocks > 1 && static_cast<int64_t>(rows) * blocks > 2 * sms && slice_of(blocks / 2) * sizeof(T) <= kTwoAnSm) blocks /= 2;
    a.slice = slice_of(blocks);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(rows) * blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(a.slice) * sizeof(T);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = blocks;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, sample_kernel<T>, a) != cudaSuccess) {
        (void)cudaGetLastError();
        return MOE_ERR_CUDA;
    }
    return MOE_OK;
}

}  // namespace

extern "C" moe_status_t moe_sample(moe_dtype_t dtype, const void* logits, int64_t ld, int rows, int V, const float* temperature,
                                   const int32_t* top_k, const float* top_p, const float* min_p, const float* u, int32_t* token,
                                   float* logprob, moe_stream_t stream) {
    MOE_CHECK_ARG(dtype == MOE_BF16 || dtype == MOE_F32);
    MOE_CHECK_ARG(logits && u && token && rows >= 1 && V >= 1 && ld >= V);
    MOE_CHECK_ARG(moe::aligned_to(logits, dtype == MOE_BF16 ? 2 : 4) && moe::aligned16(temperature) && moe::aligned16(top_k) &&
                  moe::aligned16(top_p) && moe::aligned16(min_p) && moe::aligned16(u) && moe::aligned16(token) && moe::aligned16(logprob));
    if (V > kMaxV || rows > (1 << 27)) return MOE_ERR_UNSUPPORTED;
    const Args a{logits, ld, V, 0, temperature, top_k, top_p, min_p, u, token, logprob};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return dtype == MOE_BF16 ? launch<__nv_bfloat16>(a, rows, s) : launch<float>(a, rows, s);
}
