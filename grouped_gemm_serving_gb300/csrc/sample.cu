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
// closer (its tokens are sorted by one block if they are few, else its range of
// values is divided again, down to tokens of one value, which are counted); and for
// the draw.  No pass sorts the vocabulary.
//
// A draw falls to another token wherever a running sum is off by more than u is from
// it, so sums are exact: weights are integers, multiples of 2^-44 of the largest,
// that add up in any order, and good to some 2^-37 of themselves.  With weights in
// fp32 (2^-23) one row in ten thousand of a flat distribution over 131072 tokens would
// draw its neighbour.
#include <cooperative_groups.h>

#include "common.cuh"

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kBinsPerOctave = 32;   // of the first histogram: 64 octaves below the largest weight
constexpr int kSorted = 1024;        // tokens that one block sorts
constexpr int kMaxBlocks = 8;        // of a cluster
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

// exp((l - L) / T) in units of 2^-44, for l <= L.
struct Weight {
    float top;       // L
    float ch, cl;    // log2(e) / T in two parts
    const uint64_t* powers;

    // t = (l - L) c = m / 64 + r with |r| <= 1/128, and 2^t = 2^(m / 64) e^(r ln 2): a table
    // of 64 powers and four terms of the series (as in P. Tang's table-driven
    // exponentials).  t, r and the series' first term are kept in two floats each.
    __device__ __forceinline__ uint64_t operator()(float l) const {
        if (l == top) return 1ull << 44;
        const float d = l - top;
        const float p = d * ch;
        if (!(p > -46.0f)) return 0;   // less than a unit; -infinity; NaN of infinity times 0
        const float b = d - l, de = (l - (d - b)) + (-top - b);   // d + de = l - L
        const float pe = fmaf(d, ch, -p) + fmaf(d, cl, de * ch);
        const float big = 12582912.0f;   // 1.5 * 2^23
        const float shifted = fmaf(p, 64.0f, big);
        const int m = __float_as_int(shifted) - __float_as_int(big);
        const float rh = fmaf(shifted - big, -0.015625f, p);
        constexpr float kLn2 = 0.693147182f, kLn2Rest = -1.90465421e-9f;   // ln 2 in two floats
        const float y = rh * kLn2;
        const float ye = fmaf(rh, kLn2, -y) + fmaf(rh, kLn2Rest, pe * kLn2);
        const float rest = fmaf(ye, y, ye) + y * y * fmaf(y, fmaf(y, 0.0416666679f, 0.166666672f), 0.5f);
        const int e = __float2int_rn(y * 137438953472.0f) + __float2int_rn(rest * 137438953472.0f);   // e^.. - 1 in 2^-37
        const uint64_t power = powers[m & 63];
        const uint64_t w = power + static_cast<uint64_t>((static_cast<int64_t>(e) * static_cast<int32_t>(power >> 32)) >> 5);
        const int shift = 18 - (m >> 6);
        return shift < 64 ? w >> shift : 0;
    }
};

// A token's place in the order, larger first: its logit's key, then its index.
__device__ __forceinline__ uint64_t place_of(float l, int i) { return static_cast<uint64_t>(moe::order_key(l)) << 32 | static_cast<uint32_t>(~i); }

template <typename T>
struct Slice;
template <>
struct Slice<float> {
    static constexpr int kVec = 4;
    __device__ static __forceinline__ void get(const void* s, int v, float (&l)[4]) {
        const float4 x = static_cast<const float4*>(s)[v];
        l[0] = x.x, l[1] = x.y, l[2] = x.z, l[3] = x.w;
    }
    __device__ static __forceinline__ void put(void* s, int v, const float (&l)[4]) { static_cast<float4*>(s)[v] = make_float4(l[0], l[1], l[2], l[3]); }
    __device__ static __forceinline__ float value(float x) { return x; }
};
template <>
struct Slice<__nv_bfloat16> {
    static constexpr int kVec = 8;
    __device__ static __forceinline__ void get(const void* s, int v, float (&l)[8]) {
        const uint4 x = static_cast<const uint4*>(s)[v];
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            l[2 * i] = moe::bf16_lo(w[i]);
            l[2 * i + 1] = moe::bf16_hi(w[i]);
        }
    }
    __device__ static __forceinline__ void put(void* s, int v, const float (&l)[8]) {   // values of bf16: cut in half
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __byte_perm(__float_as_uint(l[2 * i]), __float_as_uint(l[2 * i + 1]), 0x7632);
        static_cast<uint4*>(s)[v] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ static __forceinline__ float value(__nv_bfloat16 x) { return __bfloat162float(x); }
};

struct Shared {
    uint32_t n[kBins], lo[kBins], hi[kBins];   // histogram: tokens, and their weights in two halves
    uint64_t list[kSorted];
    uint64_t powers[64];
    uint64_t warp[kWarps];
    uint64_t best[kMaxBlocks], total[kMaxBlocks];   // every block's, written by them
    uint64_t found[3];                                // written by the block that found it
    uint32_t listed;
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 2)
sample_kernel(const Args a) {
    using S = Slice<T>;
    constexpr int kVec = S::kVec;
    extern __shared__ __align__(16) uint8_t slice[];
    __shared__ Shared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int blocks = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int row = blockIdx.x / blocks, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int i0 = rank * a.slice;   // the slice's first token
    // a warp goes over consecutive vectors of the slice
    const int vectors = a.slice / kVec, each = (vectors + kWarps - 1) / kWarps;
    const int v_begin = min(vectors, warp * each), v_end = min(vectors, v_begin + each);
    const auto remote = [&](auto* p, int r) { return cluster.map_shared_rank(p, r); };

    // ---- the row into shared memory; the largest logit and its first place
    uint64_t best = 0;
    {
        const T* from = static_cast<const T*>(a.logits) + static_cast<int64_t>(row) * a.ld;
        const bool aligned = (reinterpret_cast<uintptr_t>(from) & 15) == 0;
        for (int v = v_begin + lane; v < v_end; v += 32) {
            const int i = i0 + v * kVec;
            float l[kVec];
            if (aligned && i + kVec <= a.V) {
                S::get(from + i, 0, l);
            } else {
#pragma unroll
                for (int j = 0; j < kVec; ++j) l[j] = i + j < a.V ? S::value(from[i + j]) : -INFINITY;
            }
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                if (l[j] != l[j]) l[j] = -INFINITY;   // NaN: never drawn
                const uint64_t p = place_of(l[j], i + j);
                best = p > best ? p : best;
            }
            S::put(slice, v, l);
        }
        if (tid < 64) sh.powers[tid] = kPowers[tid];
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            const uint64_t o = __shfl_xor_sync(0xffffffffu, best, off);
            best = o > best ? o : best;
        }
        if (lane == 0) sh.warp[warp] = best;
        __syncthreads();
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
    const float temperature = a.temperature ? a.temperature[row] : 1.0f;
    if (top == -INFINITY || !(temperature >= 1.17549435e-38f)) {   // nothing to draw from, or greedy
        if (rank == 0 && tid == 0) {
            a.token[row] = top == -INFINITY ? -1 : static_cast<int32_t>(~static_cast<uint32_t>(best));
            if (a.logprob) a.logprob[row] = top == -INFINITY ? -INFINITY : 0.0f;
        }
        cluster.sync();   // no block leaves while another may write to it
        return;
    }
    const double c = 1.4426950408889634 / static_cast<double>(temperature);
    Weight weight;
    weight.top = top;
    weight.ch = static_cast<float>(c);
    weight.cl = static_cast<float>(c - static_cast<double>(weight.ch));
    weight.powers = sh.powers;

    // fn(l, i): a count or weight of token i.  Sums over the row: every block's in
    // sh.total, the warps' in sh.warp.
    const auto sums = [&](auto fn) {
        uint64_t mine = 0;
        for (int v = v_begin + lane; v < v_end; v += 32) {
            float l[kVec];
            S::get(slice, v, l);
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
    // After sums(fn): calls take(l, i) on the thread that holds the first token at which
    // the running sum exceeds `target`.
    const auto locate = [&](auto fn, uint64_t target, auto take) {
        uint64_t before = 0;
        for (int r = 0; r < rank; ++r) before += sh.total[r];
        for (int i = 0; i < warp; ++i) before += sh.warp[i];
        if (target < before || target >= before + sh.warp[warp]) return;
        for (int v = v_begin; v < v_end; v += 32) {
            float l[kVec];
            uint64_t w[kVec], mine = 0;
#pragma unroll
            for (int j = 0; j < kVec; ++j) l[j] = -INFINITY, w[j] = 0;
            if (v + lane < v_end) {
                S::get(slice, v + lane, l);
#pragma unroll
                for (int j = 0; j < kVec; ++j) {
                    w[j] = fn(l[j], i0 + (v + lane) * kVec + j);
                    mine += w[j];
                }
            }
            uint64_t upto = mine;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const uint64_t o = __shfl_up_sync(0xffffffffu, upto, off);
                if (lane >= off) upto += o;
            }
            const uint64_t all = __shfl_sync(0xffffffffu, upto, 31);
            if (target < before + all) {
                uint64_t at = before + upto - mine;
                if (target >= at && target < at + mine) {
#pragma unroll
                    for (int j = 0; j < kVec; ++j) {
                        if (target >= at && target < at + w[j]) take(l[j], i0 + (v + lane) * kVec + j);
                        at += w[j];
                    }
                }
                return;
            }
            before += all;
        }
    };

    // The token at which the sum in the order reaches a target: the place of the
    // last one kept.  Among the tokens at or before `cut` in the order; by_weight: the
    // target is the share p of their weights, else the number k.
    const auto cut_at = [&](uint64_t cut, bool by_weight, int k, float p) {
        uint64_t target = static_cast<uint64_t>(k), above = 0, in_bin;
        uint32_t low = 0, high = 0;   // keys of the bin, once known
        int shift = -1;               // -1: the first histogram, of distances to the largest
        const float scale = static_cast<float>(c) * kBinsPerOctave;
        for (;;) {
            const auto bin_of = [&](float l, uint32_t key) {
                if (shift < 0) return l == -INFINITY ? kBins - 1 : min(kBins - 1, static_cast<int>((top - l) * scale));
                return static_cast<int>((high - key) >> shift);
            };
            const auto inside = [&](uint64_t place) {
                const uint32_t key = static_cast<uint32_t>(place >> 32);
                return place >= cut && (shift < 0 || (key >= low && key <= high));
            };
            for (int i = tid; i < kBins; i += kThreads) sh.n[i] = sh.lo[i] = sh.hi[i] = 0;
            __syncthreads();
            for (int v = v_begin + lane; v < v_end; v += 32) {
                float l[kVec];
                S::get(slice, v, l);
#pragma unroll
                for (int j = 0; j < kVec; ++j) {
                    const uint64_t place = place_of(l[j], i0 + v * kVec + j);
                    if (!inside(place)) continue;
                    const int bin = bin_of(l[j], static_cast<uint32_t>(place >> 32));
                    atomicAdd(&sh.n[bin], 1u);
                    if (by_weight) {
                        const uint64_t w = weight(l[j]);
                        const uint32_t w_lo = static_cast<uint32_t>(w);
                        uint32_t w_hi = static_cast<uint32_t>(w >> 32);
                        if (w_lo && atomicAdd(&sh.lo[bin], w_lo) + w_lo < w_lo) ++w_hi;   // carry
                        if (w_hi) atomicAdd(&sh.hi[bin], w_hi);
                    }
                }
            }
            cluster.sync();
            // this block's share of the bins, over all blocks; running sums over them
            const int per = kBins / blocks;   // at most kThreads
            uint64_t n = 0, w = 0;
            if (tid < per)
                for (int r = 0; r < blocks; ++r) {
                    n += *remote(&sh.n[rank * per + tid], r);
                    if (by_weight) w += static_cast<uint64_t>(*remote(&sh.hi[rank * per + tid], r)) * 4294967296ull + *remote(&sh.lo[rank * per + tid], r);
                }
            const uint64_t mine = by_weight ? w : n;
            uint64_t upto = mine;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const uint64_t o = __shfl_up_sync(0xffffffffu, upto, off);
                if (lane >= off) upto += o;
            }
            if (lane == 31) sh.warp[warp] = upto;
            __syncthreads();
            for (int i = 0; i < warp; ++i) upto += sh.warp[i];
            if (tid < blocks) {
                uint64_t all = 0;
                for (int i = 0; i < kWarps; ++i) all += sh.warp[i];
                *remote(&sh.total[rank], tid) = all;
            }
            cluster.sync();
            uint64_t before = above;
            if (by_weight && shift < 0) {   // the share of the sum
                uint64_t all = 0;
                for (int r = 0; r < blocks; ++r) all += sh.total[r];
                target = static_cast<uint64_t>(ceil(static_cast<double>(p) * static_cast<double>(all)));
            }
            if (target == 0) target = 1;   // the first token is always kept
            for (int r = 0; r < rank; ++r) before += sh.total[r];
            if (tid < per && before + upto >= target && before + upto - mine < target)
                for (int r = 0; r < blocks; ++r) {
                    uint64_t* to = remote(&sh.found[0], r);
                    to[0] = static_cast<uint64_t>(rank * per + tid);
                    to[1] = before + upto - mine;
                    to[2] = n;
                }
            if (tid == 0) sh.listed = 0;
            cluster.sync();
            const int bin = static_cast<int>(sh.found[0]);
            above = sh.found[1];
            in_bin = sh.found[2];
            const auto in_this = [&](float l, uint64_t place) { return inside(place) && bin_of(l, static_cast<uint32_t>(place >> 32)) == bin; };
            if (in_bin <= kSorted) {   // the first block sorts them
                for (int v = v_begin + lane; v < v_end; v += 32) {
                    float l[kVec];
                    S::get(slice, v, l);
#pragma unroll
                    for (int j = 0; j < kVec; ++j) {
                        const uint64_t place = place_of(l[j], i0 + v * kVec + j);
                        if (in_this(l[j], place)) {
                            const uint32_t at = atomicAdd(remote(&sh.listed, 0), 1u);
                            if (at < kSorted) *remote(&sh.list[at], 0) = place;
                        }
                    }
                }
                cluster.sync();
                if (rank == 0) {
                    int size = 32;
                    while (size < static_cast<int>(in_bin)) size *= 2;
                    for (int i = tid; i < size; i += kThreads)
                        if (i >= static_cast<int>(in_bin)) sh.list[i] = 0;
                    __syncthreads();
                    for (int block = 2; block <= size; block *= 2)   // bitonic, larger first
                        for (int step = block / 2; step > 0; step /= 2) {
                            for (int i = tid; i < size / 2; i += kThreads) {
                                const int x = 2 * step * (i / step) + i % step, y = x + step;
                                const uint64_t p0 = sh.list[x], p1 = sh.list[y];
                                if ((p0 < p1) == ((x & block) == 0)) {
                                    sh.list[x] = p1;
                                    sh.list[y] = p0;
                                }
                            }
                            __syncthreads();
                        }
                    if (!by_weight) {
                        if (tid == 0) sh.found[0] = sh.list[target - above - 1];
                    } else {
                        // two tokens a thread
                        uint64_t first = 0, second = 0;
                        const int at = 2 * tid;
                        if (at < static_cast<int>(in_bin)) first = weight(moe::key_value(static_cast<uint32_t>(sh.list[at] >> 32)));
                        if (at + 1 < static_cast<int>(in_bin)) second = weight(moe::key_value(static_cast<uint32_t>(sh.list[at + 1] >> 32)));
                        uint64_t sum = first + second;
#pragma unroll
                        for (int off = 1; off < 32; off <<= 1) {
                            const uint64_t o = __shfl_up_sync(0xffffffffu, sum, off);
                            if (lane >= off) sum += o;
                        }
                        if (lane == 31) sh.warp[warp] = sum;
                        __syncthreads();
                        for (int i = 0; i < warp; ++i) sum += sh.warp[i];
                        sum += above;
                        if (sum - second >= target && sum - second - first < target) sh.found[0] = sh.list[at];
                        else if (sum >= target && sum - second < target) sh.found[0] = sh.list[at + 1];
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
                float l[kVec];
                S::get(slice, v, l);
#pragma unroll
                for (int j = 0; j < kVec; ++j) {
                    const uint64_t place = place_of(l[j], i0 + v * kVec + j);
                    if (!in_this(l[j], place)) continue;
                    const uint32_t key = static_cast<uint32_t>(place >> 32);
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
                const auto tie = [&](float l, int i) { return static_cast<uint64_t>(moe::order_key(l) == high && place_of(l, i) >= cut); };
                cluster.sync();   // sh.total has been read
                sums(tie);
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

    uint64_t cut = 0;
    const int k = a.top_k ? a.top_k[row] : 0;
    if (k > 0 && k < a.V) cut = cut_at(cut, false, k, 0.0f);
    const float p = a.top_p ? a.top_p[row] : 1.0f;
    if (p < 1.0f) cut = cut_at(cut, true, 0, p);
    float least = -INFINITY;   // min-p: of the logits
    if (a.min_p && a.min_p[row] > 0.0f)
        least = __double2float_ru(static_cast<double>(top) + static_cast<double>(temperature) * log(fmin(static_cast<double>(a.min_p[row]), 1.0)));

    // ---- the draw
    const auto kept = [&](float l, int i) -> uint64_t { return l >= least && place_of(l, i) >= cut ? weight(l) : 0; };
    const uint64_t all = sums(kept);
    const float u = a.u[row];
    const double at = static_cast<double>(u) * static_cast<double>(all);
    uint64_t target = u > 0.0f ? (at < static_cast<double>(all) ? static_cast<uint64_t>(at) : all - 1) : 0;
    if (target >= all) target = all - 1;
    locate(kept, target, [&](float l, int i) {
        a.token[row] = i;
        if (a.logprob)
            a.logprob[row] = static_cast<float>((l == top ? 0.0 : (static_cast<double>(l) - static_cast<double>(top)) / static_cast<double>(temperature)) -
                                                log(static_cast<double>(all) * 0x1p-44));
    });
    cluster.sync();   // no block leaves while another may read its sums
}

template <typename T>
moe_status_t launch(Args a, int rows, cudaStream_t s) {
    static std::atomic<int> allowed[moe::kMaxDevices];
    int dev = 0;
    MOE_CHECK_CUDA(cudaGetDevice(&dev));
    if (dev < 0 || dev >= moe::kMaxDevices) return MOE_ERR_CUDA;
    if (!allowed[dev].load(std::memory_order_relaxed)) {
        MOE_CHECK_CUDA(cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxV / kMaxBlocks * static_cast<int>(sizeof(T))));
        allowed[dev].store(1, std::memory_order_relaxed);
    }
    const int blocks = kMaxBlocks;
    a.slice = ((a.V + blocks - 1) / blocks + 7) / 8 * 8;
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
