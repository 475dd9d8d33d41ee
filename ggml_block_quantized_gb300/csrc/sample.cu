// sample.cu - the next token of each row of logits (include/qstep.h, qsample).
//
// A row is read once into the shared memory of a cluster of thread blocks (one
// block, or up to 16 for long rows and few of them), each holding a contiguous
// slice, a thread eight logits of each 4096. What follows are passes over that
// memory:
//  * the largest logit m;
//  * with top_k, the threads' own largest logits, a histogram of which gives a cut
//    that k tokens reach, and few others; with min_p alone its weight is the cut.
//    The tokens above it are sent to the row's first block, which goes on alone.
//  * With a large top_k, or top_p alone, a histogram of m - l (with top_p: and of
//    what the tokens of a bin weigh less than its first would, in 16 bits) gives
//    the bins in which the border lies, one or two. Their tokens go to the first
//    block, which finds the last one kept by the sum of the weights before them.
//  * Then, as without filters, the token at which the sum of the kept weights, in
//    index order, passes its target: sums of 256 tokens each, then these one by one.
// The first block compares up to kList tokens with each other, all pairs at once.
// More of them, and rows whose border's bins hold too many (equal logits, as a
// rule) or whose top_p follows a large top_k, are searched: for each filter a
// histogram's bin in which the count or the weights' sum passes its target, that
// bin divided again by the bits of the logit until kList tokens are left, or until
// all in it are equal and their border is found by index.
//
// Weights are 64-bit integers in units of 2^-44 of the largest. So sums, the
// histogram's atomic ones among them, depend on no order, every pass agrees with
// every other, and a border is off by the weights' own roundings alone, 2^-35 of a
// sum and half a unit a token: with 32-bit sums a token in some thousands would
// differ from the one that 64 bits give, since with 10^5 tokens that many borders
// share the unit interval. 2^x for them takes
// an argument in two floats, a table of 64 powers and a polynomial of degree 5, two
// logits at a time in packed instructions, 27 a logit. 256 rows of 130001 logits in
// f16 take 96 us without filters, 51 with a top_k of 40, 223 with a top_p of 0.9,
// 133 with settings of their own, where issue slots are 55% used and warps wait for
// each other at the passes' barriers first. One row of 32000 in f32 takes 7.2, 8.0
// and 19.1: there it is one chain of loads, joins of the cluster and sums.
#include <cooperative_groups.h>

#include <algorithm>
#include <array>
#include <atomic>
#include <cfloat>
#include <cmath>

#include "packed.cuh"
#include "step_kernels.cuh"

namespace cg = cooperative_groups;

namespace qg {

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kSet = 8;          // neighbouring logits of a thread
constexpr int kRowSets = kThreads, kSegment = 32 * kSet;  // sets, one a thread, that follow each other; logits of a warp there
constexpr int kBins = 1024;
constexpr int kCap = 2048;       // tokens that go to one block (16 KB of its memory)
constexpr int kList = 128;       // tokens that are compared with each other
constexpr int kMaxCluster = 16;
constexpr int kUnit = 44;        // weights are in units of 2^-44
constexpr uint64_t kOne = 1ull << kUnit;
constexpr float kLeastTemperature = 0x1p-60f;
constexpr float kRange = 64.0f;  // of m - l that the first histogram tells apart
constexpr float kLog2E = 1.44269502162933349609375f, kLog2ERest = 1.925963033500e-8f;

struct Settings {
    float t, u, top_p, min_p;
    int top_k, row;
};

struct Shared {
    float2 power[64];                 // 2^(i / 64) in two floats
    uint64_t sum[kBins];              // of a histogram: weights, and tokens
    uint32_t count[kBins];
    uint64_t all[kCap];               // tokens sent to the first block: (key, ~index)
    uint64_t list[kList], near[kList], weight[kList];  // of a bin's tokens: this block's, the cluster's, their weights
    uint64_t ahead[kList];            // weights before a token, and how many tokens
    uint32_t rank[kList];
    uint64_t segment[2 * kThreads];   // kept weights of kSegment logits
    alignas(16) uint64_t warp_sum[kWarps], warp_most[kWarps], warp_least[kWarps];
    alignas(16) uint32_t warp_count[kWarps];
    struct { uint32_t lo, above, hi, up_to; } range;
    alignas(16) uint4 told;
    uint64_t block_sum[2][kMaxCluster][2];
    float2 extremes[kWarps];
    float2 block_extremes[kMaxCluster];
    alignas(16) uint32_t kinds[kWarps];  // of rows: how many a warp has
    Settings settings;
    uint32_t list_count;
    uint64_t total;
    struct { uint64_t before, value; uint32_t place, count; } found;
};

struct Border {  // the last token kept
    uint32_t key;
    uint32_t index;
};

// Order of the logits as unsigned numbers, and back.
__device__ __forceinline__ uint32_t key_of(float l) {
    const uint32_t u = __float_as_uint(l);
    return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float logit_of(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}
// Eight logits as they are kept: NaN, which is never chosen, as -inf, and -0 as 0; their extremes go on (low of what is
// not -inf: x + (x - x) is NaN there, which a minimum passes over).
struct Extremes32 {
    float top = -INFINITY, low = INFINITY;
    __device__ __forceinline__ void take(float4 (&v)[2]) {
        float *x = reinterpret_cast<float *>(v);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[i] = fmaxf(x[i], -INFINITY) + 0.0f;
            top = fmaxf(top, x[i]);
            low = fminf(low, x[i] + (x[i] - x[i]));
        }
    }
    __device__ __forceinline__ float2 get() const { return make_float2(top, low); }
};
struct Extremes16 {
    __half2 top = __half2half2(__ushort_as_half(0xFC00u)), low = __half2half2(__ushort_as_half(0x7C00u));
    __device__ __forceinline__ void take(uint4 (&v)[1]) {
        __half2 *x = reinterpret_cast<__half2 *>(v);
        const __half2 none = __half2half2(__ushort_as_half(0xFC00u)), zero = __half2half2(__ushort_as_half(0));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = __hadd2(__hmax2(x[i], none), zero);
            top = __hmax2(top, x[i]);
            low = __hmin2(low, __hadd2(x[i], __hsub2(x[i], x[i])));
        }
    }
    __device__ __forceinline__ float2 get() const {
        const float2 a = __half22float2(top), b = __half22float2(low);
        return make_float2(fmaxf(a.x, a.y), fminf(b.x, b.y));
    }
};
template <class T> struct Eight;
template <> struct Eight<float> {
    float4 v[2];
    using Extremes = Extremes32;
    __device__ __forceinline__ float2 pair(int i) const { return i & 1 ? make_float2(v[i >> 1].z, v[i >> 1].w) : make_float2(v[i >> 1].x, v[i >> 1].y); }
    __device__ __forceinline__ float2 next() {  // the first pair; the others move up
        const float2 l = make_float2(v[0].x, v[0].y);
        v[0] = make_float4(v[0].z, v[0].w, v[1].x, v[1].y), v[1].x = v[1].z, v[1].y = v[1].w;
        return l;
    }
};
template <> struct Eight<__half> {
    uint4 v[1];
    using Extremes = Extremes16;
    __device__ __forceinline__ float2 pair(int i) const {
        const uint32_t w = i == 0 ? v[0].x : i == 1 ? v[0].y : i == 2 ? v[0].z : v[0].w;
        return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    }
    __device__ __forceinline__ float2 next() {
        const float2 l = pair(0);
        v[0].x = v[0].y, v[0].y = v[0].z, v[0].z = v[0].w;
        return l;
    }
};

// exp((l - m) / T) but for a factor near 1 that all of a row's share, in units of 2^-44: 2^x for x = l c - M, c =
// log2(e) / T in two floats and M the multiple of 1/64 next to m c, so that M costs no digits. Where m c is 128 or more,
// l is taken from m first (M = 0): that is exact for all that x leaves a weight.
struct Weigher {
    const float2 *power;
    float m, base, ch, cl, magic, least, all_of_it;

    __device__ __forceinline__ void set(const float2 *table, float top, float t) {
        power = table;
        m = top;
        ch = t == INFINITY ? 0.0f : kLog2E / t;
        cl = t == INFINITY ? 0.0f : (fmaf(-ch, t, kLog2E) + kLog2ERest) / t;
        const float p = m * ch;
        const bool far = !(fabsf(p) < 128.0f);
        base = far ? m : 0.0f;
        const float high = far ? 0.0f : rintf(p * 64.0f) * 0x1p-6f;
        magic = 12582912.0f - 64.0f * high;
        least = m == INFINITY ? INFINITY : high - 46.0f;
        all_of_it = m == INFINITY ? INFINITY : NAN;  // logits of infinity: 1 each, and nothing else
    }
    // The weights of two logits, each high 2^22 + low units; live: whether there is one.
    struct Pair { uint32_t high[2], low[2]; bool live[2]; };
    __device__ __forceinline__ Pair pair(float2 l) const {
        auto both = [](float x) { return make_float2(x, x); };
        const float2 a = fadd2(l, both(-base)), xh = fmul2(a, both(ch));
        const float2 low = ffma2(a, both(cl), ffma2(a, both(ch), fmul2(a, both(-ch))));  // 2^-17 at most
        // x = k / 64 + r + low, |r| <= 2^-7: r exact
        const float2 km = ffma2(xh, both(64.0f), both(magic));
        const float2 r = ffma2(fadd2(km, both(-magic)), both(-0x1p-6f), xh);
        // 2^(r + low) - 1 = u + rest, u = r ln 2 rounded (low's square, 2^-36 at most, is left out)
        const float ln2 = 0.693147182464599609375f, ln2_rest = -1.904654323148236e-9f;
        const float2 u = fmul2(r, both(ln2)), low_ln2 = fmul2(low, both(ln2)), minus_u = fmul2(r, both(-ln2)), r2 = fmul2(r, r);
        const float2 p = ffma2(r, ffma2(r, ffma2(r, both(1.3333558146e-3f), both(9.6181291076e-3f)), both(5.5504108665e-2f)), both(2.4022650696e-1f));
        const float2 u_rest = fadd2(ffma2(r, both(ln2_rest), ffma2(r, both(ln2), minus_u)), low_ln2);
        const float2 rest = ffma2(r2, p, ffma2(low_ln2, ffma2(r2, p, u), u_rest));
        // times 2^(k / 64) = t + t_low, the product by t in two parts (the exponent: k / 64's whole part, added to 1's)
        const uint32_t k0 = __float_as_uint(km.x), k1 = __float_as_uint(km.y);
        const float2 t0 = power[k0 & 63], t1 = power[k1 & 63];
        const float2 scale = make_float2(__uint_as_float(((k0 & ~63u) << 17) + 0x3F800000u), __uint_as_float(((k1 & ~63u) << 17) + 0x3F800000u));
        const float2 t = fmul2(make_float2(t0.x, t1.x), scale), t_low = fmul2(make_float2(t0.y, t1.y), scale);
        const float2 v = fmul2(t, u), v_low = fadd2(ffma2(t, u, fmul2(t, minus_u)), ffma2(t, rest, ffma2(t_low, u, t_low)));
        // to whole numbers, by additions that leave them in the last bits
        const float whole = 8388608.0f, half = 12582912.0f;
        const float2 h = ffma2(fadd2(t, fadd2(v, v_low)), both(0x1p22f), both(whole));
        const float2 left = fadd2(fadd2(ffma2(fadd2(h, both(-whole)), both(-0x1p-22f), t), v), v_low);
        const float2 g = ffma2(left, both(0x1p44f), both(half));
        return Pair{{__float_as_uint(h.x) - 0x4B000000u, __float_as_uint(h.y) - 0x4B000000u},
                    {__float_as_uint(g.x) - 0x4B400000u, __float_as_uint(g.y) - 0x4B400000u},
                    {xh.x > least, xh.y > least}};  // (not of -inf)
    }
    __device__ __forceinline__ static uint64_t weight(uint32_t high, uint32_t low) {
        return (static_cast<uint64_t>(high) << 22) + static_cast<int64_t>(static_cast<int32_t>(low));
    }
    __device__ __forceinline__ uint64_t operator()(float l) const {
        if (l == all_of_it) return kOne;
        const Pair w = pair(make_float2(l, l));
        return w.live[0] ? weight(w.high[0], w.low[0]) : 0;
    }
};

// The place in a histogram of m - l, and its bin (NaN, of two infinities: 0).
__device__ __forceinline__ float place_in_bins(float l, float m, float scale) { return fminf(fmaxf((m - l) * scale, 0.0f), kBins - 1.0f); }
__device__ __forceinline__ uint32_t bin_of_place(float x) { return __float_as_uint(__fadd_rz(x, 8388608.0f)) & (kBins - 1u); }
__device__ __forceinline__ uint32_t bin_of(float l, float m, float scale) { return bin_of_place(place_in_bins(l, m, scale)); }

// The least logits whose bins are a or less, and b or less (NaN where b is -1): bins never fall as logits fall, so each half
// of a warp searches the keys, 16 at a time.
__device__ __forceinline__ void least_of_bins(uint32_t a, uint32_t b, float m, float scale, float &of_a, float &of_b) {
    const uint32_t half = threadIdx.x >> 4 & 1u, k = threadIdx.x & 15u, bin = half ? b + (b == ~0u) : a;
    // from the edge's place with a bin and two keys to spare on (m's bin is 0)
    uint32_t lo = key_of(-INFINITY), hi = key_of(m);
    if (m < INFINITY) {
        if (bin + 1 < kBins) lo = max(lo, key_of(m - (bin + 2) / scale) - 2u);
        hi = min(hi, max(lo, key_of(m - bin / scale) + 2u));
    }
#pragma unroll 1
    while (__any_sync(0xffffffffu, lo != hi)) {
        const uint32_t step = (hi - lo) / 16u + 1u;
        const uint32_t yes = __ballot_sync(0xffffffffu, bin_of(logit_of(min(lo + k * step, hi)), m, scale) <= bin) >> (16u * half) & 0xFFFFu;
        const uint32_t first = yes ? __ffs(yes) - 1u : 16u;
        if (first == 0) hi = lo;
        else {
            if (first < 16) hi = min(lo + first * step, hi);
            lo += (first - 1) * step + 1;
        }
    }
    of_a = logit_of(__shfl_sync(0xffffffffu, lo, 0));
    of_b = b == ~0u ? NAN : logit_of(__shfl_sync(0xffffffffu, lo, 16));
}
__device__ __forceinline__ void add_if(bool yes, uint32_t shared, uint32_t v) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %0, 0;\n\t@p red.shared.add.u32 [%1], %2;\n\t}" ::"r"(static_cast<uint32_t>(yes)), "r"(shared), "r"(v) : "memory");
}

// floor(v f) for 0 <= f <= 1, exact, and whether it was cut off.
__device__ __forceinline__ uint64_t times(uint64_t v, float f, bool &rest) {
    const uint32_t bits = __float_as_uint(f), e = bits >> 23;  // f = mantissa 2^(e - 150); below 2^-126: 0
    rest = false;
    if (e == 0) return 0;
    const uint64_t mantissa = (bits & 0x7FFFFFu) | 0x800000u, low = v * mantissa, high = __umul64hi(v, mantissa);
    const uint32_t down = 150 - e;  // 23 at least
    if (down >= 128) return 0;
    if (down >= 64) {
        rest = low != 0 || (down > 64 && (high << (128 - down)) != 0);
        return high >> (down - 64);
    }
    rest = (low << (64 - down)) != 0;
    return high << (64 - down) | low >> down;
}

__device__ __forceinline__ uint64_t warp_total(uint64_t v) {
#pragma unroll
    for (int m = 16; m; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}
__device__ __forceinline__ uint64_t warp_prefix(uint64_t v) {  // inclusive
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const uint64_t o = __shfl_up_sync(0xffffffffu, v, m);
        if ((threadIdx.x & 31) >= m) v += o;
    }
    return v;
}

// Values of the warps: the sum of all, and of those before `warp`, added to `before`. (Every warp reads them: 16 bytes at a
// time, the fewest instructions.)
__device__ __forceinline__ void add_up(const uint64_t *of_warps, int warp, uint64_t &before, uint64_t &all) {
    all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; w += 2) {
        const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(of_warps + w);
        if (w < warp) before += v.x;
        if (w + 1 < warp) before += v.y;
        all += v.x + v.y;
    }
}
__device__ __forceinline__ void add_up(const uint32_t *of_warps, int warp, uint32_t &before, uint32_t &all) {
    all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; w += 4) {
        const uint4 v = *reinterpret_cast<const uint4 *>(of_warps + w);
        if (w < warp) before += v.x;
        if (w + 1 < warp) before += v.y;
        if (w + 2 < warp) before += v.z;
        if (w + 3 < warp) before += v.w;
        all += v.x + v.y + v.z + v.w;
    }
}

struct Target {  // of a sum's share
    __device__ static __forceinline__ uint64_t share(uint64_t all, float p) {  // the least that is not below it, 1 or more
        bool rest;
        const uint64_t t = times(all, p, rest);
        return t + (rest || t == 0 ? 1 : 0);
    }
    __device__ static __forceinline__ uint64_t draw(uint64_t all, float u) {  // the first that passes u of it
        bool rest;
        const uint64_t x = u > 0.0f ? times(all, fminf(u, 1.0f), rest) : 0;
        return x >= all ? all : x + 1;
    }
};

// Tokens that are searched: a row in the cluster's shared memory, a contiguous slice a block ...
template <class T> struct RowTokens {
    static constexpr bool kSent = false;
    Shared *s;
    const T *data;             // this block's slice: sets of kSet, what lies before and behind it in the first and last is -inf
    int first, sets;           // the index of the first set's first place; sets
    int rank, blocks;
    using Type = T;
    __device__ __forceinline__ Eight<T> set(int i) const { return *reinterpret_cast<const Eight<T> *>(data + kSet * i); }
    template <class F> __device__ __forceinline__ void each(F f) const {  // f(logit, index)
        for (int i = threadIdx.x; i < sets; i += kRowSets) {
#pragma unroll 2
            for (int j = kSet * i; j < kSet * i + kSet; ++j) f(static_cast<float>(data[j]), first + j);
        }
    }
};
// ... or those sent to the first block, n in any order, by that block alone.
struct SentTokens {
    static constexpr bool kSent = true;
    static constexpr int first = 0, rank = 0, blocks = 1;
    Shared *s;
    int n, index_bits;         // log2 of the indexes that share a bin
    template <class F> __device__ __forceinline__ void each(F f) const {
        for (int i = threadIdx.x; i < n; i += kThreads) {
            const uint64_t e = s->all[i];
            f(logit_of(static_cast<uint32_t>(e >> 32)), static_cast<int>(~static_cast<uint32_t>(e)));
        }
    }
};

template <class Tokens> struct Search : Tokens {
    using Tokens::s, Tokens::first, Tokens::rank, Tokens::blocks, Tokens::each;
    int turn = 0;              // which of the two sums' places is next

    __device__ __forceinline__ void join() const {  // the whole cluster
        if (blocks == 1) __syncthreads();
        else cg::this_cluster().sync();
    }
    template <class P> __device__ __forceinline__ P *at(P *p, int block) const {
        return blocks == 1 ? p : cg::this_cluster().map_shared_rank(p, block);
    }
    // Sums over the blocks before this one, over this one, and over all; of a second thing over all (~0: none).
    struct Sums { uint64_t before, mine, all, all2; };
    __device__ __forceinline__ Sums sums(uint64_t v, uint64_t v2) {
        const uint64_t block2 = v2 == ~0ull ? 0 : block_total(v2);
        uint64_t none = 0, block;
        v = warp_total(v);
        __syncthreads();
        if ((threadIdx.x & 31) == 0) s->warp_sum[threadIdx.x >> 5] = v;
        __syncthreads();
        add_up(s->warp_sum, 0, none, block);
        uint64_t (*const place)[2] = s->block_sum[turn];
        turn ^= 1;
        if (threadIdx.x < blocks) {
            uint64_t *const there = at(&place[rank][0], threadIdx.x);
            there[0] = block, there[1] = block2;
        }
        join();
        Sums r{0, block, 0, 0};
        for (int b = 0; b < blocks; ++b) {
            if (b < rank) r.before += place[b][0];
            r.all += place[b][0], r.all2 += place[b][1];
        }
        return r;
    }
    __device__ __forceinline__ uint64_t block_total(uint64_t v) {  // over this block's threads
        v = warp_total(v);
        __syncthreads();
        if ((threadIdx.x & 31) == 0) s->warp_sum[threadIdx.x >> 5] = v;
        __syncthreads();
        uint64_t before = 0, all;
        add_up(s->warp_sum, 0, before, all);
        __syncthreads();
        return all;
    }
    // The token, in index order, at which the sum of value(logit, index) reaches target(sum of all); found.place is its
    // index, found.value its value. Returns the sum of all.
    template <class V, class G> __device__ __forceinline__ uint64_t select(V value, G target) {
        if constexpr (Tokens::kSent) {
            // by histograms of the indexes' high bits, then of the low ones
            const int bits = this->index_bits;
            uint64_t whole = 0, t = 0;
            uint32_t high = 0;
            for (int level = 0; level < 2; ++level) {
                __syncthreads();
                clear_bins();
                __syncthreads();
                each([&](float l, int i) {
                    const uint64_t v = level == 1 && static_cast<uint32_t>(i) >> bits != high ? 0 : value(l, i);
                    if (v != 0) atomicAdd(reinterpret_cast<unsigned long long *>(&s->sum[level == 0 ? i >> bits : i & ((1 << bits) - 1)]), static_cast<unsigned long long>(v));
                });
                __syncthreads();
                const uint64_t v[2] = {s->sum[2 * threadIdx.x], s->sum[2 * threadIdx.x + 1]};
                const uint32_t n[2] = {0, 0};
                if (level == 0) {
                    whole = block_total(v[0] + v[1]);
                    t = target(whole);
                }
                find_bin(v, n, false, t);
                __syncthreads();
                if (level == 0) high = s->found.place, t -= s->found.before;
            }
            __syncthreads();
            if (threadIdx.x == 0) s->found.value = s->sum[s->found.place], s->found.place += high << bits;
            __syncthreads();
            return whole;
        } else {
            for_segments([&](int i) {
                uint64_t sum = 0;
                const Eight<typename Tokens::Type> e = this->set(i);
#pragma unroll
                for (int j = 0; j < kSet; ++j) sum += value(j & 1 ? e.pair(j >> 1).y : e.pair(j >> 1).x, first + kSet * i + j);
                return sum;
            });
            return choose_segment(value, target);
        }
    }
    // f(set) of each set of this block, summed up by segments.
    template <class F> __device__ __forceinline__ void for_segments(F f) {
        int place = threadIdx.x >> 5;
        for (int i0 = 0; i0 < this->sets; i0 += kRowSets, place += kWarps) {
            const int i = i0 + threadIdx.x;
            const uint64_t sum = warp_total(i < this->sets ? f(i) : 0);
            if ((threadIdx.x & 31) == 0) s->segment[place] = sum;
        }
    }
    // select, once the segments' sums are there.
    template <class V, class G> __device__ __forceinline__ uint64_t choose_segment(V value, G target) {
        __syncthreads();
        const int segments = (this->sets + kRowSets - 1) / kRowSets * kWarps;
        uint64_t v[2];
        const uint32_t n[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < 2; ++i) v[i] = 2 * threadIdx.x + i < segments ? s->segment[2 * threadIdx.x + i] : 0;
        const Sums r = sums(v[0] + v[1], ~0ull);
        const uint64_t t = target(r.all);
        if (r.before < t && t <= r.before + r.mine) {  // in this block
            find_bin(v, n, false, t - r.before);
            __syncthreads();
            const int from = s->found.place * kSegment;
            const uint64_t before = s->found.before;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int j = from + 2 * threadIdx.x + i;
                v[i] = 2 * threadIdx.x + i < kSegment && j < kSet * this->sets ? value(static_cast<float>(this->data[j]), first + j) : 0;
            }
            find_bin(v, n, false, t - r.before - before);
            __syncthreads();
            const uint32_t place = s->found.place;
            if (threadIdx.x == place >> 1)
                for (int b = 0; b < blocks; ++b) {
                    auto *f = at(&s->found, b);
                    f->value = place & 1 ? v[1] : v[0], f->place = first + from + place;
                }
        }
        join();
        return r.all;
    }
    __device__ __forceinline__ void clear_bins() {
        for (int b = threadIdx.x; b < kBins; b += kThreads) s->sum[b] = 0, s->count[b] = 0;
    }
    // The cluster's counts (sums) of this thread's two bins: up to eight blocks' on their way at once.
    template <class P> __device__ __forceinline__ void gather(uint64_t (&v)[2], const P *p) const {
        v[0] = v[1] = 0;
        for (int b0 = 0; b0 < blocks; b0 += 8) {
            P c[8][2];
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                c[q][0] = c[q][1] = 0;
                if (b0 + q < blocks) {
                    const P *there = at(p, b0 + q) + 2 * threadIdx.x;
                    if constexpr (sizeof(P) == 4) {
                        const uint2 x = *reinterpret_cast<const uint2 *>(there);
                        c[q][0] = x.x, c[q][1] = x.y;
                    } else {
                        const ulonglong2 x = *reinterpret_cast<const ulonglong2 *>(there);
                        c[q][0] = x.x, c[q][1] = x.y;
                    }
                }
            }
#pragma unroll
            for (int q = 0; q < 8; ++q) v[0] += c[q][0], v[1] += c[q][1];
        }
    }
    __device__ __forceinline__ void bin_counts(uint32_t (&n)[2]) const {
        uint64_t v[2];
        gather(v, s->count);
        n[0] = static_cast<uint32_t>(v[0]), n[1] = static_cast<uint32_t>(v[1]);
    }
    __device__ __forceinline__ void bin_sums(uint64_t (&v)[2]) const { gather(v, s->sum); }
    // Bins of a histogram, each thread two neighbours, `rising`: counted from the last one: where the running sum of v
    // reaches `target`; found: the bin, the sum before it, and its n (left as it was where the sum does not). Every
    // thread of every block calls it, with a barrier before found is read.
    __device__ __forceinline__ void find_bin(const uint64_t (&v)[2], const uint32_t (&n)[2], bool rising, uint64_t target) {
        const uint64_t both = v[0] + v[1], up_to = warp_prefix(both);
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        if (lane == 31) s->warp_sum[warp] = up_to;
        __syncthreads();
        uint64_t before = up_to - both, whole;
        add_up(s->warp_sum, warp, before, whole);
        if (rising) before = whole - before - both;
#pragma unroll
        for (int i = 0; i < 2; ++i) {  // (no array by a variable: with all of shared memory taken, local memory is L2's)
            const bool b = rising ? i == 0 : i == 1;
            const uint64_t x = b ? v[1] : v[0];
            if (before < target && target <= before + x) s->found.place = 2 * threadIdx.x + b, s->found.before = before, s->found.count = b ? n[1] : n[0];
            before += x;
        }
    }
    // Tokens from logit `least` on (not -inf) for which take(logit) holds are sent to the first block, as far as there is room.
    template <class F> __device__ __forceinline__ void send(float least, F take) {
        uint64_t *const there = at(s->all, 0);
        uint32_t *const counter = at(&s->list_count, 0);
        for (int i = threadIdx.x; i < this->sets; i += kRowSets) {
            const Eight<typename Tokens::Type> e = this->set(i);
            float most = -INFINITY;
#pragma unroll
            for (int j = 0; j < kSet / 2; ++j) most = fmaxf(fmaxf(most, e.pair(j).x), e.pair(j).y);
            if (!(most >= least) || most == -INFINITY) continue;
            uint32_t who = 0;
#pragma unroll
            for (int j = 0; j < kSet; ++j) {
                const float l = j & 1 ? e.pair(j >> 1).y : e.pair(j >> 1).x;
                if (l >= least && l > -INFINITY && take(l)) who |= 1u << j;
            }
            if (who == 0) continue;
            uint32_t place = atomicAdd(counter, static_cast<uint32_t>(__popc(who)));
#pragma unroll
            for (int j = 0; j < kSet; ++j)
                if (who >> j & 1) {
                    if (place < kCap)
                        there[place] = static_cast<uint64_t>(key_of(j & 1 ? e.pair(j >> 1).y : e.pair(j >> 1).x)) << 32 | ~static_cast<uint32_t>(first + kSet * i + j);
                    ++place;
                }
        }
    }
    // The border at which the running value (1, or the weight) over the tokens up to `limit`, in falling order,
    // reaches `target` (at least 1, at most the sum of all). The first bins are of m - l, `scale` a unit; with weights,
    // tokens of `reach` and less are known to lie behind it.
    template <bool WEIGHTS, class W>
    __device__ __forceinline__ Border border(Border limit, uint64_t target, float m, float scale, float reach, W weigh) {
        uint32_t lo = 0, hi = 0, bin0 = 0;
        int shift = -1;  // -1: the first histogram, of m - l
        auto member = [&](float l, int i, uint32_t &bin) {
            const uint32_t key = key_of(l);
            if (key < limit.key || (key == limit.key && static_cast<uint32_t>(i) > limit.index)) return false;
            bin = bin_of(l, m, scale);
            if (shift < 0) return true;
            if (bin != bin0 || key < lo || key > hi) return false;
            bin = (key - lo) >> shift;
            return true;
        };
        for (;;) {
            __syncthreads();
            clear_bins();
            if (threadIdx.x == 0) s->list_count = 0;
            __syncthreads();
            each([&](float l, int i) {
                uint32_t bin;
                if (WEIGHTS && !(l > reach)) return;
                if (!member(l, i, bin)) return;
                atomicAdd(&s->count[bin], 1u);
                if (WEIGHTS) atomicAdd(reinterpret_cast<unsigned long long *>(&s->sum[bin]), static_cast<unsigned long long>(weigh(l)));
            });
            join();
            uint64_t v[2];
            uint32_t n[2];
            bin_counts(n);
            if (WEIGHTS) bin_sums(v);
            else v[0] = n[0], v[1] = n[1];
            // bins of the first histogram fall with the logit, those of the others rise
            find_bin(v, n, shift >= 0, target);
            join();  // (the histograms have been read, too)
            const uint32_t bin = s->found.place, in_bin = s->found.count;
            target -= s->found.before;
            if (shift < 0) {
                bin0 = bin;
                lo = bin == kBins - 1 ? 0u : key_of(m - (bin + 2) / scale);
                hi = key_of(bin == 0 ? INFINITY : m - (bin - 1) / scale);
            } else {
                lo += bin << shift;
                const uint32_t top = lo + ((1u << shift) - 1u);
                hi = top < lo || top > hi ? hi : top;
            }
            const uint32_t width = hi - lo;
            shift = width < kBins ? 0 : 22 - __clz(width);
            if (in_bin <= kList) break;
            if (lo == hi) {  // so many equal ones: the border is found by index
                const uint64_t each_one = WEIGHTS ? weigh(logit_of(lo)) : 1, nth = (target + each_one - 1) / each_one;
                __syncthreads();
                select([&](float x, int i) -> uint64_t { return key_of(x) == lo && (lo != limit.key || static_cast<uint32_t>(i) <= limit.index); },
                       [&](uint64_t) { return nth; });
                return Border{lo, s->found.place};
            }
        }
        // the few tokens left, compared with each other by every block
        each([&](float l, int i) {
            uint32_t bin;
            if (WEIGHTS && !(l > reach)) return;
            if (!member(l, i, bin)) return;
            s->list[atomicAdd(&s->list_count, 1u)] = static_cast<uint64_t>(key_of(l)) << 32 | ~static_cast<uint32_t>(i);
        });
        join();
        int n = 0;
        for (int b = 0; b < blocks; ++b) {
            const int m = static_cast<int>(*at(&s->list_count, b));
            if (static_cast<int>(threadIdx.x) < m) s->near[n + threadIdx.x] = at(s->list, b)[threadIdx.x];
            n += m;
        }
        compare(s, n, [&](uint64_t e) -> uint64_t { return WEIGHTS ? weigh(logit_of(static_cast<uint32_t>(e >> 32))) : 1; },
                [](uint64_t a, uint64_t b) { return a > b; });
        if (threadIdx.x < n && s->ahead[threadIdx.x] < target && target <= s->ahead[threadIdx.x] + s->weight[threadIdx.x])
            s->found.value = s->near[threadIdx.x];
        join();
        const uint64_t e = s->found.value;
        return Border{static_cast<uint32_t>(e >> 32), ~static_cast<uint32_t>(e)};
    }
    // For each of s->near's first n tokens (kList at most), all pairs at once: its weight, how many of the others come
    // before it, and what those weigh.
    template <class W, class L> __device__ static __forceinline__ void compare(Shared *s, int n, W weight, L before) {
        int n2 = 16;
        while (n2 < n) n2 *= 2;
        if (threadIdx.x < kList) s->ahead[threadIdx.x] = 0, s->rank[threadIdx.x] = 0;
        __syncthreads();
        if (threadIdx.x < n) s->weight[threadIdx.x] = weight(s->near[threadIdx.x]);
        __syncthreads();
        const int i = threadIdx.x & (n2 - 1), per = n2 * n2 / kThreads + (n2 * n2 < kThreads), j0 = threadIdx.x / n2 * per;
        if (i < n) {
            const uint64_t e = s->near[i];
            uint64_t sum = 0;
            uint32_t many = 0;
            for (int j = j0; j < min(j0 + per, n); ++j)
                if (before(s->near[j], e)) sum += s->weight[j], ++many;
            if (many > 0) {
                atomicAdd(&s->rank[i], many);
                atomicAdd(reinterpret_cast<unsigned long long *>(&s->ahead[i]), static_cast<unsigned long long>(sum));
            }
        }
        __syncthreads();
    }
};

// The weights' sum of a set (no logit of infinity).
template <class T> __device__ __forceinline__ uint64_t weigh_set(Eight<T> e, const Weigher &weigh) {
    uint32_t high = 0, low = 0;
#pragma unroll 2
    for (int j = 0; j < kSet / 2; ++j) {
        const Weigher::Pair w = weigh.pair(e.next());
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (w.live[i]) high += w.high[i], low += w.low[i];
    }
    return Weigher::weight(high, low);
}

enum Todo { kNothing, kSelect, kTopP, kAll };

// The filters that `todo` leaves open, by a search each, and the token.
struct Chosen { int32_t token; float prob; };
template <class Tokens>
__device__ __forceinline__ Chosen search_all(Search<Tokens> &search, int todo, Border last, int top_k, float top_p, float min_p, float u,
                                             float t, int vocab, float m, float scale, const Weigher &weigh) {
    auto kept = [&](float l, int i) {
        if (last.key == 0) return true;
        const uint32_t key = key_of(l);
        return key > last.key || (key == last.key && static_cast<uint32_t>(i) <= last.index);
    };
    if (todo == kAll && top_k > 0) last = search.template border<false>(last, top_k, m, scale, 0.0f, weigh);
    if (todo != kSelect && top_p < 1.0f) {
        uint64_t mine = 0;
        search.each([&](float l, int i) {
            if (kept(l, i)) mine += weigh(l);
        });
        const uint64_t all = search.sums(mine, ~0ull).all;
        // Weights below (1 - top_p) / vocab of the sum are all past the border: their sum is less than what is cut.
        const float least = (1.0f - top_p) * (static_cast<float>(all) * (1.0f / kOne)) / static_cast<float>(vocab);
        const float reach = weigh.m == INFINITY ? 0.0f : weigh.m + (log2f(least) - 0.02f) * t * 0.694f - 1e-6f * fabsf(weigh.m);
        last = search.template border<true>(last, Target::share(all, top_p), m, scale, reach, weigh);
    }
    const uint64_t light = min_p > 0.0f ? Target::share(weigh(weigh.m), min_p) : 0;
    auto value = [&](float l, int i) -> uint64_t {
        if (!kept(l, i)) return 0;
        const uint64_t w = weigh(l);
        return w >= light ? w : 0;
    };
    auto target = [&](uint64_t all) { return Target::draw(all, u); };
    uint64_t all;
    if constexpr (!Tokens::kSent) {
        if (last.key == 0 && light == 0 && weigh.m < INFINITY) {  // all of them: the weights two by two
            search.for_segments([&](int i) { return weigh_set(search.set(i), weigh); });
            all = search.choose_segment(value, target);
        } else {
            all = search.select(value, target);
        }
    } else {
        all = search.select(value, target);
    }
    return Chosen{static_cast<int32_t>(search.s->found.place), static_cast<float>(search.s->found.value) / static_cast<float>(all)};
}

// The first block's n tokens, all that may be kept, and the filters: the token.
__device__ __forceinline__ Chosen choose_sent(Shared *s, int n, int index_bits, int top_k, float top_p, float min_p, float u, float t,
                                              int vocab, float m, float scale, const Weigher &weigh) {
    using Sent = Search<SentTokens>;
    if (n > kList) {
        Sent sent;
        sent.s = s, sent.n = n, sent.index_bits = index_bits;
        return search_all(sent, kAll, Border{0u, 0xFFFFFFFFu}, top_k > 0 && top_k < n ? top_k : 0, top_p, min_p, u, t, vocab, m, scale, weigh);
    }
    const int i = threadIdx.x;
    if (i < n) s->near[i] = s->all[i];
    if (i == 0) s->total = 0;
    Sent::compare(s, n, [&](uint64_t e) { return weigh(logit_of(static_cast<uint32_t>(e >> 32))); }, [](uint64_t a, uint64_t b) { return a > b; });
    const bool in = i < n && (top_k == 0 || s->rank[i] < static_cast<uint32_t>(top_k));
    uint64_t w = in ? s->weight[i] : 0;
    if (top_p < 1.0f) {
        const uint64_t sum = warp_total(w);
        if ((i & 31) == 0 && sum > 0) atomicAdd(reinterpret_cast<unsigned long long *>(&s->total), static_cast<unsigned long long>(sum));
        __syncthreads();
        if (i < n && s->ahead[i] >= Target::share(s->total, top_p)) w = 0;
    }
    if (min_p > 0.0f && w < Target::share(weigh(weigh.m), min_p)) w = 0;
    __syncthreads();
    if (i == 0) s->total = 0;
    // the kept weights, in the order of the indexes (~index falls)
    Sent::compare(s, n, [&](uint64_t) { return w; }, [](uint64_t a, uint64_t b) { return static_cast<uint32_t>(a) > static_cast<uint32_t>(b); });
    const uint64_t sum = warp_total(w);
    if ((i & 31) == 0 && sum > 0) atomicAdd(reinterpret_cast<unsigned long long *>(&s->total), static_cast<unsigned long long>(sum));
    __syncthreads();
    const uint64_t all = s->total, draw = Target::draw(all, u);
    if (i < n && s->ahead[i] < draw && draw <= s->ahead[i] + w) s->found.place = ~static_cast<uint32_t>(s->near[i]), s->found.value = w;
    __syncthreads();
    return Chosen{static_cast<int32_t>(s->found.place), static_cast<float>(s->found.value) / static_cast<float>(all)};
}

// The first block's n tokens, of the bins in which the border lies: the last one kept, with `target` (a count, or a sum
// of weights) to be reached among them.
template <bool WEIGHTS>
__device__ __forceinline__ Border border_of_sent(Shared *s, int n, int index_bits, uint64_t target, float m, float scale, const Weigher &weigh) {
    Search<SentTokens> sent;
    sent.s = s, sent.n = n, sent.index_bits = index_bits;
    return sent.template border<WEIGHTS>(Border{0u, 0xFFFFFFFFu}, target, m, scale, -INFINITY, weigh);
}

// A row's settings, and what they mean.
__device__ __forceinline__ Settings settings_of(const SampleParams &p, int64_t r) {
    return Settings{p.temperature ? p.temperature[r] : 1.0f, p.uniform[r], p.top_p ? p.top_p[r] : 1.0f, p.min_p ? p.min_p[r] : 0.0f,
                    p.top_k ? p.top_k[r] : 0, static_cast<int>(r)};
}
__device__ __forceinline__ void check(Settings &a, int vocab) {
    if (a.top_k < 0 || a.top_k >= vocab) a.top_k = 0;
    if (!(a.top_p < 1.0f)) a.top_p = 1.0f;  // (NaN: all)
    if (!(a.min_p > 0.0f)) a.min_p = 0.0f;
}
// Those of the row that is i-th by what they cost: first the rows whose logits are gone through twice (top_p without a small
// top_k), then those that weigh all of them, then the others. A row a thread.
__device__ __forceinline__ Settings settings_in_order(const SampleParams &p, Shared *s, int i) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Settings a;
    int place = -1;  // of the row's kind in the order
    if (threadIdx.x < p.n) {
        a = settings_of(p, threadIdx.x);
        check(a, p.vocab);
        const bool few = !(a.t >= kLeastTemperature) || (a.top_k > 0 && a.top_k <= kThreads / 2 * p.blocks);
        place = few ? 2 : a.top_p < 1.0f || a.top_k > 0 ? 0 : a.min_p > 0.0f ? 2 : 1;
    }
    uint32_t mine = 0, many = 0;  // ten bits a kind
#pragma unroll
    for (int c = 0; c < 3; ++c) {
        const uint32_t who = __ballot_sync(0xffffffffu, place == c);
        if (place == c) mine = __popc(who & ((1u << lane) - 1u));
        many |= __popc(who) << 10 * c;
    }
    if (lane == 0) s->kinds[warp] = many;
    __syncthreads();
    uint32_t before = 0, all;
    add_up(s->kinds, warp, before, all);
    const uint32_t at = mine + (place > 0 ? all & 1023u : 0u) + (place > 1 ? all >> 10 & 1023u : 0u) + (before >> 10 * max(place, 0) & 1023u);
    if (place >= 0 && at == static_cast<uint32_t>(i)) s->settings = a;
    __syncthreads();
    return s->settings;
}

// SORTED: the dear rows first.
template <class T, bool SORTED>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleParams p) {
    extern __shared__ __align__(16) uint8_t smem[];
    Shared *const s = reinterpret_cast<Shared *>(smem);
    T *const space = reinterpret_cast<T *>(smem + (sizeof(Shared) + 31) / 32 * 32);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Search<RowTokens<T>> row;
    row.s = s;
    row.blocks = p.blocks;
    row.rank = static_cast<int>(blockIdx.x % p.blocks);
    if (threadIdx.x < 64) s->power[threadIdx.x] = p.power[threadIdx.x];
    if (threadIdx.x == 0) s->list_count = 0;
    row.clear_bins();
    if (p.blocks > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    pdl_allow_dependents();
    pdl_wait_prior_grids();
    const int i_row = static_cast<int>(blockIdx.x / p.blocks);
    Settings a = SORTED ? settings_in_order(p, s, i_row) : settings_of(p, i_row);
    const int64_t r = SORTED ? a.row : i_row;

    // ---- the row, as far from a boundary of eight elements here as there
    const int slice0 = row.rank * p.slice, count = max(0, min(p.vocab - slice0, p.slice));
    const T *const src = static_cast<const T *>(p.logits) + r * p.stride + slice0;
    const int pad = static_cast<int>(reinterpret_cast<uintptr_t>(src) / sizeof(T) & 7u);
    row.data = space;
    row.first = slice0 - pad;
    row.sets = count > 0 ? (pad + count + kSet - 1) / kSet : 0;
    typename Eight<T>::Extremes extremes;
    constexpr int kAhead = sizeof(T) == 4 ? 4 : 8;  // sets that a thread has under way
    for (int i0 = threadIdx.x; i0 < row.sets; i0 += kRowSets * kAhead) {
        Eight<T> e[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int i = kSet * (i0 + kRowSets * k) - pad;
            if (i >= 0 && i + kSet <= count) {
                e[k] = *reinterpret_cast<const Eight<T> *>(src + i);
            } else {
                T *x = reinterpret_cast<T *>(&e[k]);
#pragma unroll
                for (int j = 0; j < kSet; ++j) x[j] = i + j >= 0 && i + j < count ? src[i + j] : static_cast<T>(-INFINITY);
            }
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            extremes.take(e[k].v);
            if (i0 + kRowSets * k < row.sets) *reinterpret_cast<Eight<T> *>(space + kSet * (i0 + kRowSets * k)) = e[k];
        }
    }
    check(a, p.vocab);
    const float t = a.t, u = a.u, top_p = a.top_p, min_p = a.min_p;
    const int top_k = a.top_k;
    float top = extremes.get().x, low = extremes.get().y;
    const float mine_top = top;
#pragma unroll
    for (int m = 16; m; m >>= 1) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
        low = fminf(low, __shfl_xor_sync(0xffffffffu, low, m));
    }
    if (lane == 0) s->extremes[warp] = make_float2(top, low);
    if (p.blocks > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // the others' memory is there
    __syncthreads();
    if (warp == 0) {
        float2 e = s->extremes[lane % kWarps];
#pragma unroll
        for (int m = kWarps / 2; m; m >>= 1) {
            e.x = fmaxf(e.x, __shfl_xor_sync(0xffffffffu, e.x, m));
            e.y = fminf(e.y, __shfl_xor_sync(0xffffffffu, e.y, m));
        }
        if (lane < row.blocks) row.at(s->block_extremes, lane)[row.rank] = e;
    }
    row.join();
    top = -INFINITY, low = INFINITY;
#pragma unroll 4
    for (int b = 0; b < row.blocks; ++b) top = fmaxf(top, s->block_extremes[b].x), low = fminf(low, s->block_extremes[b].y);

    Chosen chosen{-1, 0.0f};
    if (top == -INFINITY) {  // no token
    } else if (!(t >= kLeastTemperature) || top_k == 1 || top_p <= 0.0f || min_p > 1.0f) {  // the first alone
        uint32_t first = 0xFFFFFFFFu;
        if (mine_top == top)
            row.each([&](float l, int i) {
                if (l == top && first == 0xFFFFFFFFu) first = i;
            });
        first = __reduce_min_sync(0xffffffffu, first);
        if (lane == 0 && first != 0xFFFFFFFFu)  // (list_count holds 0 less 1 less the least index so far)
            for (int b = 0; b < row.blocks; ++b) atomicMax(row.at(&s->list_count, b), 0u - 1u - first);
        row.join();
        chosen = Chosen{static_cast<int32_t>(0u - 1u - s->list_count), 1.0f};
    } else {
        Weigher weigh;
        weigh.set(s->power, top, t);
        Border last{0u, 0xFFFFFFFFu};
        int todo = kSelect;  // what is left: the filters (kAll, kTopP), the selection, or nothing
        // bins per unit of m - l, a power of two, over so much
        auto bins_over = [&](float most) { return __uint_as_float(__float_as_uint((kBins - 1) / fminf(fmaxf(top - low, 0x1p-100f), most)) & 0x7F800000u); };
        const bool by_weight = top_k == 0 && top_p < 1.0f;
        const float scale = bins_over(by_weight ? fminf(31.0f * t, FLT_MAX) : kRange);
        const int index_bits = max(0, 22 - __clz(p.vocab - 1));  // of an index, but the highest ten
        if (top_k > 0 ? top_k <= kThreads / 2 * row.blocks : top_p == 1.0f && min_p > 0.0f) {
            // ---- a cut that as many tokens reach, by the threads' own largest (about half as many again where half of the
            // threads have one), or that min_p gives
            uint32_t last_bin = 0;
            if (top_k > 0) {
                if (mine_top > -INFINITY) atomicAdd(&s->count[bin_of(mine_top, top, scale)], 1u);
                if (threadIdx.x == 0) s->found.place = kBins - 1;
                row.join();
                uint32_t n[2];
                row.bin_counts(n);
                const uint64_t count[2] = {n[0], n[1]};
                row.find_bin(count, n, false, static_cast<uint64_t>(top_k));
                __syncthreads();
                last_bin = s->found.place;
            }
            const float reach = top == INFINITY ? 0.0f : top + (log2f(min_p) - 0.02f) * t * 0.694f - 1e-6f * fabsf(top);  // (of min_p alone)
            // (the bins are half open, and their ends and places rounded: a little more is sent)
            const float cut = top_k == 0 ? reach : last_bin == kBins - 1 || top == INFINITY ? -INFINITY : top - (last_bin + 1.01f) / scale - 1e-6f * fabsf(top);
            row.send(cut, [](float) { return true; });
            row.join();
            const uint32_t n = *row.at(&s->list_count, 0);
            if (n <= kCap) {  // the first block goes on alone, in its own memory, and stays until the others have read it
                todo = kNothing;
                if (p.blocks > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
                if (row.rank == 0) chosen = choose_sent(s, n, index_bits, top_k, top_p, min_p, u, t, p.vocab, top, scale, weigh);
                if (p.blocks > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
            } else if (top_k > 0) {
                todo = kAll;
            }
        } else if (top_k > 0 || by_weight) {
            todo = kAll;
        }
        if (todo == kAll) {
            // ---- the bins in which the border lies
            row.join();  // (the memory is used again)
            row.clear_bins();
            if (threadIdx.x == 0) s->list_count = 0, s->found.place = kBins - 1, s->found.count = ~0u;
            row.join();
            // s->sum: what a bin's tokens weigh less than its first possible one, in 2^-16 of that, in 32 bits (atomics of 64
            // are loops: 292 us instead of 219 with the count in the high bits, 256 rows of 130001, top_p 0.5). Tokens of
            // -inf are in no bin: with 64 rows, some of them masked, their one bin's atomics took half of the time.
            const float per_bin = weigh.ch / scale;  // log2 of the weights' ratio over a bin, 0.1 at most
            const uint32_t counts = smem_addr(s->count), less_at = smem_addr(s->sum);
            for (int i = threadIdx.x; i < row.sets; i += kRowSets) {
                Eight<T> e = row.set(i);
#pragma unroll 2
                for (int j = 0; j < kSet / 2; ++j) {
                    const float2 l2 = e.next();
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const float l = q ? l2.y : l2.x, x = place_in_bins(l, top, scale), up = __fadd_rz(x, 8388608.0f);
                        const uint32_t b = __float_as_uint(up) & (kBins - 1u);
                        add_if(l > -INFINITY, counts + 4 * b, 1u);
                        if (by_weight) {
                            float y;
                            asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"((x - (up - 8388608.0f)) * -per_bin));
                            add_if(l > -INFINITY && b + 1 < kBins, less_at + 8 * b, __float_as_uint(fmaf(1.0f - y, 65536.0f, 12582912.0f)) - 0x4B400000u);
                        }
                    }
                }
            }
            row.join();
            uint32_t bin_lo = 0, bin_hi = 0, above = 0, in = 0;  // the bins, and the tokens in those before them, and in them
            if (row.rank == 0) {  // (the others reading the histograms, too, took longer than they wait so)
                uint32_t n[2];
                row.bin_counts(n);
                if (by_weight) {
                    // what the bins weigh at most and at least, off by 2^-15 in all: half a unit of 2^-16 for each token and
                    // the steps to it; of the last bin's tokens only the upper bound is known
                    uint64_t less[2], most[2], least[2];
                    row.bin_sums(less);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int b = 2 * threadIdx.x + i;
                        float y;
                        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(-b * per_bin));
                        y *= static_cast<float>(n[i]) - static_cast<float>(less[i]) * 0x1p-16f;
                        if (top == INFINITY) y = b == 0 ? static_cast<float>(n[i]) : 0.0f;
                        most[i] = __float2ull_rn(y * (1.0f + 0x1p-15f) * kOne);
                        least[i] = b + 1 < kBins || top == INFINITY ? __float2ull_rn(y * (1.0f - 0x1p-15f) * kOne) : 0;
                    }
                    // where the sums, at most, reach the target at least, and the other way round; the tokens before and up to there
                    const uint64_t m2 = most[0] + most[1], l2 = least[0] + least[1];
                    const uint64_t up_m = warp_prefix(m2), up_l = warp_prefix(l2);
                    const uint32_t up_n = static_cast<uint32_t>(warp_prefix(n[0] + n[1]));
                    if (lane == 31) s->warp_most[warp] = up_m, s->warp_least[warp] = up_l, s->warp_count[warp] = up_n;
                    if (threadIdx.x == 0) s->range = {kBins - 1, 0, kBins - 1, ~0u};
                    __syncthreads();
                    uint64_t before_m = up_m - m2, before_l = up_l - l2, whole_m, whole_l;
                    uint32_t before_n = up_n - (n[0] + n[1]), whole_n;
                    add_up(s->warp_most, warp, before_m, whole_m);
                    add_up(s->warp_least, warp, before_l, whole_l);
                    add_up(s->warp_count, warp, before_n, whole_n);
                    const uint64_t target_lo = Target::share(whole_l, top_p), target_hi = Target::share(whole_m, top_p);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if (before_m < target_lo && target_lo <= before_m + most[i]) s->range.lo = 2 * threadIdx.x + i, s->range.above = before_n;
                        before_m += most[i], before_n += n[i];
                        if (before_l < target_hi && target_hi <= before_l + least[i]) s->range.hi = 2 * threadIdx.x + i, s->range.up_to = before_n;
                        before_l += least[i];
                    }
                    __syncthreads();
                    bin_lo = s->range.lo, bin_hi = s->range.hi, above = s->range.above;
                    in = (s->range.up_to == ~0u ? whole_n : s->range.up_to) - above;
                } else {
                    const uint64_t count[2] = {n[0], n[1]};
                    row.find_bin(count, n, false, static_cast<uint64_t>(top_k));
                    __syncthreads();
                    bin_lo = bin_hi = s->found.place;
                    above = static_cast<uint32_t>(s->found.before), in = s->found.count;
                    if (in == ~0u) {  // (fewer tokens than top_k: all but those of -inf)
                        const bool last = threadIdx.x == kThreads - 1;
                        const uint64_t both = row.block_total(static_cast<uint64_t>(n[0] + (last ? 0 : n[1])) << 32 | (last ? n[1] : 0));
                        above = static_cast<uint32_t>(both >> 32), in = static_cast<uint32_t>(both);
                    }
                }
                if (threadIdx.x < row.blocks) *row.at(&s->told, threadIdx.x) = make_uint4(bin_lo, bin_hi, above, in);
            }
            row.join();
            bin_lo = s->told.x, bin_hi = s->told.y, above = s->told.z, in = s->told.w;
            if (in <= kCap) {
                uint64_t before = 0, all = 0;  // weights of the bins before these, and of all
                uint64_t target = top_k - above;
                // the bins' edges as logits: from `from` on up to bin_hi, from `ahead` on before bin_lo (NaN: none)
                float from, ahead;
                least_of_bins(bin_hi, bin_lo - 1, top, scale, from, ahead);
                row.send(from, [&](float l) { return !(l >= ahead); });
                if (by_weight) {
                    row.for_segments([&](int i) {
                        Eight<T> e = row.set(i);
                        uint32_t high[2] = {0, 0}, low[2] = {0, 0};  // of the bins before these, and from them on
                        uint64_t infinite = 0;
#pragma unroll 2
                        for (int j = 0; j < kSet / 2; ++j) {
                            const float2 l = e.next();
                            const Weigher::Pair w = weigh.pair(l);
#pragma unroll
                            for (int q = 0; q < 2; ++q) {
                                const bool first = (q ? l.y : l.x) >= ahead;
                                if (w.live[q] && first) high[0] += w.high[q], low[0] += w.low[q];
                                if (w.live[q] && !first) high[1] += w.high[q], low[1] += w.low[q];
                                if ((q ? l.y : l.x) == weigh.all_of_it) infinite += kOne;
                            }
                        }
                        const uint64_t first = Weigher::weight(high[0], low[0]);
                        before += first, all += first + Weigher::weight(high[1], low[1]) + infinite;
                        return first;
                    });
                    const auto sums = row.sums(before, all);
                    target = Target::share(sums.all2, top_p) - sums.all;
                } else {
                    row.join();
                }
                if (row.rank == 0) {
                    // finer bins from the first one's edge on (what lies a rounding above it counts as in the first)
                    const float edge = top == INFINITY ? top : top - bin_lo / scale, finer = scale * __uint_as_float((127u + __clz(bin_hi - bin_lo) - 22u) << 23);
                    const uint32_t n = s->list_count;  // (tokens of -inf are in no list; where the border lies among them, all others stay)
                    Border b{key_of(-INFINITY), 0xFFFFFFFFu};
                    if (by_weight) b = border_of_sent<true>(s, n, index_bits, target, edge, finer, weigh);
                    else if (target <= n) b = border_of_sent<false>(s, n, index_bits, target, edge, finer, weigh);
                    __syncthreads();
                    if (threadIdx.x < row.blocks) row.at(&s->found, threadIdx.x)->value = static_cast<uint64_t>(b.key) << 32 | b.index;
                }
                row.join();
                last = Border{static_cast<uint32_t>(s->found.value >> 32), static_cast<uint32_t>(s->found.value)};
                todo = !by_weight && top_p < 1.0f ? kTopP : kSelect;
                if (by_weight && min_p == 0.0f) {
                    // the segments' sums lack only the bins' tokens that stay
                    auto kept = [&](float l, int i) {
                        const uint32_t key = key_of(l);
                        return key > last.key || (key == last.key && static_cast<uint32_t>(i) <= last.index);
                    };
                    for (int i = threadIdx.x; i < row.sets; i += kRowSets) {
                        const Eight<T> e = row.set(i);
                        const float lowest = logit_of(last.key);
#pragma unroll
                        for (int j = 0; j < kSet; ++j) {
                            const float l = j & 1 ? e.pair(j >> 1).y : e.pair(j >> 1).x;
                            if (l >= lowest && !(l >= ahead) && kept(l, row.first + kSet * i + j))
                                atomicAdd(reinterpret_cast<unsigned long long *>(&s->segment[i >> 5]), static_cast<unsigned long long>(weigh(l)));
                        }
                    }
                    const uint64_t sum = row.choose_segment([&](float l, int i) -> uint64_t { return kept(l, i) ? weigh(l) : 0; },
                                                            [&](uint64_t all) { return Target::draw(all, u); });
                    chosen = Chosen{static_cast<int32_t>(s->found.place), static_cast<float>(s->found.value) / static_cast<float>(sum)};
                    todo = kNothing;
                }
            }
            if (todo != kNothing) row.join();  // (the memory is used again)
        }
        if (todo != kNothing) chosen = search_all(row, todo, last, top_k, top_p, min_p, u, t, p.vocab, top, bins_over(kRange), weigh);
    }
    if (row.rank == 0 && threadIdx.x == 0) {
        p.token[r] = chosen.token;
        if (p.prob) p.prob[r] = chosen.prob;
    }
}

template <class T> int slice_smem(int slice) {
    return (static_cast<int>(sizeof(Shared)) + 31) / 32 * 32 + (slice + 2 * kSet) * static_cast<int>(sizeof(T));
}

template <class T> cudaError_t launch(SampleParams p, int n, int sms, int device, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    const uint64_t bit = 1ull << (device & 63);
    if (!(done.load(std::memory_order_acquire) & bit)) {
        for (auto kernel : {sample_kernel<T, false>, sample_kernel<T, true>}) {
            cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
            if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e != cudaSuccess) return e;
        }
        done.fetch_or(bit, std::memory_order_acq_rel);
    }
    // blocks of a row: as many as its size asks for (two blocks a multiprocessor), and more while there are
    // multiprocessors without a row. (64 rows of 32000 with mixed filters: 41.4 us; with twice the blocks 44.9, with
    // top_p alone 62 instead of 37. One row of 32000 with all filters: 9.6 us by eight blocks, 11.0 by sixteen.)
    auto slice = [&](int blocks) { return (p.vocab + kSet * blocks - 1) / (kSet * blocks) * kSet; };
    p.blocks = 1;
    while (p.blocks < kMaxCluster &&
           (slice_smem<T>(slice(p.blocks)) > kSmemLimit / 2 || (static_cast<int64_t>(n) * p.blocks <= sms && slice(p.blocks) > 4096 && p.blocks < 8)))
        p.blocks *= 2;
    p.slice = slice(p.blocks);
    // More rows than are at work at once: the dear ones first, so that none of them is left for the end (256 rows of 130001
    // with mixed filters: 166 us in the rows' order, 143 so, before later steps; rows that are alike pay 3 us for it, 45 in all
    // with a top_k of 40).
    p.n = n;
    const bool sorted = n <= kThreads && static_cast<int64_t>(n) * p.blocks > 2 * sms && (p.top_k || p.top_p || p.min_p || p.temperature);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(n) * p.blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = slice_smem<T>(p.slice);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.blocks, attr[1].val.clusterDim.y = 1, attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, sorted ? sample_kernel<T, true> : sample_kernel<T, false>, p);
}

}  // namespace

cudaError_t launch_sample(SampleParams p, int type, int n, int sms, int device, cudaStream_t s) {
    static const std::array<float2, 64> power = [] {  // 2^(i / 64) in two floats
        std::array<float2, 64> t;
        for (int i = 0; i < 64; ++i) {
            const double x = std::exp2(i / 64.0);
            t[i].x = static_cast<float>(x), t[i].y = static_cast<float>(x - static_cast<double>(t[i].x));
        }
        return t;
    }();
    std::copy(power.begin(), power.end(), p.power);
    return type == QG_F32 ? launch<float>(p, n, sms, device, s) : launch<__half>(p, n, sms, device, s);
}

}  // namespace qg
