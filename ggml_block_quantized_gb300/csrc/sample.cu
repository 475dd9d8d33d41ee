// sample.cu - the next token of each row of logits (include/qstep.h, qsample).
//
// A row is read once into the shared memory of a cluster of thread blocks (one
// block, or up to 16 for long rows and few of them), each holding a contiguous
// slice, each warp a contiguous part of it. What follows are passes over that
// memory:
//  * the largest logit m;
//  * with top_k, the threads' own largest logits, a histogram of which gives a cut
//    that k tokens reach, and few others; with min_p alone its weight is the cut.
//    The tokens above it are sent to the row's first block, which sorts them (logit
//    falling, index rising), takes the prefix that the filters keep, sorts that by
//    index and finds the token there.
//  * With a large top_k, or top_p alone, a histogram of m - l (with top_p: and of
//    what the tokens of a bin weigh less than its first would, in 16 bits) gives
//    the bins in which the border lies, one or two. Their tokens go to the first
//    block, which sorts them and, with the sum of the weights before them, finds
//    the last token kept.
//  * Then, as without filters, the token at which the sum of the kept weights, in
//    index order, passes its target: sums per warp, then the block goes through the
//    one warp's part again.
// Where those bins hold too many tokens (equal ones, as a rule), or top_p follows a
// large top_k, bins are divided again, by the bits of the logit, until at most
// kList tokens are in one, or until all in it are equal and their border is found
// by counting in index order.
//
// Weights are 64-bit integers in units of 2^-44 of the largest. So sums, the
// histogram's atomic ones among them, depend on no order, every pass agrees with
// every other, and a border is met as in exact arithmetic: with 32-bit sums a
// token in some thousands would differ from the one that 64 bits give, since
// with 10^5 tokens that many borders share the unit interval. 2^x for them takes
// an argument in two floats, a table of 64 powers and a polynomial of degree 5.
#include <cooperative_groups.h>

#include <algorithm>
#include <array>
#include <atomic>
#include <cfloat>
#include <cmath>

#include "step_kernels.cuh"

namespace cg = cooperative_groups;

namespace qg {

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 1024;
constexpr int kCap = 1024;       // tokens that one block sorts
constexpr int kList = 128;       // tokens whose order is counted directly
constexpr int kMaxCluster = 16;
constexpr int kUnit = 44;        // weights are in units of 2^-44
constexpr uint64_t kOne = 1ull << kUnit;
constexpr float kLeastTemperature = 0x1p-60f;
constexpr float kRange = 64.0f;  // of m - l that the first histogram tells apart
constexpr float kLog2E = 1.44269502162933349609375f, kLog2ERest = 1.925963033500e-8f;

struct Shared {
    float2 power[64];                 // 2^(i / 64) in two floats
    union {
        struct {
            uint64_t sum[kBins];      // weights of a bin
            uint32_t count[kBins];
        };
        uint64_t weight[kCap];        // of the listed tokens
    };
    uint64_t all[kCap];               // (key, ~index) of listed tokens, in the first block
    uint64_t list[kList];             // of a bin's tokens, this block's
    uint64_t warp_sum[kWarps];
    uint64_t block_sum[2][kMaxCluster];
    float2 extremes[kWarps];
    float2 block_extremes[kMaxCluster];
    uint32_t list_count, kept;
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
// Eight logits as they are kept: NaN, which is never chosen, as -inf, and -0 as 0; their extremes go on.
__device__ __forceinline__ void take8(float4 (&v)[2], float &top, float &low) {
    float *x = reinterpret_cast<float *>(v);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[i] = fmaxf(x[i], -INFINITY) + 0.0f;
        top = fmaxf(top, x[i]);
        if (x[i] > -INFINITY) low = fminf(low, x[i]);
    }
}
__device__ __forceinline__ void take8(uint4 (&v)[1], float &top, float &low) {
    __half2 *x = reinterpret_cast<__half2 *>(v);
    const __half2 none = __half2half2(__ushort_as_half(0xFC00u)), zero = __half2half2(__ushort_as_half(0));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[i] = __hadd2(__hmax2(x[i], none), zero);
        const float2 f = __half22float2(x[i]);
        top = fmaxf(top, fmaxf(f.x, f.y));
        if (f.x > -INFINITY) low = fminf(low, f.x);
        if (f.y > -INFINITY) low = fminf(low, f.y);
    }
}
template <class T> struct Eight;
template <> struct Eight<float> { float4 v[2]; };
template <> struct Eight<__half> { uint4 v[1]; };

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
    __device__ __forceinline__ uint64_t operator()(float l) const {
        const float a = l - base, xh = a * ch;
        if (l == all_of_it) return kOne;
        if (!(xh > least)) return 0;  // (-inf among them)
        const float low = fmaf(a, cl, fmaf(a, ch, -xh));  // 2^-17 at most
        // x = k / 64 + r + low, |r| <= 2^-7: r exact
        const float km = fmaf(xh, 64.0f, magic);
        const int k = static_cast<int>(__float_as_uint(km)) - 0x4B400000;
        const float r = fmaf(km - magic, -0x1p-6f, xh);
        // 2^(r + low) - 1 = u + rest, u = r ln 2 rounded (low's square, 2^-36 at most, is left out)
        const float ln2 = 0.693147182464599609375f, ln2_rest = -1.904654323148236e-9f;
        const float u = r * ln2, low_ln2 = low * ln2;
        const float p = fmaf(r, fmaf(r, fmaf(r, 1.3333558146e-3f, 9.6181291076e-3f), 5.5504108665e-2f), 2.4022650696e-1f);
        const float r2 = r * r, rest = fmaf(r2, p, fmaf(low_ln2, fmaf(r2, p, u), fmaf(r, ln2_rest, fmaf(r, ln2, -u)) + low_ln2));
        const float2 t = power[k & 63];
        const float v = t.x * u;  // times t.x + t.y, the product by t.x in two parts
        const float v_low = fmaf(t.x, u, -v) + fmaf(t.x, rest, fmaf(t.y, u, t.y));
        // to whole units: v + v_low in units of 2^-28, the rest in 2^-44 (conversions by addition: the instruction is four times slower)
        const float round = 12582912.0f, vi = fmaf(v + v_low, 0x1p28f, round);
        const float ri = fmaf(fmaf(vi - round, -0x1p-28f, v) + v_low, 0x1p44f, round);
        const int64_t part = static_cast<int64_t>(static_cast<int>(__float_as_uint(vi)) - 0x4B400000) * (1 << (kUnit - 28)) +
                             (static_cast<int>(__float_as_uint(ri)) - 0x4B400000);
        const uint64_t whole = static_cast<uint64_t>((__float_as_uint(t.x) & 0x7FFFFFu) | 0x800000u) * (1u << (kUnit - 23)) + part;
        const int down = -(k >> 6);
        return down <= 0 ? whole : (whole + (1ull << (down - 1))) >> down;
    }
};

// The bin of a histogram of m - l.
__device__ __forceinline__ uint32_t bin_of(float l, float m, float scale) {
    return min(static_cast<uint32_t>(max(__float2int_rz((m - l) * scale), 0)), kBins - 1u);
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

// A row in the cluster's shared memory.
template <class T> struct Row {
    Shared *s;
    const T *data;             // this block's slice
    int first, count, part;    // its first index and size; a warp's part of it (a multiple of 64)
    int rank, blocks;
    int turn = 0;              // which of the two sums' places is next

    __device__ __forceinline__ float logit(int i) const { return static_cast<float>(data[i]); }
    template <class F> __device__ __forceinline__ void each(F f) const {  // f(logit, index)
        const int lane = threadIdx.x & 31, from = (threadIdx.x >> 5) * part;
        const int to = min(from + part, count);
        for (int i = from + lane; i < to; i += 32) f(logit(i), first + i);
    }
    __device__ __forceinline__ void join() const {  // the whole cluster
        if (blocks == 1) __syncthreads();
        else cg::this_cluster().sync();
    }
    template <class P> __device__ __forceinline__ P *at(P *p, int block) const {
        return blocks == 1 ? p : cg::this_cluster().map_shared_rank(p, block);
    }
    // Sums over the blocks before this one, over this one, and over all.
    struct Sums { uint64_t before, mine, all; };
    __device__ __forceinline__ Sums sums(uint64_t v) {
        v = warp_total(v);
        if ((threadIdx.x & 31) == 0) s->warp_sum[threadIdx.x >> 5] = v;
        __syncthreads();
        uint64_t block = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) block += s->warp_sum[w];
        uint64_t *const place = s->block_sum[turn];
        turn ^= 1;
        if (threadIdx.x < blocks) at(place, threadIdx.x)[rank] = block;
        join();
        Sums r{0, block, 0};
        for (int b = 0; b < blocks; ++b) {
            if (b < rank) r.before += place[b];
            r.all += place[b];
        }
        return r;
    }
    // The token, in index order, at which the sum of value(logit, index) reaches target(sum of all); found.place is its
    // index, found.value its value. Returns the sum of all.
    template <class V, class G> __device__ __forceinline__ uint64_t select(V value, G target) {
        uint64_t mine = 0;
        each([&](float l, int i) { mine += value(l, i); });
        const Sums r = sums(mine);
        const uint64_t t = target(r.all);
        if (r.before < t && t <= r.before + r.mine) {  // in this block: it goes through the one warp's part again
            uint64_t before = r.before;
            int w = 0;
            while (t > before + s->warp_sum[w]) before += s->warp_sum[w++];
            __syncthreads();
            const int from = w * part, to = min(from + part, count), per = (part + kThreads - 1) / kThreads;
            const int i0 = from + per * threadIdx.x, i1 = min(i0 + per, to);
            uint64_t sum = 0;
            for (int i = i0; i < i1; ++i) sum += value(logit(i), first + i);
            const uint64_t up_to = warp_prefix(sum);
            if ((threadIdx.x & 31) == 31) s->warp_sum[threadIdx.x >> 5] = up_to;
            __syncthreads();
            before += up_to - sum;
            for (int v = 0; v < (threadIdx.x >> 5); ++v) before += s->warp_sum[v];
            if (before < t && t <= before + sum)
                for (int i = i0; i < i1; ++i) {
                    const uint64_t v = value(logit(i), first + i);
                    before += v;
                    if (before >= t) {
                        for (int b = 0; b < blocks; ++b) {
                            auto *f = at(&s->found, b);
                            f->place = first + i, f->value = v;
                        }
                        break;
                    }
                }
        }
        join();
        return r.all;
    }
    // Bins of a histogram, in order of place(bin), each thread two neighbours: where the running sum of v reaches
    // `target`. found: the bin, the sum before it, and its n. Every thread of every block calls it.
    __device__ __forceinline__ void find_bin(const uint64_t (&v)[2], const uint32_t (&n)[2], bool rising, uint64_t target) {
        const uint64_t both = v[0] + v[1], up_to = warp_prefix(both);
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        if (lane == 31) s->warp_sum[warp] = up_to;
        __syncthreads();
        uint64_t before = up_to - both;
        for (int w = 0; w < warp; ++w) before += s->warp_sum[w];
        if (rising) {  // counted from the last bin
            uint64_t whole = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) whole += s->warp_sum[w];
            before = whole - before - both;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int b = rising ? 1 - i : i;
            if (before < target && target <= before + v[b]) s->found.place = 2 * threadIdx.x + b, s->found.before = before, s->found.count = n[b];
            before += v[b];
        }
    }
    __device__ __forceinline__ uint64_t block_total(uint64_t v) {  // over this block's threads
        v = warp_total(v);
        __syncthreads();
        if ((threadIdx.x & 31) == 0) s->warp_sum[threadIdx.x >> 5] = v;
        __syncthreads();
        uint64_t all = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) all += s->warp_sum[w];
        __syncthreads();
        return all;
    }
    __device__ __forceinline__ void clear_bins(bool weights) {
        for (int b = threadIdx.x; b < kBins; b += kThreads) {
            s->count[b] = 0;
            if (weights) s->sum[b] = 0;
        }
    }
    __device__ __forceinline__ void bin_counts(uint32_t (&n)[2]) const {
        n[0] = n[1] = 0;
        for (int b = 0; b < blocks; ++b) {
            const uint2 c = *reinterpret_cast<const uint2 *>(at(s->count, b) + 2 * threadIdx.x);
            n[0] += c.x, n[1] += c.y;
        }
    }
    // Tokens for which take(logit) holds are sent to the first block, as far as there is room.
    template <class F> __device__ __forceinline__ void send(F take) {
        const int lane = threadIdx.x & 31, from = (threadIdx.x >> 5) * part, to = min(from + part, count);
        uint64_t *const there = at(s->all, 0);
        uint32_t *const counter = at(&s->list_count, 0);
        for (int i0 = from; i0 < to; i0 += 32) {
            const int i = i0 + lane;
            const float l = i < to ? logit(i) : -INFINITY;
            const bool in = i < to && take(l);
            const uint32_t who = __ballot_sync(0xffffffffu, in);
            if (who == 0) continue;
            uint32_t place = 0;
            if (lane == 0) place = atomicAdd(counter, static_cast<uint32_t>(__popc(who)));
            place = __shfl_sync(0xffffffffu, place, 0) + __popc(who & ((1u << lane) - 1));
            if (in && place < kCap) there[place] = static_cast<uint64_t>(key_of(l)) << 32 | ~static_cast<uint32_t>(first + i);
        }
    }
    // The border at which the running value (1, or the weight) over the tokens up to `limit`, in falling order,
    // reaches `target` (at least 1, at most the sum of all): value(l) is a token's.
    template <bool WEIGHTS, class W>
    __device__ __forceinline__ Border border(Border limit, uint64_t target, float m, float scale, float reach, W weigh) {
        uint32_t lo = 0, hi = 0, bin0 = 0;
        int shift = -1;  // -1: the first histogram, of m - l
        auto first_bin = [&](float l) { return bin_of(l, m, scale); };
        auto member = [&](float l, int i, uint32_t &bin) {
            const uint32_t key = key_of(l);
            if (key < limit.key || (key == limit.key && static_cast<uint32_t>(i) > limit.index)) return false;
            bin = first_bin(l);
            if (shift < 0) return true;
            if (bin != bin0 || key < lo || key > hi) return false;
            bin = (key - lo) >> shift;
            return true;
        };
        for (;;) {
            clear_bins(WEIGHTS);
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
            uint64_t v[2] = {0, 0};
            uint32_t n[2];
            bin_counts(n);
            for (int b = 0; b < blocks && WEIGHTS; ++b) v[0] += at(s->sum, b)[2 * threadIdx.x], v[1] += at(s->sum, b)[2 * threadIdx.x + 1];
            if (!WEIGHTS) v[0] = n[0], v[1] = n[1];
            // bins of the first histogram fall with the logit, those of the others rise
            find_bin(v, n, shift >= 0, target);
            join();  // (the histograms have been read, too)
            const uint32_t bin = s->found.place, in_bin = s->found.count;
            target -= s->found.before;
            if (shift < 0) {
                bin0 = bin;
                lo = bin == kBins - 1 ? 0u : key_of(m - (bin + 2) / scale);
                hi = key_of(m - (bin == 0 ? 0.0f : (bin - 1) / scale));
            } else {
                lo += bin << shift;
                const uint32_t top = lo + ((1u << shift) - 1u);
                hi = top < lo || top > hi ? hi : top;
            }
            const uint32_t width = hi - lo;
            shift = width < kBins ? 0 : 22 - __clz(width);
            if (in_bin <= kList) break;
            if (lo == hi) {  // so many equal ones: the border is found by index
                const float l = logit_of(lo);
                const uint64_t each_one = WEIGHTS ? weigh(l) : 1;
                const uint64_t nth = (target + each_one - 1) / each_one;
                __syncthreads();
                select([&](float x, int i) -> uint64_t { return key_of(x) == lo && (lo != limit.key || static_cast<uint32_t>(i) <= limit.index); },
                       [&](uint64_t) { return nth; });
                return Border{lo, s->found.place};
            }
            __syncthreads();
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
            for (int i = threadIdx.x; i < m; i += kThreads) {
                const uint64_t e = at(s->list, b)[i];
                s->all[n + i] = e;
                s->weight[n + i] = WEIGHTS ? weigh(logit_of(static_cast<uint32_t>(e >> 32))) : 1;
            }
            n += m;
        }
        __syncthreads();
        if (threadIdx.x < n) {
            const uint64_t e = s->all[threadIdx.x], v = s->weight[threadIdx.x];
            uint64_t before = 0;
            for (int i = 0; i < n; ++i) before += s->all[i] > e ? s->weight[i] : 0;
            if (before < target && target <= before + v) s->found.value = e;
        }
        join();
        const uint64_t e = s->found.value;
        __syncthreads();  // (what is found next is written to the same place)
        return Border{static_cast<uint32_t>(e >> 32), ~static_cast<uint32_t>(e)};
    }
};

// A block's 2 kThreads places: thread (w, lane) has 64 w + lane and the one 32 on.
__device__ __forceinline__ int place_of(int i) { return 64 * (threadIdx.x >> 5) + (threadIdx.x & 31) + 32 * i; }

// Sorts the first n places (a power of two, 64 at least; the others hold 0) so that they fall; `space` holds 2 kThreads.
// Neighbours up to 32 apart meet by shuffles, the others in memory.
__device__ __forceinline__ void sort_falling(uint64_t (&v)[2], int n, uint64_t *space) {
    for (int size = 2; size <= n; size *= 2)
        for (int stride = size / 2; stride > 0; stride /= 2) {
            uint64_t o[2] = {v[1], v[0]};
            if (stride < 64 && 64 * static_cast<int>(threadIdx.x >> 5) >= n) continue;
            if (stride >= 64) {
                __syncthreads();
#pragma unroll
                for (int i = 0; i < 2; ++i) space[place_of(i)] = v[i];
                __syncthreads();
#pragma unroll
                for (int i = 0; i < 2; ++i) o[i] = space[place_of(i) ^ stride];
            } else if (stride < 32) {
#pragma unroll
                for (int i = 0; i < 2; ++i) o[i] = __shfl_xor_sync(0xffffffffu, v[i], stride);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int at = place_of(i);
                const bool larger = ((at & stride) == 0) == ((at & size) == 0);
                if ((o[i] > v[i]) == larger) v[i] = o[i];
            }
        }
}
// Running sums in the order of the places: what lies before each, and the whole.
__device__ __forceinline__ uint64_t running(Shared *s, const uint64_t (&w)[2], uint64_t (&before)[2]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint64_t a = warp_prefix(w[0]), b = warp_prefix(w[1]), half = __shfl_sync(0xffffffffu, a, 31);
    __syncthreads();  // (the places may still be read)
    if (lane == 31) s->warp_sum[warp] = half + b;
    __syncthreads();
    uint64_t base = 0, all = 0;
#pragma unroll
    for (int v = 0; v < kWarps; ++v) {
        if (v < warp) base += s->warp_sum[v];
        all += s->warp_sum[v];
    }
    before[0] = base + a - w[0], before[1] = base + half + b - w[1];
    return all;
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

__device__ __forceinline__ int places(int n) {  // a power of two
    int n2 = 64;
    while (n2 < n) n2 *= 2;
    return n2;
}

// The listed tokens of a row (s->all, n of them, sorted here), by one block. The tokens before them weigh `ahead` and
// stay; of these, the first top_k (0: all); then those before which, `ahead` included, less than `target` has been
// passed, a share of the sum of the first top_k where target is 0; then those of min_p. Returns how many stay, a prefix.
__device__ __forceinline__ int keep_listed(Shared *s, int n, int top_k, float top_p, float min_p, uint64_t ahead, uint64_t target,
                                           const Weigher &weigh, uint64_t (&v)[2], uint64_t (&w)[2]) {
    if (threadIdx.x == 0) s->kept = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) v[i] = place_of(i) < n ? s->all[place_of(i)] : 0;
    sort_falling(v, places(n), s->all);
    if (top_k > 0) n = min(n, top_k);
    uint64_t before[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) w[i] = place_of(i) < n ? weigh(logit_of(static_cast<uint32_t>(v[i] >> 32))) : 0;
    const uint64_t all = running(s, w, before);
    if (target == 0) target = top_p < 1.0f ? Target::share(all, top_p) : ~0ull;
    const uint64_t light = min_p > 0.0f ? Target::share(weigh(weigh.m), min_p) : 1;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (w[i] >= light && ahead + before[i] < target) atomicMax(&s->kept, static_cast<uint32_t>(place_of(i) + 1));
    __syncthreads();
    return static_cast<int>(s->kept);
}

// The token among the first n places, sorted by their indexes; found.place and found.value. Returns the sum of all.
__device__ __forceinline__ uint64_t choose_listed(Shared *s, int n, const uint64_t (&v)[2], uint64_t (&w)[2], float u) {
    uint64_t e[2], before[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        s->weight[place_of(i)] = w[i];
        e[i] = place_of(i) < n ? v[i] << 32 | static_cast<uint32_t>(place_of(i)) : 0;  // (~index falls)
    }
    __syncthreads();
    sort_falling(e, places(n), s->all);
#pragma unroll
    for (int i = 0; i < 2; ++i) w[i] = place_of(i) < n ? s->weight[static_cast<uint32_t>(e[i])] : 0;
    const uint64_t all = running(s, w, before), t = Target::draw(all, u);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (before[i] < t && t <= before[i] + w[i]) s->found.place = ~static_cast<uint32_t>(e[i] >> 32), s->found.value = w[i];
    __syncthreads();
    return all;
}

enum Todo { kNothing, kSelect, kTopP, kAll };

template <class T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleParams p) {
    extern __shared__ __align__(16) uint8_t smem[];
    Shared *const s = reinterpret_cast<Shared *>(smem);
    T *const space = reinterpret_cast<T *>(smem + (sizeof(Shared) + 31) / 32 * 32);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t r = blockIdx.x / p.blocks;
    Row<T> row;
    row.s = s;
    row.blocks = p.blocks;
    row.rank = static_cast<int>(blockIdx.x % p.blocks);
    row.part = p.part;
    row.first = row.rank * kWarps * p.part;
    row.count = max(0, min(p.vocab - row.first, kWarps * p.part));
    if (threadIdx.x < 64) s->power[threadIdx.x] = p.power[threadIdx.x];
    if (threadIdx.x == 0) s->list_count = 0;
    row.clear_bins(false);
    if (p.blocks > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    pdl_allow_dependents();
    pdl_wait_prior_grids();

    // ---- the row, as far from a boundary of eight elements here as there
    const T *const src = static_cast<const T *>(p.logits) + r * p.stride + row.first;
    const int pad = static_cast<int>(reinterpret_cast<uintptr_t>(src) / sizeof(T) & 7u);
    row.data = space + pad;
    float top = -INFINITY, low = INFINITY;
    constexpr int kAhead = sizeof(T) == 4 ? 4 : 8;  // sets of eight that a thread has under way
    for (int i0 = 8 * threadIdx.x - pad; i0 < row.count; i0 += 8 * kThreads * kAhead) {
        Eight<T> e[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int i = i0 + 8 * kThreads * k;
            if (i >= 0 && i + 8 <= row.count) {
                e[k] = *reinterpret_cast<const Eight<T> *>(src + i);
            } else {
                T *x = reinterpret_cast<T *>(&e[k]);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = i + j >= 0 && i + j < row.count ? src[i + j] : static_cast<T>(-INFINITY);
            }
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int i = i0 + 8 * kThreads * k;
            take8(e[k].v, top, low);
            if (i < row.count) *reinterpret_cast<Eight<T> *>(space + pad + i) = e[k];
        }
    }
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
    for (int b = 0; b < row.blocks; ++b) top = fmaxf(top, s->block_extremes[b].x), low = fminf(low, s->block_extremes[b].y);

    // ---- the settings
    const float t = p.temperature ? p.temperature[r] : 1.0f;
    float top_p = p.top_p ? p.top_p[r] : 1.0f, min_p = p.min_p ? p.min_p[r] : 0.0f;
    int top_k = p.top_k ? p.top_k[r] : 0;
    if (top_k < 0 || top_k >= p.vocab) top_k = 0;
    if (!(top_p < 1.0f)) top_p = 1.0f;  // (NaN: all)
    if (!(min_p > 0.0f)) min_p = 0.0f;
    const float u = p.uniform[r];
    int32_t token = -1;
    float prob = 0.0f;
    if (top > -INFINITY) {
        if (!(t >= kLeastTemperature) || top_k == 1 || top_p <= 0.0f || min_p > 1.0f) {  // the first alone
            uint32_t first = 0xFFFFFFFFu;
            if (mine_top == top)
                for (int i0 = 8 * threadIdx.x - pad; i0 < row.count && first == 0xFFFFFFFFu; i0 += 8 * kThreads)
                    for (int i = max(i0, 0); i < min(i0 + 8, row.count); ++i)
                        if (first == 0xFFFFFFFFu && row.logit(i) == top) first = row.first + i;
            first = __reduce_min_sync(0xffffffffu, first);
            if (lane == 0 && first != 0xFFFFFFFFu)  // (list_count holds 0 less the least index so far)
                for (int b = 0; b < row.blocks; ++b) atomicMax(row.at(&s->list_count, b), 0u - 1u - first);
            row.join();
            token = static_cast<int32_t>(0u - 1u - s->list_count), prob = 1.0f;
        } else {
            Weigher weigh;
            weigh.set(s->power, top, t);
            Border last{0u, 0xFFFFFFFFu};
            int todo = kSelect;  // what is left: the filters (kAll, kTopP), the selection, or nothing
            // bins per unit of m - l, a power of two, over so much
            auto bins_over = [&](float most) { return __uint_as_float(__float_as_uint((kBins - 1) / fminf(fmaxf(top - low, 0x1p-100f), most)) & 0x7F800000u); };
            const bool by_weight = top_k == 0 && top_p < 1.0f;
            const float scale = bins_over(by_weight ? fminf(32.0f * t, FLT_MAX) : kRange);
            const float reach = top == INFINITY ? 0.0f : top + (log2f(min_p) - 0.02f) * t * 0.694f - 1e-6f * fabsf(top);  // (of min_p alone)
            if (top_k > 0 ? top_k <= kThreads * row.blocks : top_p == 1.0f && min_p > 0.0f) {
                // ---- a cut that as many tokens reach, by the threads' own largest, or that min_p gives
                uint32_t last_bin = 0;
                if (top_k > 0) {
                    if (mine_top > -INFINITY) atomicAdd(&s->count[bin_of(mine_top, top, scale)], 1u);
                    row.join();
                    uint32_t n[2];
                    row.bin_counts(n);
                    const uint64_t count[2] = {n[0], n[1]};
                    if (threadIdx.x == 0) s->found.place = kBins - 1;
                    __syncthreads();
                    row.find_bin(count, n, false, static_cast<uint64_t>(top_k));
                    __syncthreads();
                    last_bin = s->found.place;
                }
                row.send([&](float l) { return top_k > 0 ? bin_of(l, top, scale) <= last_bin : l > reach; });
                row.join();
                const uint32_t n = *row.at(&s->list_count, 0);
                if (n <= kCap) {  // the first block goes on alone, in its own memory, and stays until the others have read it
                    todo = kNothing;
                    if (p.blocks > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
                }
                if (n > kCap && top_k > 0) todo = kAll;
                if (todo == kNothing && row.rank == 0) {
                    uint64_t v[2], w[2];
                    const int kept = keep_listed(s, n, top_k, top_p, min_p, 0, 0, weigh, v, w);
                    const uint64_t all = choose_listed(s, kept, v, w, u);
                    token = static_cast<int32_t>(s->found.place);
                    prob = static_cast<float>(s->found.value) / static_cast<float>(all);
                }
                if (todo == kNothing && p.blocks > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
            } else if (top_k > 0 || by_weight) {
                todo = kAll;
            }
            if (todo == kAll) {
                // ---- the bins in which the border lies
                row.join();  // (the memory is used again)
                row.clear_bins(true);
                if (threadIdx.x == 0) s->list_count = 0;
                row.join();
                uint32_t *const deficit = reinterpret_cast<uint32_t *>(s->sum);  // of a bin's tokens' weights, in 2^-16 of its first possible one
                const float per_bin = weigh.ch / scale;                         // log2 of the weights' ratio over a bin, 0.1 at most
                row.each([&](float l, int) {
                    const uint32_t b = bin_of(l, top, scale);
                    atomicAdd(&s->count[b], 1u);
                    if (by_weight && b + 1 < kBins) {
                        float y;
                        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(((top - l) * scale - b) * -per_bin));
                        atomicAdd(&deficit[b], static_cast<uint32_t>(__float2int_rn((1.0f - y) * 65536.0f)));
                    }
                });
                row.join();
                uint32_t n[2];
                row.bin_counts(n);
                uint32_t bin_lo, bin_hi;
                if (by_weight) {
                    // what the bins weigh at most and at least, off by 2^-15 in all: half a unit of 2^-16 for each token and
                    // the steps to it; of the last bin's tokens only the upper bound is known
                    uint64_t most[2], least[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int b = 2 * threadIdx.x + i;
                        uint32_t less = 0;
                        for (int q = 0; q < row.blocks; ++q) less += row.at(deficit, q)[b];
                        float y;
                        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(-b * per_bin));
                        y *= static_cast<float>(n[i]) - static_cast<float>(less) * 0x1p-16f;
                        if (top == INFINITY) y = b == 0 ? static_cast<float>(n[i]) : 0.0f;
                        most[i] = __float2ull_rn(y * (1.0f + 0x1p-15f) * kOne);
                        least[i] = b + 1 < kBins || top == INFINITY ? __float2ull_rn(y * (1.0f - 0x1p-15f) * kOne) : 0;
                    }
                    const uint64_t all_most = row.block_total(most[0] + most[1]), all_least = row.block_total(least[0] + least[1]);
                    if (threadIdx.x == 0) s->found.place = kBins - 1;
                    __syncthreads();
                    row.find_bin(most, n, false, Target::share(all_least, top_p));
                    __syncthreads();
                    bin_lo = s->found.place;
                    __syncthreads();
                    if (threadIdx.x == 0) s->found.place = kBins - 1;
                    __syncthreads();
                    row.find_bin(least, n, false, Target::share(all_most, top_p));
                    __syncthreads();
                    bin_hi = max(bin_lo, s->found.place);
                } else {
                    const uint64_t count[2] = {n[0], n[1]};
                    row.find_bin(count, n, false, static_cast<uint64_t>(top_k));
                    __syncthreads();
                    bin_lo = bin_hi = s->found.place;
                }
                uint32_t above = 0, in = 0;  // tokens in the bins before these, and in them
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t b = 2 * threadIdx.x + i;
                    if (b < bin_lo) above += n[i];
                    else if (b <= bin_hi) in += n[i];
                }
                const uint64_t both = row.block_total(static_cast<uint64_t>(above) << 32 | in);
                above = static_cast<uint32_t>(both >> 32), in = static_cast<uint32_t>(both);
                if (in <= kCap) {
                    uint64_t before = 0, after = 0;
                    row.send([&](float l) {
                        const uint32_t b = bin_of(l, top, scale);
                        if (by_weight) {
                            const uint64_t w = weigh(l);
                            if (b < bin_lo) before += w;
                            else after += w;
                        }
                        return b >= bin_lo && b <= bin_hi;
                    });
                    uint64_t ahead = 0, target = ~0ull;
                    if (by_weight) {
                        ahead = row.sums(before).all;
                        target = Target::share(ahead + row.sums(after).all, top_p);
                    }
                    if (threadIdx.x == 0) s->found.count = 0;  // (1 once the first block has found the border)
                    row.join();
                    if (row.rank == 0) {
                        uint64_t v[2], w[2];
                        const int kept = keep_listed(s, in, by_weight ? 0 : top_k - static_cast<int>(above), 1.0f, 0.0f, ahead, target, weigh, v, w);
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            if (place_of(i) + 1 == kept)
                                for (int b = 0; b < row.blocks; ++b) row.at(&s->found, b)->value = v[i], row.at(&s->found, b)->count = 1;
                    }
                    row.join();
                    if (s->found.count != 0) {
                        last = Border{static_cast<uint32_t>(s->found.value >> 32), ~static_cast<uint32_t>(s->found.value)};
                        todo = !by_weight && top_p < 1.0f ? kTopP : kSelect;
                    }
                }
                row.join();  // (the memory is used again)
            }
            if (todo != kNothing) {
                // ---- any number of them
                auto kept = [&](float l, int i) {
                    const uint32_t key = key_of(l);
                    return key > last.key || (key == last.key && static_cast<uint32_t>(i) <= last.index);
                };
                if (todo == kAll && top_k > 0) last = row.template border<false>(last, top_k, top, bins_over(kRange), 0.0f, weigh);
                if (todo != kSelect && top_p < 1.0f) {
                    uint64_t mine = 0;
                    row.each([&](float l, int i) {
                        if (kept(l, i)) mine += weigh(l);
                    });
                    const uint64_t all = row.sums(mine).all;
                    // Weights below (1 - top_p) / vocab of the sum are all past the border: their sum is less than what is cut.
                    const float least = (1.0f - top_p) * (static_cast<float>(all) * (1.0f / kOne)) / static_cast<float>(p.vocab);
                    const float reach = top == INFINITY ? 0.0f : top + (log2f(least) - 0.02f) * t * 0.694f - 1e-6f * fabsf(top);
                    last = row.template border<true>(last, Target::share(all, top_p), top, bins_over(kRange), reach, weigh);
                }
                const uint64_t light = min_p > 0.0f ? Target::share(weigh(top), min_p) : 0;
                const uint64_t all = row.select(
                    [&](float l, int i) -> uint64_t {
                        if (!kept(l, i)) return 0;
                        const uint64_t w = weigh(l);
                        return w >= light ? w : 0;
                    },
                    [&](uint64_t all) { return Target::draw(all, u); });
                token = static_cast<int32_t>(s->found.place);
                prob = static_cast<float>(s->found.value) / static_cast<float>(all);
            }
        }
    }
    if (row.rank == 0 && threadIdx.x == 0) {
        p.token[r] = token;
        if (p.prob) p.prob[r] = prob;
    }
}

template <class T> int slice_smem(int part) {
    return (static_cast<int>(sizeof(Shared)) + 31) / 32 * 32 + (kWarps * part + 16) * static_cast<int>(sizeof(T));
}

template <class T> cudaError_t launch(SampleParams p, int n, int sms, int device, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    const uint64_t bit = 1ull << (device & 63);
    if (!(done.load(std::memory_order_acquire) & bit)) {
        cudaError_t e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        done.fetch_or(bit, std::memory_order_acq_rel);
    }
    // blocks of a row: as many as its size asks for, and more while there are multiprocessors without a row
    auto part = [&](int blocks) { return (p.vocab + 64 * kWarps * blocks - 1) / (64 * kWarps * blocks) * 64; };
    p.blocks = 1;
    while (p.blocks < kMaxCluster &&
           (slice_smem<T>(part(p.blocks)) > kSmemLimit / 2 || (static_cast<int64_t>(n) * p.blocks * 2 <= sms && part(p.blocks) >= 256 && p.blocks < 8)))
        p.blocks *= 2;
    p.part = part(p.blocks);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(n) * p.blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = slice_smem<T>(p.part);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.blocks, attr[1].val.clusterDim.y = 1, attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, sample_kernel<T>, p);
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
