// sample.cu - the next token of each row of logits (include/qstep.h, qsample).
//
// A row is read once into the shared memory of a cluster of thread blocks (one
// block, or up to 16 for long rows and few of them), each holding a contiguous
// slice, each warp a contiguous part of it. What follows are passes over that
// memory, joined through the cluster:
//  * the largest logit m;
//  * where top_k or top_p holds: the last token kept, as a border in the order
//    (logit falling, index rising). A histogram of m - l (linear bins of a power
//    of two, so that bins follow the logits' order exactly) gives the bin in
//    which the count or the weights' sum passes its target; that bin is divided
//    again, now by the bits of the logit, until at most kList tokens are in it,
//    whose places among each other are counted directly; or until all in it are
//    equal, where the border's index is found by counting in index order;
//  * the token at which the sum of the kept weights, in index order, passes its
//    target: sums per warp, then the one warp goes through its part again.
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
#include <cmath>

#include "step_kernels.cuh"

namespace cg = cooperative_groups;

namespace qg {

namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kBins = kThreads;  // a thread a bin
constexpr int kList = 128;       // tokens whose order is counted directly
constexpr int kMaxCluster = 16;
constexpr int kUnit = 44;        // weights are in units of 2^-44
constexpr uint64_t kOne = 1ull << kUnit;
constexpr float kLeastTemperature = 0x1p-60f;
constexpr float kRange = 64.0f;  // of m - l that the first histogram tells apart

struct Shared {
    float2 power[64];                 // 2^(i / 64) in two floats
    uint64_t sum[kBins];              // weights of a bin
    uint32_t count[kBins];
    uint64_t list[kList], all[kList]; // (key, ~index) of a bin's tokens: this block's, the cluster's
    uint64_t weight[kList];
    uint64_t warp_sum[kWarps];
    uint64_t block_sum[2][kMaxCluster];
    float2 extremes[kWarps];
    float2 block_extremes[kMaxCluster];
    uint32_t list_count;
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
__device__ __forceinline__ float plain_logit(float l) { return l != l ? -INFINITY : l + 0.0f; }  // NaN: never chosen; -0 is 0

__device__ __forceinline__ void load8(const float *p, float (&v)[8]) {
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load8(const __half *p, float (&v)[8]) {
    const uint4 a = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
}

// exp((l - m) / T) in units of 2^-44: 2^x for x = (l - m) log2(e) / T.
struct Weigher {
    const float2 *power;
    float m, ch, cl;  // log2(e) / T in two floats
    __device__ __forceinline__ uint64_t operator()(float l) const {
        if (m == INFINITY) return l == INFINITY ? kOne : 0;
        // l - m in two floats
        const float dh = l - m, b = dh - l;
        const float dl = (l - (dh - b)) - (m + b);
        const float xh = dh * ch;
        if (!(xh > -46.0f)) return 0;  // (-inf among them)
        float xl = fmaf(dh, ch, -xh);
        xl = fmaf(dh, cl, xl);
        xl = fmaf(dl, ch, xl);
        // x = k / 64 + r, |r| <= 2^-7 (and a little)
        const float km = fmaf(xh, 64.0f, 12582912.0f);
        const int k = static_cast<int>(__float_as_uint(km)) - 0x4B400000;
        const float r = fmaf(km - 12582912.0f, -0x1p-6f, xh);
        // a = (r + xl) ln 2 in two floats, exp(a) - 1 = a + a^2/2 + ...
        const float ln2 = 0.693147182464599609375f, ln2_rest = -1.904654323148236e-9f;
        const float ah = r * ln2;
        const float al = fmaf(xl, ln2, fmaf(r, ln2_rest, fmaf(r, ln2, -ah)));
        const float a2 = ah * ah;
        const float a2_rest = fmaf(ah, ah, -a2);
        const float high = a2 * ah * fmaf(ah, fmaf(ah, 1.0f / 120.0f, 1.0f / 24.0f), 1.0f / 6.0f);
        const float rest = fmaf(ah, al, fmaf(0.5f, a2_rest, al)) + high;  // exp(a) - 1 = ah + a2 / 2 + rest
        const float2 p = power[k & 63];
        // times p.x + p.y, the products by p.x exact
        const float u = p.x * ah, v = p.x * (0.5f * a2);
        const float low = fmaf(p.x, ah, -u) + fmaf(p.x, 0.5f * a2, -v) + fmaf(p.x, rest, fmaf(p.y, ah, p.y));
        const int part = __float2int_rn(u * 0x1p37f) + __float2int_rn(v * 0x1p37f) + __float2int_rn(low * 0x1p37f);
        const uint64_t whole = (static_cast<uint64_t>((__float_as_uint(p.x) & 0x7FFFFFu) | 0x800000u) << (kUnit - 23)) +
                               (static_cast<int64_t>(part) << (kUnit - 37));
        const int down = -(k >> 6);  // k <= 0
        return down == 0 ? whole : (whole + (1ull << (down - 1))) >> down;
    }
};

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
struct Row {
    Shared *s;
    const float *data;         // this block's slice
    int first, count, part;    // its first index and size; a warp's part of it (a multiple of 32)
    int rank, blocks;
    int turn = 0;              // which of the two sums' places is next

    template <class F> __device__ __forceinline__ void each(F f) const {  // f(logit, index)
        const int lane = threadIdx.x & 31, from = (threadIdx.x >> 5) * part;
        const int to = min(from + part, count);
        for (int i = from + lane; i < to; i += 32) f(data[i], first + i);
    }
    __device__ __forceinline__ void join() const {  // the whole cluster
        if (blocks == 1) __syncthreads();
        else cg::this_cluster().sync();
    }
    template <class T> __device__ __forceinline__ T *at(T *p, int block) const {
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
    template <class V, class T> __device__ __forceinline__ uint64_t select(V value, T target) {
        uint64_t mine = 0;
        each([&](float l, int i) { mine += value(l, i); });
        const Sums r = sums(mine);
        const uint64_t t = target(r.all);
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        uint64_t before = r.before;
        for (int w = 0; w < warp; ++w) before += s->warp_sum[w];
        if (before < t && t <= before + s->warp_sum[warp]) {
            const int from = warp * part, to = min(from + part, count);
            for (int i0 = from; i0 < to; i0 += 32) {
                const int i = i0 + lane;
                const uint64_t v = i < to ? value(data[i], first + i) : 0;
                const uint64_t past = before + warp_prefix(v);
                const uint32_t reached = __ballot_sync(0xffffffffu, past >= t);
                if (reached) {
                    if (lane == __ffs(reached) - 1)
                        for (int b = 0; b < blocks; ++b) {
                            auto *f = at(&s->found, b);
                            f->place = first + i, f->value = v;
                        }
                    break;
                }
                before = __shfl_sync(0xffffffffu, past, 31);
            }
        }
        join();
        return r.all;
    }
    // The border at which the running value (1, or the weight) over the tokens up to `limit`, in falling order,
    // reaches `target` (at least 1, at most the sum of all): value(l) is a token's.
    template <bool WEIGHTS, class W>
    __device__ __forceinline__ Border border(Border limit, uint64_t target, float m, float scale, float reach, W weigh) {
        uint32_t lo = 0, hi = 0, bin0 = 0;
        int shift = -1;  // -1: the first histogram, of m - l
        auto first_bin = [&](float l) { return min(static_cast<uint32_t>(max(__float2int_rz((m - l) * scale), 0)), kBins - 1u); };
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
            s->count[threadIdx.x] = 0;
            if (WEIGHTS) s->sum[threadIdx.x] = 0;
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
            uint64_t v = 0;
            uint32_t n = 0;
            for (int b = 0; b < blocks; ++b) {
                n += at(s->count, b)[threadIdx.x];
                if (WEIGHTS) v += at(s->sum, b)[threadIdx.x];
            }
            if (!WEIGHTS) v = n;
            const uint64_t up_to = warp_prefix(v);
            const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
            if (lane == 31) s->warp_sum[warp] = up_to;
            __syncthreads();
            uint64_t before = up_to - v;
            for (int w = 0; w < warp; ++w) before += s->warp_sum[w];
            // bins of the first histogram fall with the logit, those of the others rise: counted from the end
            uint64_t whole = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) whole += s->warp_sum[w];
            if (shift >= 0) before = whole - before - v;
            if (before < target && target <= before + v) s->found.place = threadIdx.x, s->found.before = before, s->found.count = n;
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

template <class T>
__global__ void __launch_bounds__(kThreads, 1) sample_kernel(const SampleParams p) {
    extern __shared__ __align__(16) uint8_t smem[];
    Shared *const s = reinterpret_cast<Shared *>(smem);
    float *const space = reinterpret_cast<float *>(smem + (sizeof(Shared) + 31) / 32 * 32);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t r = blockIdx.x / p.blocks;
    Row row;
    row.s = s;
    row.blocks = p.blocks;
    row.rank = static_cast<int>(blockIdx.x % p.blocks);
    row.part = p.part;
    row.first = row.rank * kWarps * p.part;
    row.count = max(0, min(p.vocab - row.first, kWarps * p.part));
    if (threadIdx.x < 64) s->power[threadIdx.x] = p.power[threadIdx.x];
    if (p.blocks > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    pdl_allow_dependents();
    pdl_wait_prior_grids();

    // ---- the row, as far from a 32-byte boundary here as (eight elements) there
    const T *const src = static_cast<const T *>(p.logits) + r * p.stride + row.first;
    const int pad = static_cast<int>(reinterpret_cast<uintptr_t>(src) / sizeof(T) & 7u);
    row.data = space + pad;
    float top = -INFINITY, low = INFINITY;
    for (int i = 8 * threadIdx.x - pad; i < row.count; i += 8 * kThreads) {
        float v[8];
        if (i >= 0 && i + 8 <= row.count) {
            load8(src + i, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = plain_logit(v[j]);
            float4 *dst = reinterpret_cast<float4 *>(space + pad + i);
            dst[0] = make_float4(v[0], v[1], v[2], v[3]);
            dst[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[j] = -INFINITY;
                if (i + j >= 0 && i + j < row.count) space[pad + i + j] = v[j] = plain_logit(static_cast<float>(src[i + j]));
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            top = fmaxf(top, v[j]);
            if (v[j] > -INFINITY) low = fminf(low, v[j]);
        }
    }
#pragma unroll
    for (int m = 16; m; m >>= 1) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
        low = fminf(low, __shfl_xor_sync(0xffffffffu, low, m));
    }
    if (lane == 0) s->extremes[warp] = make_float2(top, low);
    if (p.blocks > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // the others' memory is there
    __syncthreads();
    if (warp == 0) {
        float2 e = s->extremes[lane];
#pragma unroll
        for (int m = 16; m; m >>= 1) {
            e.x = fmaxf(e.x, __shfl_xor_sync(0xffffffffu, e.x, m));
            e.y = fminf(e.y, __shfl_xor_sync(0xffffffffu, e.y, m));
        }
        if (lane < row.blocks) row.at(s->block_extremes, lane)[row.rank] = e;
    }
    row.join();
    top = -INFINITY, low = INFINITY;
    for (int b = 0; b < row.blocks; ++b) top = fmaxf(top, s->block_extremes[b].x), low = fminf(low, s->block_extremes[b].y);

    // ---- the settings
    const float t = p.temperature ? p.temperature[r] : 1.0f, top_p = p.top_p ? p.top_p[r] : 1.0f, min_p = p.min_p ? p.min_p[r] : 0.0f;
    const int top_k = p.top_k ? p.top_k[r] : 0;
    int32_t token = -1;
    float prob = 0.0f;
    if (top > -INFINITY) {
        if (!(t >= kLeastTemperature) || top_k == 1 || top_p <= 0.0f || min_p > 1.0f) {  // the first alone
            row.select([&](float l, int) -> uint64_t { return l == top; }, [](uint64_t) -> uint64_t { return 1; });
            token = static_cast<int32_t>(s->found.place), prob = 1.0f;
        } else {
            Weigher weigh;
            weigh.power = s->power;
            weigh.m = top;
            weigh.ch = t == INFINITY ? 0.0f : 1.44269502162933349609375f / t;
            weigh.cl = t == INFINITY ? 0.0f : (fmaf(-weigh.ch, t, 1.44269502162933349609375f) + 1.925963033500e-8f) / t;
            // bins per unit of m - l, a power of two
            const float range = fminf(fmaxf(top - low, 0x1p-100f), kRange);
            const float scale = __uint_as_float(__float_as_uint((kBins - 1) / range) & 0x7F800000u);
            Border last{0u, 0xFFFFFFFFu};
            auto kept = [&](float l, int i) {
                const uint32_t key = key_of(l);
                return key > last.key || (key == last.key && static_cast<uint32_t>(i) <= last.index);
            };
            if (top_k > 0 && top_k < p.vocab) last = row.border<false>(last, top_k, top, scale, 0.0f, weigh);
            if (top_p < 1.0f) {
                uint64_t mine = 0;
                row.each([&](float l, int i) {
                    if (kept(l, i)) mine += weigh(l);
                });
                const uint64_t all = row.sums(mine).all;
                bool rest;
                uint64_t target = times(all, top_p, rest);
                target += rest || target == 0 ? 1 : 0;
                // Weights below (1 - top_p) / vocab of the sum are all past the border: their sum is less than what is cut.
                const float least = (1.0f - top_p) * (static_cast<float>(all) * (1.0f / kOne)) / static_cast<float>(p.vocab);
                const float reach = top == INFINITY ? 0.0f : top + (log2f(least) - 0.01f) * t * 0.694f - 1e-6f * fabsf(top);
                last = row.border<true>(last, target, top, scale, reach, weigh);
            }
            const uint64_t least = min_p > 0.0f ? __float2ull_ru(min_p * kOne) : 0;
            const float u = p.uniform[r];
            const uint64_t all = row.select(
                [&](float l, int i) -> uint64_t {
                    if (!kept(l, i)) return 0;
                    const uint64_t w = weigh(l);
                    return w >= least ? w : 0;
                },
                [&](uint64_t all) {
                    bool rest;
                    const uint64_t x = u > 0.0f ? times(all, fminf(u, 1.0f), rest) : 0;
                    return x >= all ? all : x + 1;
                });
            token = static_cast<int32_t>(s->found.place);
            prob = static_cast<float>(s->found.value) / static_cast<float>(all);
        }
    }
    if (row.rank == 0 && threadIdx.x == 0) {
        p.token[r] = token;
        if (p.prob) p.prob[r] = prob;
    }
}

int slice_smem(int part) { return (static_cast<int>(sizeof(Shared)) + 31) / 32 * 32 + (kWarps * part + 8) * 4; }

template <class T> cudaError_t launch(const SampleParams &p, int n, int device, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    const uint64_t bit = 1ull << (device & 63);
    if (!(done.load(std::memory_order_acquire) & bit)) {
        cudaError_t e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        done.fetch_or(bit, std::memory_order_acq_rel);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(n) * p.blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = slice_smem(p.part);
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
    // blocks of a row: as many as its size asks for, and more while there are multiprocessors without a row
    auto part = [&](int blocks) { return (p.vocab + 32 * kWarps * blocks - 1) / (32 * kWarps * blocks) * 32; };
    p.blocks = 1;
    while (p.blocks < kMaxCluster &&
           (slice_smem(part(p.blocks)) > kSmemLimit || (static_cast<int64_t>(n) * p.blocks * 2 <= sms && part(p.blocks) >= 256 && p.blocks < 8)))
        p.blocks *= 2;
    p.part = part(p.blocks);
    return type == QG_F32 ? launch<float>(p, n, device, s) : launch<__half>(p, n, device, s);
}

}  // namespace qg
