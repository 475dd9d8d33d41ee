// shared_attend.cu - attention of new tokens of sequences that share a prefix,
// over the 4-bit paged cache (include/qattn.h, qkv_attend_shared).
//
// All query rows of a key/value head see the whole prefix, so it is taken once
// for all of them: an item is one key/value head and 128 of its rows (token-major
// over the call's tokens and the head's group), its units tiles of 128 prefix
// tokens. The thread blocks share out the units; each stretch of an item in a
// block's part leaves its rows' values, reference and sum in the workspace. Each
// sequence's own tokens go through kv_attend's kernels, which leave theirs there,
// too, and a last kernel joins a row's results in a fixed order.
//
// S = Q K^T and O = P V are tcgen05 products of f16 with f32 sums. A key or value
// is a code of four bits times an f16 scale, 15 bits, and so the exact sum of two
// f16 parts (one alone would be off by 2^-12); f32 queries and, for them, the
// weights are two parts as well. So S takes two products (f32: three, without low
// times low) and O as many. A row's reference, a power of 2 that its weights are
// taken against, rises in steps of 2 at least, so its sums are rescaled a few
// times in all, and O of a tile is read back and added up in f32 registers.
//
// The warps: one copies the units' groups of the cache, one makes their scales
// ready, one issues S, one O; four hold a row's softmax a thread, four its values'
// sums; eight expand codes into operands, four the keys', four the values'. With
// 128 channels a unit is 32 products of 64 cycles, so 2048 cycles for f16, half as
// many again for f32, and 128 KB of operands written; it takes 1.73 us for f16,
// 2.35 for f32. What bounds it is the expanders' chain of instructions (3.8 cycles
// each in turn, 22 a word of eight codes), then the tensor cores. 16 sequences of
// 64 heads on 65521 tokens take 75.5 us: 27 units a block 47, three launches and
// the join 11.5, queries, filling and drain 12, own tokens 6. A call with a short
// prefix is all but that first part (2 sequences on 300 tokens: 17.5 us, where
// kv_attend on whole tables takes 8.4; they meet at about 65000 sequences x tokens
// of 8 key/value heads). What other arrangements measured on the 65521, 76.0 us
// then: one warp for S and O, and eight that expand keys and values in turn, 86.0;
// pieces of a unit's keys and values in three places and three raw pieces ahead 91
// (copies were waited for); whole units' keys in one place, values in another 82.3;
// loops of the expanders unrolled 98 (instructions came from beyond their cache).
#include <algorithm>
#include <atomic>
#include <cfloat>
#include <climits>

#include "packed.cuh"
#include "tc_attend.cuh"

namespace qg {

namespace {

constexpr int kRows = 128;    // of an item
constexpr int kTokens = 128;  // of a unit
constexpr int kMaxParts = 160;

// Roles by warpgroup; the registers of each (a thread) sum up to no more than the launch's.
constexpr int kExpanders = 8;  // warps that turn codes into operands
constexpr int kThreads = (12 + kExpanders) * 32;
constexpr int kLaunchRegs = 96, kIssueRegs = 40, kSoftmaxRegs = 136, kSumRegs = 168, kExpandRegs = 64;
static_assert(128 * (kIssueRegs + kSoftmaxRegs + kSumRegs) + 32 * kExpanders * kExpandRegs <= kThreads * kLaunchRegs, "registers");

// Tensor memory: S of even and odd tiles (the weights over its first half), O, the queries, the weights' low parts.
constexpr uint32_t kTmemCols = 512, kTmemO = 256, kTmemQ = 384, kTmemLow = 448;
// log2 of the largest weight, and of the largest when the reference is set. Near f16's end its parts still hold a weight of
// 2^-39 of the largest, and the largest itself is most often a power of 2, without a rounding (f16 results of 120 rows on
// 4099 tokens differ from plain f32's by 1.4e-4; with 7 instead of 14, 2.1e-4). Steps of 2 come seldom, since a row's
// largest score soon changes little: 75.5 us for the longest case, 75.4 with 13, 75.1 with 7 and steps of 2^7.
constexpr float kHigh = 15.0f, kLow = 14.0f;

template <int D, int TERMS> struct Shape {
    using G = KvGroup<D>;
    // Operands in slices, so that the tensor cores read one of a unit while the next is made: of keys 64 channels of all
    // tokens, of values all channels of 64 tokens (D = 64: all of them), each as a high and a low part of 128-byte rows of
    // 64 channels. Two places for each kind. Queries pass through the key slices' places on their way to tensor
    // memory, f32's low parts have a place of their own.
    static constexpr int kSlices = D / 64, kPart = 128 * 128, kSlice = 2 * kPart;
    static constexpr int kSliceTokens = kTokens / kSlices;     // of a slice of values
    static constexpr int kOffV = 2 * kSlice, kOffLow = 4 * kSlice;
    static constexpr int kRaw = kTokens / 16 * G::kBytes;      // a unit's groups as they lie in the cache
    static constexpr int kOffRaw = kOffLow + (TERMS == 2 ? kSlices * kPart : 0);
    static constexpr int kSlots = D == 128 && TERMS == 2 ? 3 : 5;  // units' raw groups
    static constexpr int kOffBars = kOffRaw + kSlots * kRaw;
    static constexpr int kOffKeep = kOffBars + 512;            // [tile % 4][row]: what the sums before a tile are multiplied by
    static constexpr int kOffFactor = kOffKeep + 4 * kRows * 4;  // [stretch % 4][row]: a row's scores as powers of 2
    static constexpr int kSmem = kOffFactor + 4 * kRows * 4 + 1024;  // (alignment)
    static_assert(kSmem <= kSmemLimit, "shared memory");
};

// The prefix's length, checked, and how the thread blocks share the units: each item's among as many parts as there are for
// it, or, where that would leave a part kRestart units more, all items' as one list in equal parts. A part that ends in one
// item and begins the next drains and fills its pipeline again, and takes other queries: 14000 cycles, as many as 4 units.
constexpr int kRestart = 3;
struct Units {
    int len, tiles, per_item;  // tokens, units of an item, parts of an item (0: a list)
    int64_t all, share;        // of all items, of a part
    __device__ __forceinline__ Units(const SharedParams &p, int parts) {
        len = __ldg(p.prefix_len);
        const int64_t room = p.prefix_pages * static_cast<int64_t>(p.own.c.page_size);
        if (len < 0 || len > room) {
            record_error(p.own.err, kErrBadIndex);
            len = len < 0 ? 0 : static_cast<int>(room);
        }
        tiles = static_cast<int>((static_cast<uint32_t>(len) + kTokens - 1) / kTokens);
        const int64_t items = static_cast<int64_t>(p.own.c.n_heads) * p.row_tiles;
        all = items * tiles;
        per_item = 0;
        if (items <= parts) {  // (below 2^32 units)
            const uint32_t n = static_cast<uint32_t>(items), m = parts / n;
            const uint32_t of_one = (tiles + m - 1) / m, of_all = (static_cast<uint32_t>(all) + parts - 1) / parts;
            per_item = of_one <= of_all + kRestart ? static_cast<int>(m) : 0;
            share = per_item > 0 ? of_one : of_all;
        } else {
            share = (all + parts - 1) / parts;
        }
        if (share < 1) share = 1;
    }
};
// A stretch's place is its part's and its item's number: both rise, one of them at least from stretch to stretch.
__host__ __device__ constexpr int64_t stretch_floats(int d) { return static_cast<int64_t>(kRows) * (d + 2); }

// A stretch's rows hold the channels in the order in which the value codes lie in the cache: place 8 (8 h + u) + 2 j + b
// holds channel 64 h + 32 b + 2 u + {0, 1, 16, 17}[j].

// Walks a part's stretches, alike in every role.
struct Stretch {
    int units;                  // still to come
    int item, tile, n = 0, index = -1;
    __device__ __forceinline__ Stretch(const Units &all, int64_t part) {
        if (all.per_item > 0) {
            item = static_cast<int>(part) / all.per_item;
            tile = min((static_cast<int>(part) - item * all.per_item) * static_cast<int>(all.share), all.tiles);
            units = static_cast<int64_t>(item) * all.tiles < all.all ? min(static_cast<int>(all.share), all.tiles - tile) : 0;
        } else {
            const int64_t u = part * all.share;
            units = static_cast<int>(max(min(all.share, all.all - u), static_cast<int64_t>(0)));
            item = units <= 0 ? 0 : all.all <= UINT_MAX ? static_cast<int>(static_cast<uint32_t>(u) / all.tiles) : static_cast<int>(u / all.tiles);
            tile = static_cast<int>(u - static_cast<int64_t>(item) * all.tiles);
        }
    }
    __device__ __forceinline__ bool next(const Units &all) {
        if (units == 0) return false;
        if (index >= 0) ++item, tile = 0;
        n = min(units, all.tiles - tile);
        units -= n;
        ++index;
        return true;
    }
    // Unit by unit instead.
    __device__ __forceinline__ void step(const Units &all) {
        if (++tile == all.tiles) ++item, tile = 0;
    }
};

// code - 8 in f16 of the low (high) nibbles of bytes 0 and 2.
__device__ __forceinline__ __half2 low_codes(uint32_t w) {
    const uint32_t x = (w & 0x000F000Fu) | 0x64006400u, y = 0x64086408u;  // 1024 + c, 1032
    return __hsub2(*reinterpret_cast<const __half2 *>(&x), *reinterpret_cast<const __half2 *>(&y));
}
__device__ __forceinline__ __half2 high_codes(uint32_t w) {
    const uint32_t x = (w & 0x00F000F0u) | 0x64006400u, y = 0x2C002C00u, z = 0xD480D480u;  // (1024 + 16 c) / 16 - 72
    return __hfma2(*reinterpret_cast<const __half2 *>(&x), *reinterpret_cast<const __half2 *>(&y), *reinterpret_cast<const __half2 *>(&z));
}
__device__ __forceinline__ uint32_t bits(__half2 h) { return *reinterpret_cast<const uint32_t *>(&h); }

template <int NB> __device__ __forceinline__ void ld_words(const uint8_t *p, uint32_t (&w)[NB]) {
    if (NB == 4) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        w[0] = v.x, w[1] = v.y, w[NB - 2] = v.z, w[NB - 1] = v.w;
    } else {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        w[0] = v.x, w[1] = v.y;
    }
}
// NB f16 as NB/2 words.
template <int NB> __device__ __forceinline__ void ld_halves(const uint8_t *p, uint32_t (&w)[NB / 2]) {
    if (NB == 4) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        w[0] = v.x, w[NB / 2 - 1] = v.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t *>(p);
    }
}

// One word of a row: eight values as two f16 parts, 16 bytes of each: the value rounded to f16, and what that leaves with
// its sign turned (minus is the scale's negative), which the products turn back. Above f16's end two parts hold it exactly
// (four bits times eleven). The low part is at most 2^-11 of the high one: f32 drops low times low.
__device__ __forceinline__ void expand_word(uint32_t w, __half2 scale, __half2 minus, uint8_t *high, uint8_t *low) {
    const __half2 c[4] = {low_codes(w), low_codes(w >> 8), high_codes(w), high_codes(w >> 8)};
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 x = __hmul2(c[i], scale);
        h[i] = bits(x);
        l[i] = bits(__hfma2(c[i], minus, x));
    }
    *reinterpret_cast<uint4 *>(high) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4 *>(low) = make_uint4(l[0], l[1], l[2], l[3]);
}

// Makes a unit's raw scales (keys' or values') ready: 0 for tokens that do not count (rows past `rows`, groups in no
// page), infinities as NaN, and all times the power of two that takes the largest to 2^8 .. 2^9 (f16 exponent fields),
// whose exponent is returned. The unit's values are then below 2^13 and exact down to 2^-33 of that. One warp: a lane
// has two words of four tokens in two places, which its neighbours' follow.
template <int D> __device__ __forceinline__ int prepare_scales(uint8_t *scales, int rows, uint32_t groups) {
    constexpr int kChunks = kTokens * (D / 16) / 512, kPer = 256 / D;  // 16-byte chunks of a lane, tokens of one
    const int lane = threadIdx.x & 31;
    uint8_t *const at = scales + lane / (D / 16) * KvGroup<D>::kBytes + lane % (D / 16) * 16;
    constexpr int kStep = 512 / D * KvGroup<D>::kBytes;
    uint32_t x[kChunks][4], m = 0;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        const uint4 v = *reinterpret_cast<const uint4 *>(at + i * kStep);
        x[i][0] = v.x, x[i][1] = v.y, x[i][2] = v.z, x[i][3] = v.w;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const int row = (32 * i + lane) * kPer + w * kPer / 4;
            if (row >= rows || !((groups >> (row >> 4)) & 1)) x[i][w] = 0;
            m = __vmaxu2(m, x[i][w] & 0x7FFF7FFFu);
        }
    }
    const uint32_t most = __reduce_max_sync(0xffffffffu, max(m & 0xFFFFu, m >> 16)) >> 10;
    const int e = 23 - static_cast<int>(most == 0 ? 1 : most);
    // 2^e in two factors of f16's range
    const __half2 up = __float2half2_rn(__uint_as_float(static_cast<uint32_t>(127 + min(e, 15)) << 23));
    const __half2 more = __float2half2_rn(__uint_as_float(static_cast<uint32_t>(127 + max(e - 15, 0)) << 23));
    const __half2 zero = __float2half2_rn(0.0f);
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        uint32_t y[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const __half2 d = *reinterpret_cast<const __half2 *>(&x[i][w]);
            y[w] = bits(__hfma2(d, zero, __hmul2(__hmul2(d, up), more)));
        }
        *reinterpret_cast<uint4 *>(at + i * kStep) = make_uint4(y[0], y[1], y[2], y[3]);
    }
    return e;
}

__device__ __forceinline__ void copy16_or_zeros(uint32_t dst, const void *src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void tc_st4(uint32_t taddr, const uint32_t (&v)[4]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}

// Bounded wait that gives up once another thread of the block has set the abort flag. Most are short: the clock is read
// every 64 polls only, and the loop is kept small.
template <int NS> __device__ __forceinline__ bool poll_wait(uint32_t bar, uint32_t parity, const volatile int *abort_flag) {
    uint64_t t0 = 0;
#pragma unroll 1
    for (uint32_t i = 1; i < kWaitLimitPolls; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if (NS > 0) __nanosleep(NS);
        if ((i & 63u) == 0) {
            const uint64_t now = global_timer_ns();
            if (i == 64) t0 = now;
            if (*abort_flag || now - t0 > kWaitLimitNs) return false;
        }
    }
    return false;
}

// A wait tells a phase from the next by its parity alone, so no waiter may come to one before its predecessor is complete,
// nor after its successor is. Each waits for every phase of its barriers in turn (the key warps twice for the last slice's
// before a stretch), and for the next one of the same barrier something is needed that the waiter does only afterwards.
template <int D, class T>
__global__ void __launch_bounds__(kThreads, 1) prefix_kernel(const SharedParams p) {
    constexpr int TERMS = sizeof(T) == 4 ? 2 : 1, NB = D / 32;
    using Sh = Shape<D, TERMS>;
    using G = KvGroup<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *const smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);  // (the swizzle's atoms are 1024 bytes)
    const uint32_t base = smem_addr(smem), bars = base + Sh::kOffBars;
    const uint32_t raw_full = bars, raw_empty = raw_full + 8 * Sh::kSlots, scaled_k = raw_empty + 8 * Sh::kSlots;
    const uint32_t scaled_v = scaled_k + 8 * Sh::kSlots, s_full = scaled_v + 8 * Sh::kSlots, p_ready = s_full + 16, o_full = p_ready + 16;
    const uint32_t o_free = o_full + 16, mfinal = o_free + 8, q_open = mfinal + 16, q_staged = q_open + 8;
    const uint32_t ready = q_staged + 8, free = ready + 32;  // of the slices' places: two of keys, two of values; up to 39 barriers: 312 bytes
    uint8_t *const words = smem + Sh::kOffBars + 320;
    uint32_t *const tmem_slot = reinterpret_cast<uint32_t *>(words);
    volatile int *const abort_flag = reinterpret_cast<volatile int *>(words + 4);
    volatile int *const groups = reinterpret_cast<volatile int *>(words + 16);     // [tile % 16]: its groups that lie in a page
    // [tile % 8]: the scales' exponents (the warp that finds them is five tiles ahead of those that expand values at most,
    // and these two ahead of the values' sums)
    volatile int *const k_exp = reinterpret_cast<volatile int *>(words + 80);
    volatile int *const v_exp = reinterpret_cast<volatile int *>(words + 112);
    volatile float *const keep = reinterpret_cast<volatile float *>(smem + Sh::kOffKeep);
    volatile float *const factor = reinterpret_cast<volatile float *>(smem + Sh::kOffFactor);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const KvAttendParams &a = p.own;

    if (threadIdx.x == 0) {
        for (int i = 0; i < Sh::kSlots; ++i) {
            mbar_init(raw_full + 8 * i, 1);
            mbar_init(raw_empty + 8 * i, kExpanders);
            mbar_init(scaled_k + 8 * i, 1);
            mbar_init(scaled_v + 8 * i, 1);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(s_full + 8 * x, 1);
            mbar_init(p_ready + 8 * x, 4);
            mbar_init(o_full + 8 * x, 1);
            mbar_init(mfinal + 8 * x, 1);
        }
        mbar_init(o_free, 4);
        mbar_init(q_staged, kExpanders);
        mbar_init(q_open, kExpanders / 2);
        for (int i = 0; i < 4; ++i) {
            mbar_init(ready + 8 * i, kExpanders / 2);
            mbar_init(free + 8 * i, 1);
        }
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        tc_alloc(smem_addr(tmem_slot), kTmemCols);
        tc_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait_prior_grids();
    pdl_allow_dependents();
    const Units units(p, gridDim.x);
    Stretch st(units, blockIdx.x);
    const int n_units = st.units;
    // A wait of a whole warp that gives up sets the abort flag, with which the others give up soon.
    auto failed = [&](int32_t code) {
        if (lane == 0) record_error(a.err, code);
        *abort_flag = 1;
        __syncwarp();
    };
    auto wait = [&](uint32_t bar, uint32_t parity) {
        return static_cast<bool>(__all_sync(0xffffffffu, poll_wait<20>(bar, parity & 1u, abort_flag)));
    };

    if (warp < 4) {
        fewer_registers<kIssueRegs>();
        if (warp == 0) {
            // ---------------- copies: a unit's groups
            bool ok = true;
            int n = 0;
#pragma unroll 1
            for (; n < n_units; ++n, st.step(units)) {
                // this lane's group, as a byte offset in the cache; -1: none
                int64_t src = -1;
                const int t = st.tile * kTokens + 16 * (lane & 7);
                if (t < units.len) {
                    const int page = __ldg(p.prefix_table + t / a.c.page_size);
                    if (page < 0 || page >= a.c.n_pages) record_error(a.err, kErrBadIndex);
                    else src = ((static_cast<int64_t>(page) * a.c.n_heads + st.item / p.row_tiles) * a.c.page_groups + t % a.c.page_size / 16) * G::kBytes;
                }
                const int slot = n % Sh::kSlots;
                if (n >= Sh::kSlots) ok = wait(raw_empty + 8 * slot, n / Sh::kSlots - 1);
                if (!ok) break;
                const uint32_t valid = __ballot_sync(0xffffffffu, src >= 0) & 255u;
                const uint32_t dst = base + Sh::kOffRaw + slot * Sh::kRaw, bar = raw_full + 8 * slot;
                if (lane == 0) {
                    groups[n % 16] = static_cast<int>(valid);
                    mbar_arrive_expect_tx(bar, __popc(valid) * G::kBytes);
                }
                __syncwarp();
                if (src >= 0 && lane < 8) bulk_copy_g2s_plain(dst + lane * G::kBytes, a.c.data + src, G::kBytes, bar);
            }
            if (!ok) failed(kErrProducerWait);
            // leave no copy in flight into this block's shared memory
            bool landed = true;
            for (int k = n > Sh::kSlots ? n - Sh::kSlots : 0; k < n; ++k)
                landed = mbar_wait_bounded(raw_full + 8 * (k % Sh::kSlots), (k / Sh::kSlots) & 1) && landed;
            if (!landed) record_error(a.err, kErrDrainWait);
            __syncwarp();
        } else if (warp != 2) {
            // ---------------- products (the whole warp, one lane issues): S warp 1, O warp 3. A warp that issues stands
            // still while the tensor cores' short queue is full, so that with one warp for both its waits and commits
            // between the products would leave them idle.
            const uint32_t issue = lane == 0;
            constexpr uint32_t kIdS = tc_idesc_f16(128, kTokens), kIdO = tc_idesc_f16(128, D) | kIdescNMajorB;
            constexpr uint32_t kPart = Sh::kPart / 16;
            auto tight = [&](uint32_t bar, uint32_t parity) { return static_cast<bool>(__all_sync(0xffffffffu, poll_wait<0>(bar, parity & 1u, abort_flag))); };
            bool ok = true;
            // Small terms first: what the tensor cores cut off at each sum is then of the small ones. For f32 that holds
            // over both slices of a unit (slice by slice its error was up to twice as large), which wait for each other
            // then; f16 results, rounded to 2^-11, take them as they come.
            // (loops rolled: what runs once a unit comes from instruction memory each time)
            auto of_unit = [&](int i, uint32_t bars, auto &&low, auto &&high) {
                auto come = [&](int h) {
                    ok = ok && tight(bars + 8 * ((i + h) & 1), (i + h) >> 1);
                    tc_fence_after();
                    return ok;
                };
                if (TERMS == 2)
#pragma unroll 1
                    for (int h = 0; h < Sh::kSlices; ++h) {
                        if (!come(h)) return;
                        low(h, (i + h) & 1);
                    }
#pragma unroll 1
                for (int h = 0; h < Sh::kSlices; ++h) {
                    if (TERMS == 1) {
                        if (!come(h)) return;
                        low(h, (i + h) & 1);
                    }
                    high(h, (i + h) & 1);
                    commit(issue, bars + 32 + 8 * ((i + h) & 1));  // (free)
                }
            };
            if (warp == 1) {
                for (int n = 0; ok && n < n_units; ++n) {
                    const uint32_t s = tmem + 128 * (n & 1);
                    ok = n < 2 || tight(o_full + 8 * (n & 1), (n - 2) >> 1);
                    of_unit(
                        n * Sh::kSlices, ready,
                        [&](int h, int place) {
                            const uint32_t k = desc_lo(base + place * Sh::kSlice, 1);
                            if (TERMS == 2) mma_s<64>(issue, s, desc_lo(base + Sh::kOffLow + h * Sh::kPart, 1), k, kIdS, kDescHi, h > 0);
                            mma_s_tm<64>(issue, s, tmem + kTmemQ + 32 * h, k + kPart, kIdS | kIdescMinusB, kDescHi, TERMS == 2 || h > 0);
                        },
                        [&](int h, int place) { mma_s_tm<64>(issue, s, tmem + kTmemQ + 32 * h, desc_lo(base + place * Sh::kSlice, 1), kIdS, kDescHi, 1); });
                    if (ok) commit(issue, s_full + 8 * (n & 1));
                }
            } else {
                for (int n = 0; ok && n < n_units; ++n) {
                    const uint32_t w = tmem + 128 * (n & 1), w_low = tmem + kTmemLow;
                    auto desc = [&](int place) { return desc_lo(base + Sh::kOffV + place * Sh::kSlice, Sh::kSliceTokens * 128 / 16); };
                    ok = tight(p_ready + 8 * (n & 1), n >> 1) && (n == 0 || tight(o_free, n - 1));
                    of_unit(
                        n * Sh::kSlices, ready + 16,
                        [&](int h, int place) {
                            const uint32_t v = desc(place);
                            if (TERMS == 2) mma_pv<Sh::kSliceTokens>(issue, tmem + kTmemO, w_low + 32 * h, v, kIdO, h > 0, kDescHi);
                            mma_pv<Sh::kSliceTokens>(issue, tmem + kTmemO, w + 32 * h, v + kPart, kIdO | kIdescMinusB, TERMS == 2 || h > 0, kDescHi);
                        },
                        [&](int h, int place) { mma_pv<Sh::kSliceTokens>(issue, tmem + kTmemO, w + 32 * h, desc(place), kIdO, 1, kDescHi); });
                    if (ok) commit(issue, o_full + 8 * (n & 1));
                }
            }
            if (!ok) failed(kErrConsumerWait);
            // every product complete before tensor memory is freed, after a wait that gave up, too
            const uint32_t end = mfinal + 4 * (warp & 2);
            commit(issue, end);
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(end, 0)) && issue) record_error(a.err, kErrDrainWait);
            __syncwarp();
        } else {
            // ---------------- scales, in place
            bool ok = true;
#pragma unroll 1
            for (int n = 0; n < n_units; ++n, st.step(units)) {
                const int slot = n % Sh::kSlots;
                ok = wait(raw_full + 8 * slot, n / Sh::kSlots);
                if (!ok) break;
#pragma unroll 1
                for (int values = 0; values < 2; ++values) {
                    const int e = prepare_scales<D>(smem + Sh::kOffRaw + slot * Sh::kRaw + (values ? G::kVS : G::kKS),
                                                    min(kTokens, units.len - st.tile * kTokens), static_cast<uint32_t>(groups[n % 16]));
                    fence_proxy_async_smem();  // (the next copy to this place comes after these writes)
                    __syncwarp();
                    if (lane == 0) {
                        (values ? v_exp : k_exp)[n & 7] = e;
                        mbar_arrive((values ? scaled_v : scaled_k) + 8 * slot);
                    }
                }
            }
            if (!ok) failed(kErrConsumerWait);
        }
    } else if (warp < 8) {
        // ---------------- softmax: thread = row = tensor-memory lane
        more_registers<kSoftmaxRegs>();
        const int row = 32 * (warp & 3) + lane;
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        bool ok = true;
        int n = 0;
        while (ok && st.next(units)) {
            float ref = -INFINITY, sum = 0.0f;
            for (int j = 0; j < st.n; ++j, ++n) {
                ok = wait(s_full + 8 * (n & 1), n >> 1);
                if (!ok) break;
                tc_fence_after();
                const uint32_t s_t = tmem + lanes + 128 * (n & 1), low_t = tmem + lanes + kTmemLow;
                const int rows = min(kTokens, units.len - (st.tile + j) * kTokens);
                const uint32_t in_page = static_cast<uint32_t>(groups[n % 16]);
                const bool full = rows == kTokens && in_page == 255u;
                const float c = fminf(fmaxf(factor[(st.index & 3) * kRows + row] * __uint_as_float(static_cast<uint32_t>(127 - k_exp[n & 7]) << 23), 1e-37f), FLT_MAX);
                auto load = [&](int i, uint32_t (&v)[32]) {
                    tm_ld32(s_t + 32 * i, v);
                    tm_wait_ld(v);
                    if (!full) {
                        uint32_t seen = (in_page >> (2 * i) & 1u ? 0x0000FFFFu : 0u) | (in_page >> (2 * i) & 2u ? 0xFFFF0000u : 0u);
                        seen &= rows >= 32 * i + 32 ? 0xFFFFFFFFu : rows <= 32 * i ? 0u : (1u << (rows - 32 * i)) - 1;
#pragma unroll
                        for (int q = 0; q < 32; ++q)
                            if (!(seen >> q & 1u)) v[q] = 0xFF800000u;
                    }
                };
                // (rolled loops throughout: the roles of a scheduler run through as many pieces of code, and unrolled ones
                // came from instruction memory each time)
                float top = -INFINITY;
#pragma unroll 1
                for (int i = 0; i < 4; ++i) {
                    uint32_t v[32];
                    load(i, v);
                    float m[2] = {top, __uint_as_float(v[0])};
#pragma unroll
                    for (int q = 1; q < 31; q += 2) m[q / 2 & 1] = fmaxf(fmaxf(m[q / 2 & 1], __uint_as_float(v[q])), __uint_as_float(v[q + 1]));
                    top = fmaxf(fmaxf(m[0], m[1]), __uint_as_float(v[31]));
                }
                top *= c;
                float down = 1.0f;
                if (top - kHigh > ref) {
                    const float next = fmaxf(top - kLow, -FLT_MAX);
                    down = exp2_approx(ref - next);
                    ref = next;
                    sum *= down;
                }
                keep[(n & 3) * kRows + row] = down;
                const float r = ref == -INFINITY ? 0.0f : ref;  // (no token seen yet: weights of 0)
                const float2 c2 = make_float2(c, c), r2 = make_float2(-r, -r);
                if (TERMS == 2 && n > 0) ok = wait(o_full + 8 * ((n - 1) & 1), (n - 1) >> 1);  // the low parts' place is one
                if (!ok) break;
                // Weights are summed unit by unit, as the values are: what a long sum rounds is then the same above and below
                // the line. (In one sum, 2^18 equal weights beside one of 2^21 times their size were off by 1.2e-3.)
                float2 of_unit = make_float2(0.0f, 0.0f);
#pragma unroll 1
                for (int i = 0; i < 4; ++i) {
                    uint32_t v[32], w[16], w_low[16];
                    load(i, v);
#pragma unroll
                    for (int q = 0; q < 16; ++q) {
                        float2 e = ffma2(make_float2(__uint_as_float(v[2 * q]), __uint_as_float(v[2 * q + 1])), c2, r2);
                        e.x = exp2_approx(e.x), e.y = exp2_approx(e.y);
                        of_unit = fadd2(of_unit, e);
                        w[q] = pack_half2(e.x, e.y);
                        if (TERMS == 2) {
                            const float2 h = unpack_half2(w[q]);
                            w_low[q] = pack_half2(e.x - h.x, e.y - h.y);
                        }
                    }
                    tc_st16(s_t + 16 * i, w);
                    if (TERMS == 2) tc_st16(low_t + 16 * i, w_low);
                }
                sum += of_unit.x + of_unit.y;
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_ready + 8 * (n & 1));
            }
            if (ok)
                reinterpret_cast<float2 *>(p.stretches + (blockIdx.x + static_cast<int64_t>(st.item)) * stretch_floats(D) + kRows * D)[row] =
                    make_float2(ref, sum);
        }
        if (!ok) failed(kErrConsumerWait);
    } else if (warp < 12) {
        // ---------------- the values' sums: a row a thread, in registers (in tensor memory every addition cuts off)
        more_registers<kSumRegs>();
        const int row = 32 * (warp & 3) + lane;
        const uint32_t o_t = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + kTmemO;
        bool ok = true;
        int n = 0;
        while (ok && st.next(units)) {
            float2 o[D / 2];
#pragma unroll
            for (int i = 0; i < D / 2; ++i) o[i] = make_float2(0.0f, 0.0f);
            for (int j = 0; j < st.n; ++j, ++n) {
                ok = wait(o_full + 8 * (n & 1), n >> 1);
                if (!ok) break;
                tc_fence_after();
                const float f = keep[(n & 3) * kRows + row], u = __uint_as_float(static_cast<uint32_t>(127 - v_exp[n & 7]) << 23);
                const float2 u2 = make_float2(u, u);
                if (__any_sync(0xffffffffu, f != 1.0f)) {
                    const float2 f2 = make_float2(f, f);
#pragma unroll
                    for (int i = 0; i < D / 2; ++i) o[i] = fmul2(o[i], f2);
                }
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    uint32_t v[32];
                    tm_ld32(o_t + 32 * i, v);
                    tm_wait_ld(v);
                    if (i + 1 == D / 32) {  // all of O has been read
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(o_free);
                    }
#pragma unroll
                    for (int q = 0; q < 16; ++q)
                        o[16 * i + q] = ffma2(make_float2(__uint_as_float(v[2 * q]), __uint_as_float(v[2 * q + 1])), u2, o[16 * i + q]);
                }
            }
            if (!ok) break;
            float *out = p.stretches + (blockIdx.x + static_cast<int64_t>(st.item)) * stretch_floats(D) + row * D;
#pragma unroll
            for (int i = 0; i < D / 2; i += 4) {
                const uint32_t w[8] = {__float_as_uint(o[i].x), __float_as_uint(o[i].y), __float_as_uint(o[i + 1].x), __float_as_uint(o[i + 1].y),
                                       __float_as_uint(o[i + 2].x), __float_as_uint(o[i + 2].y), __float_as_uint(o[i + 3].x), __float_as_uint(o[i + 3].y)};
                store32(out + 2 * i, w, true);
            }
        }
        if (!ok) failed(kErrConsumerWait);
    } else {
        // ---------------- codes to operands
        fewer_registers<kExpandRegs>();
        // four warps the keys', four the values': what one side waits for (operands that are on their way to shared memory,
        // places) does not keep the other
        const int w = warp - 12;
        const bool values = w >= kExpanders / 2;
        constexpr bool kHalves = D == 128;
        // Rows of a warp, 32 apart: so that eight lanes that store together have eight different chunk places. A lane takes
        // four words at a time: of keys those of blocks 2 h and 2 h + 1 (h the slice) in two rows, to chunks part and
        // 4 + part; of values two units of both block pairs in one row, or of D = 64's one in two.
        const int part = lane & 3, x = lane >> 2, row_x = 8 * (w & 3) + (values ? x : (x & 1) * 4 + (x >> 1)), vr = kv_value_row(row_x & 15);
        const int group_at = (row_x >> 4) * G::kBytes;
        const int codes_at = group_at + (values ? G::kV + vr * G::kRow + (part ^ (vr & 2)) * (4 * NB) : (row_x & 15) * G::kRow + part * (4 * NB));
        const int scales_at = group_at + (values ? G::kVS : G::kKS) + (row_x & 15) * G::kScaleRow;
        const int first = row_x * 128 + (((values ? 2 * part : part) ^ (row_x & 7)) << 4);
        const int second = row_x * 128 + (((values ? 2 * part + 1 : part + 4) ^ (row_x & 7)) << 4);
        const bool pairs = kHalves && values;  // both block pairs, and a row in two turns
        const uint32_t even = values ? 0x3210 : 0x1010, odd = values ? 0x3210 : 0x3232;
        const uint32_t my_ready = ready + (values ? 16 : 0), my_free = free + (values ? 16 : 0), my_scaled = values ? scaled_v : scaled_k;
        bool ok = true;
        int n = 0;
        // slice i, half h of unit n
        auto expand = [&](int i, int h) {
            const int slot = n % Sh::kSlots;
            if (h == 0) ok = wait(my_scaled + 8 * slot, n / Sh::kSlots) && wait(raw_full + 8 * slot, n / Sh::kSlots);
            if (ok && i >= 2) ok = wait(my_free + 8 * (i & 1), (i - 2) >> 1);
            if (!ok) return;
            const uint8_t *const raw = smem + Sh::kOffRaw + slot * Sh::kRaw;
            uint8_t *const to = smem + (values ? Sh::kOffV : 0) + (i & 1) * Sh::kSlice;
            const uint8_t *codes = raw + codes_at + (pairs ? h * (4 * G::kBytes) : kHalves ? 8 * h : 0);
            const uint8_t *scales = raw + scales_at + (pairs ? h * (4 * G::kBytes) : kHalves ? 4 * h : 0);
            uint32_t c[2][2], d[2], c_next[2][2], d_next[2];
            auto load = [&]() {
                ld_words<2>(codes, c_next[0]);
                ld_words<2>(codes + (pairs ? 8 : 2 * G::kBytes), c_next[1]);
                d_next[0] = *reinterpret_cast<const uint32_t *>(scales);
                d_next[1] = *reinterpret_cast<const uint32_t *>(scales + (pairs ? 4 : 2 * G::kBytes));
                codes += pairs ? 2 * G::kBytes : 4 * G::kBytes, scales += pairs ? 2 * G::kBytes : 4 * G::kBytes;
            };
            uint8_t *a = to + first, *b = to + (pairs ? first + Sh::kSliceTokens * 128 : second);
            const int next = pairs ? second - first : 32 * 128;  // (of pairs b - a is the same for both)
            load();
#pragma unroll 1
            for (int s = 0; s < 2; ++s) {
                uint32_t minus[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    c[k][0] = c_next[k][0], c[k][1] = c_next[k][1], d[k] = d_next[k];
                    minus[k] = d[k] ^ 0x80008000u;
                }
                if (s == 0) load();
                auto two = [](uint32_t x, uint32_t select) {
                    x = __byte_perm(x, 0, select);
                    return *reinterpret_cast<const __half2 *>(&x);
                };
                const int x = pairs ? 1 : 0;  // (the scales of the first row's second word and of the second's first)
                expand_word(c[0][0], two(d[0], even), two(minus[0], even), a, a + Sh::kPart);
                expand_word(c[0][1], two(x ? d[1] : d[0], odd), two(x ? minus[1] : minus[0], odd), b, b + Sh::kPart);
                expand_word(c[1][0], two(x ? d[0] : d[1], even), two(x ? minus[0] : minus[1], even), a + next, a + next + Sh::kPart);
                expand_word(c[1][1], two(d[1], odd), two(minus[1], odd), b + next, b + next + Sh::kPart);
                a += pairs ? 32 * 128 : 64 * 128, b += pairs ? 32 * 128 : 64 * 128;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                if (h == Sh::kSlices - 1) mbar_arrive(raw_empty + 8 * slot);
                mbar_arrive(my_ready + 8 * (i & 1));
            }
        };
        while (ok && st.next(units)) {
            // ---- the stretch's queries, in the keys' order of channels: they come through the key slices' places, once the
            // last one's products are complete, as the key warps see
            const int i0 = n * Sh::kSlices;
            if (!values) {
                ok = (i0 < 2 || wait(free + 8 * (i0 & 1), (i0 - 2) >> 1)) && (i0 < 1 || wait(free + 8 * ((i0 - 1) & 1), (i0 - 1) >> 1));
                if (ok && lane == 0) mbar_arrive(q_open);
            }
            if (ok) ok = wait(q_open, st.index);
            if (!ok) break;
            const int head = st.item / p.row_tiles, row0 = st.item % p.row_tiles * kRows;
            constexpr int kRowBytes = D * static_cast<int>(sizeof(T)), kChunks = kRowBytes / 16, kAtOnce = kExpanders * 32 / kChunks;
#pragma unroll 1
            for (int r = w * (32 / kChunks) + lane / kChunks; r < kRows; r += kAtOnce) {
                const int k = lane % kChunks, row = row0 + r, tok = row / a.group;
                const bool there = tok < a.n_tok;
                const T *src = static_cast<const T *>(a.q);
                if (there) src += tok * a.q_stride + (static_cast<int64_t>(head) * a.group + row - tok * a.group) * D + k * (16 / sizeof(T));
                copy16_or_zeros(base + r * kRowBytes + ((k ^ (r & 7)) << 4), src, there);
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(q_staged);
            ok = wait(q_staged, 0);
            if (!ok) break;
            if (w < 4 * Sh::kSlices) {  // 64 channels of a row a thread
                const int r = 32 * (w & 3) + lane, h = w >> 2;
                const uint8_t *const mine = smem + r * kRowBytes;
                auto chunk = [&](int k) { return mine + ((k ^ (r & 7)) << 4); };
                float up = a.scale < 0.0f ? -1.0f : 1.0f, back = fabsf(a.scale) * 1.4426950408889634f;
                if (TERMS == 2) {  // the largest magnitude to 2^10 .. 2^11
                    float big = 0.0f;
#pragma unroll 2
                    for (int k = 0; k < kChunks; ++k) {
                        const float4 x = *reinterpret_cast<const float4 *>(chunk(k));
                        big = fmaxf(fmaxf(big, fmaxf(fabsf(x.x), fabsf(x.y))), fmaxf(fabsf(x.z), fabsf(x.w)));
                    }
                    int e = static_cast<int>(__float_as_uint(big) >> 23) - 127;
                    if (e == 128) e = 0;         // infinities
                    if (e < -117) e = -117;      // (2^(10 - e) is an f32)
                    up *= __uint_as_float(static_cast<uint32_t>(137 - e) << 23);
                    back *= __uint_as_float(static_cast<uint32_t>(127 + e) << 23) * 0x1p-10f;
                }
                if (h == 0) factor[(st.index & 3) * kRows + r] = fmaxf(back, 1e-37f);  // never 0, which times -inf would be NaN
#pragma unroll 1
                for (int i = 0; i < 8; ++i) {
                    const int e = 64 * h + 32 * (i >> 2) + 4 * (i & 3);  // the first element
                    float x[8];
                    if constexpr (TERMS == 2) {
                        const float4 y = *reinterpret_cast<const float4 *>(chunk(e / 4)), z = *reinterpret_cast<const float4 *>(chunk(e / 4 + 4));
                        x[0] = y.x, x[1] = y.y, x[2] = y.z, x[3] = y.w, x[4] = z.x, x[5] = z.y, x[6] = z.z, x[7] = z.w;
                    } else {
                        const uint2 y = *reinterpret_cast<const uint2 *>(chunk(e / 8) + 2 * (e & 7)), z = *reinterpret_cast<const uint2 *>(chunk(e / 8 + 2) + 2 * (e & 7));
                        const uint32_t two[4] = {y.x, y.y, z.x, z.y};
#pragma unroll
                        for (int k = 0; k < 4; ++k) x[2 * k] = unpack_half2(two[k]).x, x[2 * k + 1] = unpack_half2(two[k]).y;
                    }
                    uint32_t high[4], low[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {  // elements 0 2 | 1 3 | 16 18 | 17 19
                        const int k0 = (k & 2) * 2 + (k & 1);
                        const float y = x[k0] * up, z = x[k0 + 2] * up;
                        high[k] = pack_half2(y, z);
                        const float2 f = unpack_half2(high[k]);
                        low[k] = pack_half2(y - f.x, z - f.y);
                    }
                    tc_st4(tmem + (static_cast<uint32_t>(32 * (w & 3)) << 16) + kTmemQ + 32 * h + 4 * i, high);
                    if (TERMS == 2)
                        *reinterpret_cast<uint4 *>(smem + Sh::kOffLow + h * Sh::kPart + r * 128 + ((i ^ (r & 7)) << 4)) = make_uint4(low[0], low[1], low[2], low[3]);
                }
                tc_wait_st();
                tc_fence_before();
                if (TERMS == 2) fence_proxy_async_smem();
            }
            // slices take the places when every warp has read its rows
            __syncwarp();
            if (lane == 0) mbar_arrive(q_staged);
            ok = wait(q_staged, 1);
            for (int j = 0; ok && j < st.n; ++j, ++n) {
#pragma unroll 1
                for (int h = 0; ok && h < Sh::kSlices; ++h) expand(n * Sh::kSlices + h, h);
            }
        }
        if (!ok) failed(kErrConsumerWait);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tc_dealloc(tmem, kTmemCols);
}

__device__ __forceinline__ void store2(float *p, float a, float b) { *reinterpret_cast<float2 *>(p) = make_float2(a, b); }
__device__ __forceinline__ void store2(__half *p, float a, float b) { *reinterpret_cast<__half2 *>(p) = __floats2half2_rn(a, b); }

// Joins each row's results: of its stretches of the prefix, and of its own tokens. Block (s, i, h): query i of sequence
// s, eight heads (of 64: sixteen); D / 4 lanes a head, each four places of a stretch's row: two channels and the two 32 after them.
// Where that would be more than kJoinBlocks blocks (offsets may name 2^24 sequences, most of them without a row) a block takes
// several queries, and sequences in sets of 32, whose offsets a warp's lanes look at.
constexpr int kJoinThreads = 256, kJoinBlocks = 1 << 20;

template <int D, class T> __global__ void __launch_bounds__(kJoinThreads) shared_join_kernel(const SharedParams p, const int parts) {
    constexpr int kLanes = D / 4, kAhead = 10;  // (stretches under way: an item has up to 19; 4 took half a microsecond more)
    pdl_allow_dependents();
    pdl_wait_prior_grids();
    const KvAttendParams &a = p.own;
    const int h = blockIdx.z * (kJoinThreads / kLanes) + threadIdx.x / kLanes;
    const Units units(p, parts);
    const int l = threadIdx.x % kLanes, channel = 64 * (l / 16) + 2 * (l / 2 % 8) + 16 * (l & 1);
    const int kv = h / a.group;
    auto join = [&](int q0, int i) {  // query i of the sequence whose rows begin at q0
        const int tok = q0 + i, row = tok * a.group + h - kv * a.group;
        const int64_t rest = static_cast<int64_t>(tok) * a.n_heads + h;
        const float2 own = __ldcg(reinterpret_cast<const float2 *>(a.rest_stats) + rest);
        float top = -INFINITY, den = 0.0f;
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        auto add = [&](float2 s, float4 v) {
            const float next = fmaxf(top, s.x), ref = next == -INFINITY ? 0.0f : next;
            const float keep = exp2_approx(top - ref), f = exp2_approx(s.x - ref);
            top = next;
            den = fmaf(den, keep, s.y * f);
            acc.x = fmaf(acc.x, keep, v.x * f), acc.y = fmaf(acc.y, keep, v.y * f);
            acc.z = fmaf(acc.z, keep, v.z * f), acc.w = fmaf(acc.w, keep, v.w * f);
        };
        auto of_own = [&](const float *row) {
            const float2 x = __ldcg(reinterpret_cast<const float2 *>(row + channel)), y = __ldcg(reinterpret_cast<const float2 *>(row + channel + 32));
            return make_float4(x.x, y.x, x.y, y.y);
        };
        if (own.y < 0.0f) {  // parts of thread blocks
            const int c = __float_as_int(own.x), n = static_cast<int>(-own.y), in = (i * a.group + h - kv * a.group) % p.parts.rows;
            const float *const first = a.partial + p.parts.first + (2 * static_cast<int64_t>(c) + 1) * p.parts.pitch;
            for (int k = 0; k < n; ++k) {
                const float *part = first + (k == 0 ? 0 : 2 * k - 1) * p.parts.pitch;
                add(__ldcg(reinterpret_cast<const float2 *>(part + p.parts.rows * D) + in), of_own(part + in * D));
            }
        } else {
            add(own, of_own(a.rest + rest * D));
        }
        if (units.tiles > 0) {
            const int item = kv * p.row_tiles + row / kRows;
            const int64_t u = static_cast<int64_t>(item) * units.tiles;
            const int c0 = units.per_item > 0 ? item * units.per_item : static_cast<int>(u / units.share);
            const int n = units.per_item > 0 ? (units.tiles + static_cast<int>(units.share) - 1) / static_cast<int>(units.share)
                                             : static_cast<int>((u + units.tiles - 1) / units.share) - c0 + 1;
            const float *const first = p.stretches + (c0 + static_cast<int64_t>(item)) * stretch_floats(D);
            for (int c = 0; c < n; c += kAhead) {
                float2 s[kAhead];
                float4 v[kAhead];
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    const float *part = first + min(c + k, n - 1) * stretch_floats(D);
                    s[k] = __ldcg(reinterpret_cast<const float2 *>(part + kRows * D) + row % kRows);
                    v[k] = __ldcg(reinterpret_cast<const float4 *>(part + row % kRows * D) + l);
                }
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    if (c + k >= n) break;
                    add(s[k], v[k]);
                }
            }
        }
        const float inv = den == 0.0f ? 0.0f : 1.0f / den;  // no token seen: zeros
        T *out = static_cast<T *>(a.out) + rest * D + channel;
        store2(out, acc.x * inv, acc.z * inv);
        store2(out + 32, acc.y * inv, acc.w * inv);
    };
    const int set = a.n_seq > static_cast<int>(gridDim.x) ? 32 : 1;
    for (int64_t s0 = static_cast<int64_t>(blockIdx.x) * set; s0 < a.n_seq; s0 += static_cast<int64_t>(gridDim.x) * set) {
        const int s = static_cast<int>(s0) + static_cast<int>(threadIdx.x & (set - 1));
        int q0 = s, m = s < a.n_seq ? 1 : 0;
        if (a.q_offsets != nullptr && m > 0) {
            q0 = __ldg(a.q_offsets + s);
            const int q1 = __ldg(a.q_offsets + s + 1);
            m = q0 < 0 || q1 < q0 || q1 > a.n_tok || q1 - q0 > a.max_q_len ? 0 : q1 - q0;
        }
        for (uint32_t some = __ballot_sync(0xffffffffu, m > 0) & (set == 1 ? 1u : ~0u); some != 0; some &= some - 1) {
            const int first = __shfl_sync(0xffffffffu, q0, __ffs(some) - 1), many = __shfl_sync(0xffffffffu, m, __ffs(some) - 1);
            for (int i = blockIdx.y; i < many && h < a.n_heads; i += gridDim.y) join(first, i);
        }
    }
}

int64_t row_tiles(int64_t n_tok, int group) { return (n_tok * group + kRows - 1) / kRows; }
size_t align(size_t n) { return (n + 255) / 256 * 256; }

template <int D, class T> cudaError_t launch(SharedParams &p, int sms, int device, cudaStream_t s) {
    using Sh = Shape<D, sizeof(T) == 4 ? 2 : 1>;
    static std::atomic<uint64_t> done{0};
    const uint64_t bit = 1ull << (device & 63);
    if (!(done.load(std::memory_order_acquire) & bit)) {
        cudaError_t e = cudaFuncSetAttribute(prefix_kernel<D, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem);
        cudaFuncAttributes attr;
        if (e == cudaSuccess) e = cudaFuncGetAttributes(&attr, prefix_kernel<D, T>);
        if (e != cudaSuccess) return e;
        if (attr.numRegs != kLaunchRegs) {  // the roles would wait for registers that the block does not have
            g_launch_step = "prefix_kernel's registers";
            return cudaErrorInvalidValue;
        }
        done.fetch_or(bit, std::memory_order_acq_rel);
    }
    const int parts = sms < kMaxParts ? sms : kMaxParts;
    cudaError_t e = launch_pdl(prefix_kernel<D, T>, parts, kThreads, Sh::kSmem, s, p);
    if (e == cudaSuccess) e = launch_kv_attend(p.own, D, sizeof(T) == 4 ? QG_F32 : QG_F16, sms, device, s);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    const int per = kJoinThreads / (D / 4), of_heads = (p.own.n_heads + per - 1) / per;  // (8192 at most)
    const int seqs = std::min(p.own.n_seq, kJoinBlocks / of_heads), queries = std::min({p.own.max_q_len, 64, std::max(1, kJoinBlocks / of_heads / seqs)});
    cfg.gridDim = dim3(static_cast<unsigned>(seqs), static_cast<unsigned>(queries), static_cast<unsigned>(of_heads));
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, shared_join_kernel<D, T>, static_cast<SharedParams>(p), parts);
}

}  // namespace

// The workspace: kv_attend's own, the rows' results of their own tokens, the stretches, which are written 32 bytes at a time
// and so begin at the next such boundary (the interface asks for 16).
constexpr size_t kStretchAlign = 32;
size_t shared_attend_workspace(int head_dim, int n_kv_heads, int group, int64_t n_tok, int max_q_len) {
    const size_t rows = static_cast<size_t>(n_tok) * group * n_kv_heads;
    return align(kv_attend_workspace(head_dim, group * max_q_len)) + align(rows * head_dim * 4) + align(rows * 8) +
           static_cast<size_t>(kMaxParts + n_kv_heads * row_tiles(n_tok, group)) * stretch_floats(head_dim) * 4 + kStretchAlign - 16;
}

cudaError_t launch_shared_attend(SharedParams p, int head_dim, int type, int sms, int device, cudaStream_t s) {
    KvAttendParams &a = p.own;
    uint8_t *at = reinterpret_cast<uint8_t *>(a.partial);
    const size_t rows = static_cast<size_t>(a.n_tok) * a.n_heads;
    at += align(kv_attend_workspace(head_dim, a.group * a.max_q_len));
    a.rest = reinterpret_cast<float *>(at);
    at += align(rows * head_dim * 4);
    a.rest_stats = reinterpret_cast<float *>(at);
    at += align(rows * 8);
    at += (0 - reinterpret_cast<uintptr_t>(at)) % kStretchAlign;
    p.stretches = reinterpret_cast<float *>(at);
    p.row_tiles = static_cast<int>(row_tiles(a.n_tok, a.group));
    p.parts = kv_attend_parts(head_dim, static_cast<int64_t>(a.group) * a.max_q_len);
    if (head_dim == 64) return type == QG_F32 ? launch<64, float>(p, sms, device, s) : launch<64, __half>(p, sms, device, s);
    return type == QG_F32 ? launch<128, float>(p, sms, device, s) : launch<128, __half>(p, sms, device, s);
}

}  // namespace qg
