// shared_attend.cu - attention of new tokens of sequences that share a prefix,
// over the 4-bit paged cache (include/qattn.h, qkv_attend_shared).
//
// All query rows of a key/value head see the whole prefix, so it is taken once
// for all of them: an item is one key/value head and 128 of its rows (token-major
// over the call's tokens and the head's group), its units tiles of 128 prefix
// tokens. The items' units form one list that the thread blocks share out in
// equal contiguous parts; each stretch of an item in a part leaves its rows'
// values, reference and sum in the workspace. Each sequence's own tokens go
// through kv_attend's kernels, which leave theirs there, too, and a last kernel
// joins a row's results in a fixed order.
#include <atomic>
#include <cfloat>

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
constexpr float kHigh = 14.0f, kLow = 7.0f;  // log2 of the largest weight, and of the largest when the reference is set

template <int D, int TERMS> struct Shape {
    using G = KvGroup<D>;
    static constexpr int kPart = kTokens * D * 2;              // one f16 part of a key, value or query tile
    static constexpr int kRawCodes = kTokens * D / 2;          // codes of a unit's keys (or values)
    static constexpr int kRaw = kRawCodes + kTokens * G::kScaleRow;
    // Operands, in the order K(0), K(1), V(0), K(2), V(1) ..., each a high and a low part of 128-byte rows of 64
    // channels: three places let them be made ready a piece ahead of the products (f32 queries leave room for two of
    // heads of 128). The queries' high parts pass through the last place on their way to tensor memory, f32's low parts
    // have one of their own.
    static constexpr bool kTwo = TERMS == 2 && D == 128;
    static constexpr int kPlaces = kTwo ? 2 : 3, kPlace = 2 * kPart;
    static constexpr int kOffLow = kPlaces * kPlace;
    static constexpr int kOffRaw = kOffLow + (TERMS == 2 ? kPart : 0);
    static constexpr int kSlots = D == 128 && !kTwo ? 3 : 6;   // raw pieces
    static constexpr int kOffBars = kOffRaw + kSlots * kRaw;
    static constexpr int kOffKeep = kOffBars + 512;            // [tile % 4][row]: what the sums before a tile are multiplied by
    static constexpr int kOffFactor = kOffKeep + 4 * kRows * 4;  // [stretch % 4][row]: a row's scores as powers of 2
    static constexpr int kSmem = kOffFactor + 4 * kRows * 4 + 1024;  // (alignment)
    static_assert(kSmem <= kSmemLimit, "shared memory");
};

// The prefix's length, checked, and the list of units.
struct Units {
    int len, tiles;      // tokens, units of an item
    int64_t all, share;  // of all items, of a part
    __device__ __forceinline__ Units(const SharedParams &p, int parts) {
        len = __ldg(p.prefix_len);
        const int64_t room = p.prefix_pages * static_cast<int64_t>(p.own.c.page_size);
        if (len < 0 || len > room) {
            record_error(p.own.err, kErrBadIndex);
            len = len < 0 ? 0 : static_cast<int>(room);
        }
        tiles = (len + kTokens - 1) / kTokens;
        all = static_cast<int64_t>(p.own.c.n_heads) * p.row_tiles * tiles;
        share = (all + parts - 1) / parts;
        if (share < 1) share = 1;
    }
};
// A stretch's place: parts and items both rise along the list, one of them at least from stretch to stretch.
__host__ __device__ constexpr int64_t stretch_floats(int d) { return static_cast<int64_t>(kRows) * (d + 2); }

// A stretch's rows hold the channels in the order in which the value codes lie in the cache: place 8 (8 h + u) + 2 j + b
// holds channel 64 h + 32 b + 2 u + {0, 1, 16, 17}[j].

// Walks a part's stretches, alike in every role.
struct Stretch {
    int64_t u, past;  // the next unit, the part's end
    int item, tile, n, index = -1;
    __device__ __forceinline__ bool next(const Units &units) {
        if (u >= past) return false;
        item = static_cast<int>(u / units.tiles);
        tile = static_cast<int>(u - static_cast<int64_t>(item) * units.tiles);
        n = static_cast<int>(min(past - u, static_cast<int64_t>(units.tiles - tile)));
        u += n;
        ++index;
        return true;
    }
};

// The pieces of a part, alike in every role: K(0), K(1), V(0), K(2), V(1), ..., V(n - 2), V(n - 1).
struct Pieces {
    __device__ static __forceinline__ int of_k(int j) { return j == 0 ? 0 : 2 * j - 1; }
    __device__ static __forceinline__ int of_v(int j, int n) { return j == n - 1 ? 2 * n - 1 : 2 * j + 2; }
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

// Two codes' values in two f16 parts, which hold them exactly (four bits times eleven) above f16's end.
__device__ __forceinline__ void two_parts(__half2 code, __half2 scale, uint32_t &high, uint32_t &low) {
    const __half2 h = __hmul2(code, scale);
    high = bits(h);
    low = bits(__hfma2(code, scale, __hneg2(h)));
}

// One word of a row: eight values into 16 bytes of each part.
__device__ __forceinline__ void expand_word(uint32_t w, __half2 scale, uint8_t *high, uint8_t *low) {
    uint4 h, l;
    two_parts(low_codes(w), scale, h.x, l.x);
    two_parts(low_codes(w >> 8), scale, h.y, l.y);
    two_parts(high_codes(w), scale, h.z, l.z);
    two_parts(high_codes(w >> 8), scale, h.w, l.w);
    *reinterpret_cast<uint4 *>(high) = h;
    *reinterpret_cast<uint4 *>(low) = l;
}

// Makes a unit's raw scales (keys' or values') ready: 0 for tokens that do not count (rows past `rows`, groups in no
// page), infinities as NaN, and all times the power of two that takes the largest to 2^8 .. 2^9 (f16 exponent fields),
// whose exponent is returned. The unit's values are then below 2^13 and exact down to 2^-33 of that. One warp: a lane
// has two words of four tokens in two places, which its neighbours' follow.
template <int D> __device__ __forceinline__ int prepare_scales(uint8_t *scales, int rows, uint32_t groups) {
    constexpr int kChunks = kTokens * (D / 16) / 512, kPer = 256 / D;  // 16-byte chunks of a lane, tokens of one
    const int lane = threadIdx.x & 31;
    uint4 *const at = reinterpret_cast<uint4 *>(scales) + lane;
    uint32_t x[kChunks][4], m = 0;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        const uint4 v = at[32 * i];
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
        at[32 * i] = make_uint4(y[0], y[1], y[2], y[3]);
    }
    return e;
}

__device__ __forceinline__ void load8(const float *p, float (&x)[8]) {  // elements 0 .. 3 and 16 .. 19
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p + 16));
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void load8(const __half *p, float (&x)[8]) {
    const uint2 a = __ldg(reinterpret_cast<const uint2 *>(p)), b = __ldg(reinterpret_cast<const uint2 *>(p + 16));
    const uint32_t w[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = unpack_half2(w[i]).x, x[2 * i + 1] = unpack_half2(w[i]).y;
}

template <int D, class T>
__global__ void __launch_bounds__(kThreads, 1) prefix_kernel(const SharedParams p) {
    constexpr int TERMS = sizeof(T) == 4 ? 2 : 1, NB = D / 32;
    using Sh = Shape<D, TERMS>;
    using G = KvGroup<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *const smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);  // (the swizzle's atoms are 1024 bytes)
    const uint32_t base = smem_addr(smem), bars = base + Sh::kOffBars;
    const uint32_t raw_full = bars, raw_empty = raw_full + 8 * Sh::kSlots, k_done = raw_empty + 8 * Sh::kSlots;
    const uint32_t s_full = k_done + 8, p_ready = s_full + 16, o_full = p_ready + 16, o_free = o_full + 8;
    const uint32_t mfinal = o_free + 8, q_staged = mfinal + 8, place_ready = q_staged + 8, place_free = place_ready + 24, scaled = place_free + 24;  // up to 33 barriers: 264 bytes
    uint8_t *const words = smem + Sh::kOffBars + 272;
    uint32_t *const tmem_slot = reinterpret_cast<uint32_t *>(words);
    volatile int *const abort_flag = reinterpret_cast<volatile int *>(words + 4);
    volatile int *const groups = reinterpret_cast<volatile int *>(words + 16);     // [tile % 16]: its groups that lie in a page
    // [tile % 8]: the scales' exponents (the warp that finds them is three tiles ahead of those that expand at most, and
    // these two ahead of the softmax)
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
            mbar_init(scaled + 8 * i, 1);
        }
        mbar_init(k_done, 1);
        for (int x = 0; x < 2; ++x) {
            mbar_init(s_full + 8 * x, 1);
            mbar_init(p_ready + 8 * x, 4);
        }
        mbar_init(o_full, 1);
        mbar_init(o_free, 4);
        mbar_init(mfinal, 1);
        mbar_init(q_staged, kExpanders);
        for (int i = 0; i < Sh::kPlaces; ++i) {
            mbar_init(place_ready + 8 * i, kExpanders);
            mbar_init(place_free + 8 * i, 1);
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
    Stretch st;
    st.u = blockIdx.x * units.share;
    st.past = min(st.u + units.share, units.all);
    // A wait of a whole warp that gives up sets the abort flag, with which the others give up soon.
    auto failed = [&](int32_t code) {
        if (lane == 0) record_error(a.err, code);
        *abort_flag = 1;
        __syncwarp();
    };
    auto wait = [&](uint32_t bar, uint32_t parity) {
        return static_cast<bool>(__all_sync(0xffffffffu, sleep_wait<20>(bar, parity & 1u, abort_flag)));
    };

    if (warp < 4) {
        fewer_registers<kIssueRegs>();
        if (warp == 0) {
            // ---------------- copies: of each unit the keys' codes and scales, then (a unit behind) the values'
            int piece = 0, last = 0;  // pieces so far
            bool ok = true;
            // this lane's group of a unit, as a byte offset in the cache; -1: none
            auto source = [&](int item, int tile) -> int64_t {
                const int t = tile * kTokens + 16 * (lane & 7);
                if (t >= units.len) return -1;
                const int page = __ldg(p.prefix_table + t / a.c.page_size);
                if (page < 0 || page >= a.c.n_pages) {
                    record_error(a.err, kErrBadIndex);
                    return -1;
                }
                return ((static_cast<int64_t>(page) * a.c.n_heads + item / p.row_tiles) * a.c.page_groups + t % a.c.page_size / 16) * G::kBytes;
            };
            auto copy = [&](int64_t src, bool values) {
                const int slot = piece % Sh::kSlots;
                if (piece >= Sh::kSlots) ok = wait(raw_empty + 8 * slot, piece / Sh::kSlots - 1);
                if (!ok) return;
                const uint32_t valid = __ballot_sync(0xffffffffu, src >= 0) & 255u;
                const uint32_t dst = base + Sh::kOffRaw + slot * Sh::kRaw, bar = raw_full + 8 * slot;
                if (lane == 0) {
                    if (!values) groups[last % 16] = static_cast<int>(valid);
                    mbar_arrive_expect_tx(bar, __popc(valid) * (18 * D / 2));
                }
                __syncwarp();
                if (src >= 0 && lane < 8)
                    bulk_copy_g2s_plain(dst + lane * (8 * D), a.c.data + src + (values ? G::kV : 0), 8 * D, bar);
                else if (src >= 0 && lane < 16)
                    bulk_copy_g2s_plain(dst + Sh::kRawCodes + (lane & 7) * D, a.c.data + src + (values ? G::kVS : G::kKS), D, bar);
                ++piece;
            };
            int64_t before = -1;  // the unit before's
            bool any = false;
            while (ok && st.next(units)) {
                for (int j = 0; ok && j < st.n; ++j, ++last) {
                    const int64_t src = source(st.item, st.tile + j);
                    copy(src, false);
                    if (ok && any) copy(before, true);
                    before = src, any = true;
                }
            }
            if (ok && any) copy(before, true);
            if (!ok) failed(kErrProducerWait);
            // leave no copy in flight into this block's shared memory
            bool landed = true;
            for (int k = piece > Sh::kSlots ? piece - Sh::kSlots : 0; k < piece; ++k)
                landed = mbar_wait_bounded(raw_full + 8 * (k % Sh::kSlots), (k / Sh::kSlots) & 1) && landed;
            if (!landed) record_error(a.err, kErrDrainWait);
            __syncwarp();
        } else if (warp == 1) {
            // ---------------- products (the whole warp, one lane issues)
            const uint32_t issue = lane == 0;
            constexpr uint32_t kIdS = tc_idesc_f16(128, kTokens), kIdO = tc_idesc_f16(128, D) | kIdescNMajorB;
            constexpr uint32_t kPart = Sh::kPart / 16;
            const uint32_t q_low = desc_lo(base + Sh::kOffLow, 1);
            const int units_in_all = static_cast<int>(st.past - st.u);
            auto tight = [&](uint32_t bar, uint32_t parity) { return static_cast<bool>(__all_sync(0xffffffffu, tc_wait(bar, parity & 1u, abort_flag))); };
            bool ok = true;
            int n = 0;  // units so far
            auto product_o = [&](int j) {
                const int piece = Pieces::of_v(j, units_in_all), place = piece % Sh::kPlaces;
                const uint32_t v = desc_lo(base + place * Sh::kPlace, 128 * 128 / 16);
                ok = tight(p_ready + 8 * (j & 1), j >> 1) && tight(place_ready + 8 * place, piece / Sh::kPlaces) && (j == 0 || tight(o_free, j - 1));
                if (!ok) return;
                tc_fence_after();
                const uint32_t w = tmem + 128 * (j & 1), w_low = tmem + kTmemLow;
                // small terms first: what the tensor cores cut off at each sum is then of the small ones
                // (one piece of code for them: what runs once a unit comes from instruction memory each time)
#pragma unroll 1
                for (int i = 2 - TERMS; i < 3; ++i)
                    mma_pv(issue, tmem + kTmemO, i == 0 ? w_low : w, i == 1 ? v + kPart : v, kIdO, i > 2 - TERMS, kDescHi);
                commit(issue, place_free + 8 * place);
                commit(issue, o_full);
            };
            while (ok && st.next(units)) {
                for (int j = 0; ok && j < st.n; ++j, ++n) {
                    const int piece = Pieces::of_k(n), place = piece % Sh::kPlaces;
                    ok = tight(place_ready + 8 * place, piece / Sh::kPlaces);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t s = tmem + 128 * (n & 1), k = desc_lo(base + place * Sh::kPlace, 1);
                    if (TERMS == 2) mma_s<D>(issue, s, q_low, k, kIdS, kDescHi, 0);
#pragma unroll 1
                    for (int i = 0; i < 2; ++i)
                        mma_s_tm<D>(issue, s, tmem + kTmemQ, i == 0 ? k + kPart : k, kIdS, kDescHi, TERMS == 2 || i > 0);
                    commit(issue, s_full + 8 * (n & 1));
                    commit(issue, place_free + 8 * place);
                    commit(issue, k_done);
                    if (n > 0) product_o(n - 1);
                }
            }
            if (ok && n > 0) product_o(n - 1);
            if (!ok) failed(kErrConsumerWait);
            commit(issue, mfinal);  // every product complete before tensor memory is freed, after a wait that gave up, too
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(mfinal, 0)) && issue) record_error(a.err, kErrDrainWait);
            __syncwarp();
        } else if (warp == 2) {
            // ---------------- scales, in place
            bool ok = true;
            int n = 0, piece = 0, before = 0;
            auto prepare = [&](int j, int tile, bool values) {
                const int slot = piece % Sh::kSlots;
                ok = wait(raw_full + 8 * slot, piece / Sh::kSlots);
                if (!ok) return;
                const int e = prepare_scales<D>(smem + Sh::kOffRaw + slot * Sh::kRaw + Sh::kRawCodes,
                                                min(kTokens, units.len - tile * kTokens), static_cast<uint32_t>(groups[j % 16]));
                fence_proxy_async_smem();  // (the next copy to this place comes after these writes)
                __syncwarp();
                if (lane == 0) {
                    (values ? v_exp : k_exp)[j & 7] = e;
                    mbar_arrive(scaled + 8 * slot);
                }
                ++piece;
            };
            while (ok && st.next(units)) {
                for (int j = 0; ok && j < st.n; ++j, ++n) {
                    prepare(n, st.tile + j, false);
                    if (ok && n > 0) prepare(n - 1, before, true);
                    before = st.tile + j;
                }
            }
            if (ok && n > 0) prepare(n - 1, before, true);
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
            float ref = -INFINITY;
            float2 sum = make_float2(0.0f, 0.0f);
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
                    sum.x *= down, sum.y *= down;
                }
                keep[(n & 3) * kRows + row] = down;
                const float r = ref == -INFINITY ? 0.0f : ref;  // (no token seen yet: weights of 0)
                const float2 c2 = make_float2(c, c), r2 = make_float2(-r, -r);
                if (TERMS == 2 && n > 0) ok = wait(o_full, n - 1);  // the low parts' place is one
                if (!ok) break;
#pragma unroll 1
                for (int i = 0; i < 4; ++i) {
                    uint32_t v[32], w[16], w_low[16];
                    load(i, v);
#pragma unroll
                    for (int q = 0; q < 16; ++q) {
                        float2 e = ffma2(make_float2(__uint_as_float(v[2 * q]), __uint_as_float(v[2 * q + 1])), c2, r2);
                        e.x = exp2_approx(e.x), e.y = exp2_approx(e.y);
                        sum = fadd2(sum, e);
                        w[q] = pack_half2(e.x, e.y);
                        if (TERMS == 2) {
                            const float2 h = unpack_half2(w[q]);
                            w_low[q] = pack_half2(e.x - h.x, e.y - h.y);
                        }
                    }
                    tc_st16(s_t + 16 * i, w);
                    if (TERMS == 2) tc_st16(low_t + 16 * i, w_low);
                }
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_ready + 8 * (n & 1));
            }
            if (ok)
                reinterpret_cast<float2 *>(p.stretches + (blockIdx.x + static_cast<int64_t>(st.item)) * stretch_floats(D) + kRows * D)[row] =
                    make_float2(ref, sum.x + sum.y);
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
                ok = wait(o_full, n);
                if (!ok) break;
                tc_fence_after();
                const float f = keep[(n & 3) * kRows + row], u = __uint_as_float(static_cast<uint32_t>(127 - v_exp[n & 7]) << 23);
                const float2 u2 = make_float2(u, u);
                if (__any_sync(0xffffffffu, f != 1.0f))
#pragma unroll
                    for (int i = 0; i < D / 2; ++i) o[i].x *= f, o[i].y *= f;
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
        const int w = warp - 12;
        bool ok = true;
        int n = 0, piece = 0;
        // a piece's operands, once `free` is: 128-byte rows of 64 channels, 16-byte chunks swizzled by the row
        auto expand = [&](bool values) {
            const int slot = piece % Sh::kSlots;
            ok = wait(scaled + 8 * slot, piece / Sh::kSlots) && wait(raw_full + 8 * slot, piece / Sh::kSlots);
            // (a barrier a place: its last piece's products are complete)
            if (ok && piece >= Sh::kPlaces) ok = wait(place_free + 8 * (piece % Sh::kPlaces), piece / Sh::kPlaces - 1);
            if (!ok) return;
            const uint8_t *const raw = smem + Sh::kOffRaw + slot * Sh::kRaw;
            // Rows of a warp: so that eight lanes that store together have eight different chunk places, and the same for
            // both of its turns, 64 rows on (8 groups' rows 4 by 4 KB: one address and constants).
            const int part = lane & 3, x = lane >> 2, row = 8 * w + (values ? x : (x & 1) * 4 + (x >> 1)), vr = kv_value_row(row & 15);
            const uint8_t *codes = raw + (values ? ((row & ~15) + vr) * G::kRow + (part ^ (vr & 2)) * (4 * NB) : row * G::kRow + part * (4 * NB));
            const uint8_t *scales = raw + Sh::kRawCodes + row * G::kScaleRow;
            uint8_t *const to = smem + piece % Sh::kPlaces * Sh::kPlace + row * 128;
            // Keys: block b's word goes to chunk 4 (b % 2) + part of half b / 2; values: units 2 part and 2 part + 1 of block
            // pair h to half h. One piece of code for both, see the softmax's loops.
            uint8_t *const first = to + (((values ? 2 * part : part) ^ (row & 7)) << 4);
            uint8_t *const second = to + (((values ? 2 * part + 1 : part + 4) ^ (row & 7)) << 4);
            uint8_t *const inner[2] = {values ? first + 128 * 128 : second, values ? second : first + 128 * 128};  // (of four words the second and third)
            const uint32_t even = values ? 0x3210 : 0x1010, odd = values ? 0x3210 : 0x3232;
#pragma unroll 1
            for (int it = 0; it < 2; ++it) {
                uint32_t c[NB], d[NB / 2];
                ld_words<NB>(codes + it * (64 * G::kRow), c);
                ld_halves<NB>(scales + it * (64 * G::kScaleRow), d);
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    const uint32_t pair = NB == 2 || i == 0 ? d[0] : i == 3 ? d[NB / 2 - 1] : (values == (i == 1)) ? d[NB / 2 - 1] : d[0];
                    const uint32_t s2 = __byte_perm(pair, 0, i & 1 ? odd : even);
                    uint8_t *t = (i == 0 ? first : NB == 2 ? second : i == 3 ? second + 128 * 128 : inner[i - 1]) + it * (64 * 128);
                    expand_word(c[i], *reinterpret_cast<const __half2 *>(&s2), t, t + Sh::kPart);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(raw_empty + 8 * slot);
                mbar_arrive(place_ready + 8 * (piece % Sh::kPlaces));
            }
            ++piece;
        };
        while (ok && st.next(units)) {
            // ---- the stretch's queries, in the keys' order of channels, once the last one's products are complete
            // (the low parts' place is read by those products, tensor memory too; the high ones pass through the place of
            // the piece that comes next, K(n))
            const int place = piece % Sh::kPlaces;
            if (n > 0) ok = wait(k_done, n - 1) && (piece < Sh::kPlaces || wait(place_free + 8 * place, piece / Sh::kPlaces - 1));
            if (!ok) break;
            uint8_t *const staged = smem + place * Sh::kPlace;
            const int head = st.item / p.row_tiles, row0 = st.item % p.row_tiles * kRows;
            constexpr int kLanes = D / 8, kStep = 8 * 32 / kLanes;  // lanes of a row, rows of the eight warps
            const int chunk = lane % kLanes, b = chunk >> 2, t = chunk & 3;
#pragma unroll 2
            for (int r0 = 0; r0 < kRows; r0 += kStep) {
                const int r = r0 + w * (32 / kLanes) + lane / kLanes, row = row0 + r, tok = row / a.group;
                float x[8] = {};
                if (tok < a.n_tok)
                    load8(static_cast<const T *>(a.q) + tok * a.q_stride + (static_cast<int64_t>(head) * a.group + row - tok * a.group) * D + 32 * b + 4 * t, x);
                float up = a.scale < 0.0f ? -1.0f : 1.0f, back = fabsf(a.scale) * 1.4426950408889634f;
                if (TERMS == 2) {  // the largest magnitude to 2^10 .. 2^11
                    float big = 0.0f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) big = fmaxf(big, fabsf(x[i]));
#pragma unroll
                    for (int m = 1; m < kLanes; m <<= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, m));
                    int e = static_cast<int>(__float_as_uint(big) >> 23) - 127;
                    if (e == 128) e = 0;         // infinities
                    if (e < -117) e = -117;      // (2^(10 - e) is an f32)
                    up *= __uint_as_float(static_cast<uint32_t>(137 - e) << 23);
                    back *= __uint_as_float(static_cast<uint32_t>(127 + e) << 23) * 0x1p-10f;
                }
                if (chunk == 0) factor[(st.index & 3) * kRows + r] = fmaxf(back, 1e-37f);  // never 0, which times -inf would be NaN
                uint32_t h[4], l[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {  // elements 0 2 | 1 3 | 16 18 | 17 19
                    const int i0 = (i & 2) * 2 + (i & 1);
                    const float y = x[i0] * up, z = x[i0 + 2] * up;
                    h[i] = pack_half2(y, z);
                    const float2 f = unpack_half2(h[i]);
                    l[i] = pack_half2(y - f.x, z - f.y);
                }
                const int to = (chunk >> 3) * (128 * 128) + r * 128 + (((chunk & 7) ^ (r & 7)) << 4);
                *reinterpret_cast<uint4 *>(staged + to) = make_uint4(h[0], h[1], h[2], h[3]);
                if (TERMS == 2) *reinterpret_cast<uint4 *>(smem + Sh::kOffLow + to) = make_uint4(l[0], l[1], l[2], l[3]);
            }
            {  // to tensor memory: a row's 64 channels a thread
                __syncwarp();
                if (lane == 0) mbar_arrive(q_staged);
                ok = wait(q_staged, 0);
                if (!ok) break;
                const int r = 32 * (w & 3) + lane, h = w >> 2;
                if (h < D / 64) {
                    uint32_t v[32];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint4 x = *reinterpret_cast<const uint4 *>(staged + h * (128 * 128) + r * 128 + ((i ^ (r & 7)) << 4));
                        v[4 * i] = x.x, v[4 * i + 1] = x.y, v[4 * i + 2] = x.z, v[4 * i + 3] = x.w;
                    }
                    tc_st32(tmem + (static_cast<uint32_t>(32 * (w & 3)) << 16) + kTmemQ + 32 * h, v);
                    tc_wait_st();
                    tc_fence_before();
                }
                // K(n) takes the place when every warp has read its rows
                __syncwarp();
                if (lane == 0) mbar_arrive(q_staged);
                ok = wait(q_staged, 1);
            }
            for (int j = 0; ok && j < st.n; ++j, ++n) {
                for (int values = 0; ok && values < (n > 0 ? 2 : 1); ++values) expand(values != 0);
            }
        }
        if (ok && n > 0) expand(true);
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
constexpr int kJoinThreads = 256;

template <int D, class T> __global__ void __launch_bounds__(kJoinThreads) shared_join_kernel(const SharedParams p, const int parts) {
    constexpr int kLanes = D / 4, kAhead = 4;
    pdl_allow_dependents();
    pdl_wait_prior_grids();
    const KvAttendParams &a = p.own;
    int q0 = blockIdx.x, m = 1;
    if (a.q_offsets != nullptr) {
        q0 = __ldg(a.q_offsets + blockIdx.x);
        const int q1 = __ldg(a.q_offsets + blockIdx.x + 1);
        m = q0 < 0 || q1 < q0 || q1 > a.n_tok || q1 - q0 > a.max_q_len ? 0 : q1 - q0;
    }
    const int h = blockIdx.z * (kJoinThreads / kLanes) + threadIdx.x / kLanes;
    if (h >= a.n_heads) return;
    const Units units(p, parts);
    const int l = threadIdx.x % kLanes, channel = 64 * (l / 16) + 2 * (l / 2 % 8) + 16 * (l & 1);
    const int kv = h / a.group;
    for (int i = blockIdx.y; i < m; i += gridDim.y) {
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
            const int c0 = static_cast<int>(u / units.share), n = static_cast<int>((u + units.tiles - 1) / units.share) - c0 + 1;
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
    const int per = kJoinThreads / (D / 4);
    cfg.gridDim = dim3(static_cast<unsigned>(p.own.n_seq), static_cast<unsigned>(p.own.max_q_len < 64 ? p.own.max_q_len : 64),
                       static_cast<unsigned>((p.own.n_heads + per - 1) / per));
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

// The workspace: kv_attend's own, the rows' results of their own tokens, the stretches.
size_t shared_attend_workspace(int head_dim, int n_kv_heads, int group, int64_t n_tok, int max_q_len) {
    const size_t rows = static_cast<size_t>(n_tok) * group * n_kv_heads;
    return align(kv_attend_workspace(head_dim, group * max_q_len)) + align(rows * head_dim * 4) + align(rows * 8) +
           static_cast<size_t>(kMaxParts + n_kv_heads * row_tiles(n_tok, group)) * stretch_floats(head_dim) * 4;
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
    p.stretches = reinterpret_cast<float *>(at);
    p.row_tiles = static_cast<int>(row_tiles(a.n_tok, a.group));
    p.parts = kv_attend_parts(head_dim, static_cast<int64_t>(a.group) * a.max_q_len);
    if (head_dim == 64) return type == QG_F32 ? launch<64, float>(p, sms, device, s) : launch<64, __half>(p, sms, device, s);
    return type == QG_F32 ? launch<128, float>(p, sms, device, s) : launch<128, __half>(p, sms, device, s);
}

}  // namespace qg
