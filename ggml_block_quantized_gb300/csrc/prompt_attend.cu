// prompt_attend.cu - causal attention over whole packed prompts
// (include/qattn.h, qattn_prompt) on the 5th-generation tensor cores.
//
// A work item is 256 query rows of one key/value head's group: tokens of one
// sequence times `pack` heads (a divisor of the group, the launch's choice), so
// that a short prompt's rows fill a tile. Two 128-row
// tiles A and B share every key/value tile of 128 tokens. The launch has a
// thread block an item, the longest first; the block that a multiprocessor runs
// takes over the next one not yet started (cluster launch control) whenever it
// needs work, and every role runs on into the next item as soon as its own
// operands allow:
//  * warp 0, lane 0: TMA producer: query tiles, and steps: value tile j with key
//    tile j + 1 (128-byte swizzle, 64 channels a box), in a ring of tiles.
//  * warp 1: issues the tcgen05.mma. S = Q K^T into 128 tensor-memory columns a
//    tile, O += P V with P read from tensor memory (f16, over S's columns) and
//    V as it lies in memory (N-major operand). The order PV_A(j) S_A(j+1)
//    PV_B(j) S_B(j+1) keeps the two tiles in turn: the tensor cores have one's
//    products while the other's softmax runs (two issuers of their own fell
//    into step, softmax with softmax: 524 us at 8192 tokens). A product leaves
//    the warp only when the one before it is nearly done, so what the warp does
//    between them is lost to the tensor cores: one wait a step and one a tile.
//  * warp 2: takes items over, finds their rows and publishes them, one ahead
//    (with four, the multiprocessors took up the list before it could balance
//    them: 374 us at 8192 tokens instead of 359).
//  * warp 3: looks through the value tiles on the diagonal. The product P V
//    takes 0 times every value that a row does not see, which is NaN for a
//    value that is not finite; such values are set to 0 in shared memory
//    before the product, and the storing warps add them to the rows that do
//    see them (a weight above 0 times an infinity or NaN is that value).
//  * warps 4..7 and 8..11: softmax of tile A and B, a row a thread: S from
//    tensor memory, running maximum, exp2, P back in f16. O is rescaled in
//    place only when a row's maximum has grown by more than 2^8 over the one
//    its weights refer to (weights then stay below 2^8, far from f16's limit).
//  * warps 12..15: divide O by the rows' sums and store, while the others are
//    in the next item.
// The softmax warps take the registers that the other two warpgroups give up.
// Only tiles on the diagonal are masked; they also hold whatever follows the
// sequence's end. S leaves out the keys that no row of the tile sees (in steps
// of 16); their P is 0.
//
// Bound: the tensor cores for long prompts. 8192 tokens, 32 query and 8 key heads
// of 128: 362 us, 1519 TFLOP/s (386 us a call once calls have followed one another
// for a second: the power limit then holds the clock at 1935 of 2070 MHz), the
// tensor pipe busy 68% of the time (S takes both operands from shared memory at
// its full width and waits for every other access there). 16 prompts of 1 .. 700
// tokens: 45 us; 61 tokens: 8.2 us, one item's chain of copies, products and
// softmax, which short prompts show at every item's start and end.
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cfloat>

#include "kv_cache.cuh"
#include "tc_attend.cuh"

namespace qg {

namespace {

constexpr int kThreads = 16 * 32;
constexpr int kItems = 1;  // items known ahead
constexpr int kSteps = 16;  // barriers of steps: more than the ring can hold (a step has a slot at least)
constexpr int kTileRows = 128, kTileKeys = 128;
constexpr uint32_t kTmemCols = 512;  // S_A, S_B, O_A, O_B at 0, 128, 256, 384
constexpr float kGrow = 8.0f;        // log2 of how far a row's weights may exceed 1

template <int D> struct Shape {
    static constexpr int kTile = 128 * D * 2;  // bytes of a query, key or value tile
    static constexpr int kSlots = D == 128 ? 5 : 10;  // key and value tiles in shared memory
    static constexpr int kTiles = (2 + kSlots) * kTile;
    static constexpr int kSmem = kTiles + 768 + 1024;  // tiles, then barriers, items and sums
    static_assert(kSmem <= kSmemLimit, "shared memory");
    static_assert(kSlots < kSteps, "a barrier for every step in flight");
};

// tc_wait of a whole warp that goes on in either case: a wait that gives up
// sets the abort flag, with which all others of the block give up soon.
__device__ __noinline__ void wait_slow(uint32_t bar, uint32_t parity, volatile int *abort_flag, int32_t *err) {
    if (!__all_sync(0xffffffffu, tc_wait(bar, parity, abort_flag))) {
        record_error(err, kErrConsumerWait);
        *abort_flag = 1;
    }
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *tm, int c0, int c1, int c2, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}

// A work item: 2 x 128 rows.
struct Item {
    int start, end;   // the sequence's rows
    int tok0;         // first token of tile A within the sequence
    int head0;        // first query head
    int tiles[2];     // key/value tiles that A and B see (0: no rows)
    int last;         // 1: no item, the end
};

// A sequence's rows [start, end) and its number of items a head pack (0 where it is left out or past the last).
struct SeqItems {
    int2 rows;
    int n;
};

// Finds items by their index, one warp together. Items come in groups of `packs`
// (one for each head pack); the groups of a launch of up to 32 sequences are
// (token tile l of its sequence, sequence), all tiles of the largest l first, so
// that the longest run first whatever the lengths are. With more sequences that
// order would take several looks at all of them for each item: there the groups
// are (class, sequence, l from its last tile on), class the power of two of the
// sequence's tiles, the largest first. The classes' sizes are counted once a
// block, and since indexes mostly rise from call to call, the search goes on at
// the 32 sequences where the last one ended: a block looks at each sequence about
// once a class, and an item never costs more than one look at all of them. (With
// the first order's search for each item 33 prompts of 5 .. 60 tokens, 32 and 8
// heads of 128, took 26.9 us instead of 24.8, 256 151 instead of 75, 4096 27 ms
// instead of 1.07, growing with the square of the sequences, so that a search could
// outlast the waits' limit; 64 of 700, where the order counts for most, 340 instead
// of 344.)
struct ItemFinder {
    SeqItems q;            // of sequence s0 + lane
    int packs, toks, s0;
    int reach;             // largest end of the sequences up to these
    int before, count;     // lane c: groups of the classes above c, and of c
    int cls, base;         // where the last search ended: its class, the class's groups in the sequences before s0

    __device__ __forceinline__ int class_of() const { return 31 - __clz(q.n); }  // (-1 without tiles)

    // The 32 sequences from s on (0, or 32 after the last ones): their offsets, and what they are as items. Left out is a
    // sequence whose offsets are out of range or fall, and one that begins before the end of an earlier one that is
    // not: so no row is in two, and the launch, which has blocks for n_tok rows, has one for every item.
    __device__ __forceinline__ int2 offsets(const PromptParams &p, int s) const {
        s += threadIdx.x & 31;
        return s < p.n_seq ? make_int2(__ldg(p.offsets + s), __ldg(p.offsets + s + 1)) : make_int2(0, 0);
    }
    __device__ __forceinline__ void settle(const PromptParams &p, int s, int2 rows) {
        const int lane = threadIdx.x & 31, from = s == 0 ? 0 : reach;
        const bool there = s + lane < p.n_seq;
        bool in = there && rows.x >= 0 && rows.y >= rows.x && rows.y <= p.n_tok;
        for (;;) {  // (once more for each sequence that begins too early)
            int end = in ? max(rows.y, from) : from;
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, end, m);
                if (lane >= m) end = max(end, o);
            }
            reach = __shfl_sync(0xffffffffu, end, 31);
            const int earlier = __shfl_up_sync(0xffffffffu, end, 1);
            const uint32_t early = __ballot_sync(0xffffffffu, in && rows.x < (lane == 0 ? from : earlier));
            if (early == 0) break;
            if (lane == __ffs(early) - 1) in = false;
        }
        if (there && !in) record_error(p.err, kErrBadIndex);
        s0 = s;
        q.rows = in ? rows : make_int2(0, 0);
        q.n = (q.rows.y - q.rows.x + toks - 1) / toks;
    }
    __device__ __forceinline__ void look(const PromptParams &p, int s) { settle(p, s, offsets(p, s)); }

    __device__ __forceinline__ void start(const PromptParams &p, int pack) {
        packs = p.n_heads / pack, toks = 2 * (kTileRows / pack);
        const int lane = threadIdx.x & 31;
        before = count = 0;
        cls = -1, base = 0;
        if (p.n_seq > 32) {
            int2 next = offsets(p, 0);
            for (int s = 0; s < p.n_seq; s += 32) {
                const int2 rows = next;
                next = offsets(p, s + 32);
                settle(p, s, rows);
                uint32_t left = __ballot_sync(0xffffffffu, q.n > 0);
                while (left) {
                    const int c = __shfl_sync(0xffffffffu, class_of(), __ffs(left) - 1);
                    const bool in = class_of() == c;
                    const int n = __reduce_add_sync(0xffffffffu, in ? q.n : 0);
                    if (lane == c) count += n;
                    left &= ~__ballot_sync(0xffffffffu, in);
                }
            }
            int from = count;  // groups of the classes from the lane's on
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const int o = __shfl_down_sync(0xffffffffu, from, m);
                if (lane + m < 32) from += o;
            }
            before = from - count;
        }
        look(p, 0);
    }

    // The sequence (its lane among q) and token tile of group `rank`; false past the last.
    __device__ __forceinline__ bool find_by_tile(const PromptParams &p, int rank, int &at, int &tile) const {
        auto tiles_from = [&](int l) { return __reduce_add_sync(0xffffffffu, max(q.n - l, 0)); };
        if (rank >= tiles_from(0)) return false;
        // the level l with tiles_from(l + 1) <= rank < tiles_from(l)
        int lo = 0, hi = (p.n_tok + toks - 1) / toks;  // tiles_from(lo) > rank >= tiles_from(hi)
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (tiles_from(mid) > rank) lo = mid;
            else hi = mid;
        }
        uint32_t has = __ballot_sync(0xffffffffu, q.n > lo);
        for (int skip = rank - tiles_from(lo + 1); skip > 0; --skip) has &= has - 1;  // sequences with a tile lo before it
        at = __ffs(has) - 1;
        tile = lo;
        return true;
    }
    __device__ __forceinline__ bool find_by_class(const PromptParams &p, int rank, int &at, int &tile) {
        const int lane = threadIdx.x & 31;
        const uint32_t is = __ballot_sync(0xffffffffu, rank >= before && rank < before + count);
        if (is == 0) return false;
        const int c = __ffs(is) - 1;
        const int r = rank - __shfl_sync(0xffffffffu, before, c);
        if (c != cls || r < base) {
            cls = c, base = 0;
            if (s0 != 0) look(p, 0);
        }
        for (;;) {
            const int mine = class_of() == c ? q.n : 0;
            int past = mine;
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, past, m);
                if (lane >= m) past += o;
            }
            const uint32_t after = __ballot_sync(0xffffffffu, past > r - base);
            if (after != 0) {
                at = __ffs(after) - 1;
                tile = __shfl_sync(0xffffffffu, past, at) - 1 - (r - base);
                return true;
            }
            base += __shfl_sync(0xffffffffu, past, 31);
            if (s0 + 32 >= p.n_seq) return false;  // (the count above has it among them)
            look(p, s0 + 32);
        }
    }

    // Item `index`; false past the last.
    __device__ __forceinline__ bool find(const PromptParams &p, int pack, int index, Item &item) {
        const int rank = index / packs;
        int at, tile;
        if (!(p.n_seq <= 32 ? find_by_tile(p, rank, at, tile) : find_by_class(p, rank, at, tile))) return false;
        item.start = __shfl_sync(0xffffffffu, q.rows.x, at);
        item.end = __shfl_sync(0xffffffffu, q.rows.y, at);
        item.tok0 = tile * toks;
        item.head0 = (index - rank * packs) * pack;
        const int len = item.end - item.start;
        for (int x = 0; x < 2; ++x) {
            const int first = item.tok0 + x * (toks / 2), past = min(len, first + toks / 2);
            item.tiles[x] = first < len ? (past + kTileKeys - 1) / kTileKeys : 0;
        }
        return true;
    }
};

// Sixteen values.
__device__ __forceinline__ void store16(__half *p, const float (&x)[16], bool wide) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = pack_half2(x[2 * i], x[2 * i + 1]);
    store32(p, w, wide);
}
__device__ __forceinline__ void store16(float *p, const float (&x)[16], bool wide) {
    uint32_t w[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(x[8 * h + i]);
        store32(p + 8 * h, w, wide);
    }
}

// Asks for the next thread block of the launch that has not started; the
// answer, 16 bytes, arrives on `bar`.
__device__ __forceinline__ void ask_block(uint32_t answer, uint32_t bar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(answer),
                 "r"(bar)
                 : "memory");
}
// Its index, -1 where none was left.
__device__ __forceinline__ int asked_block(uint32_t answer) {
    int x;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\tld.shared.b128 r, [%1];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\tmov.s32 %0, -1;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, r;\n\t}"
        : "=r"(x)
        : "r"(answer)
        : "memory");
    return x;
}

// The steps of a block, in order over its items: step 0 of an item has key tile
// 0, step j + 1 value tile j and, but for the last, key tile j + 1; a tile takes
// the next slot of the ring.
template <int SLOTS> struct Step {
    uint32_t n = 0, slot = 0;  // steps, slots so far (slot modulo SLOTS)
    __device__ __forceinline__ uint32_t bar(uint32_t first) const { return first + 8 * (n % kSteps); }
    __device__ __forceinline__ uint32_t parity() const { return n / kSteps & 1u; }
    __device__ __forceinline__ uint32_t take() {  // a slot
        const uint32_t s = slot;
        slot = s + 1 == SLOTS ? 0u : s + 1;
        return s;
    }
};

// Not 0 where one of a word's two f16 is not finite (an exponent field of
// ones, to which one more carries into the sign's place).
__device__ __forceinline__ uint32_t odd_half2(uint32_t w) { return ((w & 0x7C007C00u) + 0x04000400u) & 0x80008000u; }

// The softmax of one tile of S, a row a thread: S at s_t becomes P in place,
// `ref` and `sum` go on, O at o_t is rescaled where a maximum grew too far.
// Columns past `see` count as -inf; the warp's rows all see those up to
// see_all. grow: kGrow, infinite for a row without a query, which would else
// say with whatever it holds when its warp's rows are rescaled (their roundings).
template <int D>
__device__ __forceinline__ void softmax_tile(uint32_t s_t, uint32_t o_t, uint32_t bar, float c, bool negate,
                                             bool first, int see, int see_all, float grow, float &ref, float2 &sum) {
    uint32_t v[4][32];
#pragma unroll
    for (int i = 0; i < 4; ++i) tm_ld32(s_t + 32 * i, v[i]);
#pragma unroll
    for (int i = 0; i < 4; ++i) tm_wait_ld(v[i]);
    if (negate)
#pragma unroll
        for (int i = 0; i < 128; ++i) v[i >> 5][i & 31] ^= 0x80000000u;
    if (see_all < kTileKeys - 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (see_all < 32 * i + 31) {
#pragma unroll
                for (int q = 0; q < 32; ++q)
                    if (32 * i + q > see) v[i][q] = 0xFF800000u;
            }
    }
    float mx[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        mx[i] = __uint_as_float(v[i][0]);
#pragma unroll
        for (int q = 1; q < 31; q += 2) mx[i] = fmaxf(fmaxf(mx[i], __uint_as_float(v[i][q])), __uint_as_float(v[i][q + 1]));
        mx[i] = fmaxf(mx[i], __uint_as_float(v[i][31]));
    }
    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
    if (first) {
        ref = fmaxf(top, -FLT_MAX);  // (scores of -inf alone: weights of 0 beside it, where their own difference is NaN)
    } else if (__any_sync(0xffffffffu, top > ref + grow)) {
        // S of this tile is complete, so P V of the tiles before is, too
        const float next = fmaxf(ref, top), keep = exp2_approx(ref - next);
        ref = next;
        sum.x *= keep, sum.y *= keep;
#pragma unroll 1
        for (int i = 0; i < D; i += 32) {
            uint32_t o[32];
            tm_ld32(o_t + i, o);
            tm_wait_ld(o);
#pragma unroll
            for (int q = 0; q < 32; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * keep);
            tc_st32(o_t + i, o);
        }
    }
    const float2 c2 = make_float2(c, c), r2 = make_float2(-ref, -ref);
    float2 part[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t w[32];
#pragma unroll
        for (int q = 0; q < 32; ++q) {
            float2 e = ffma2(make_float2(__uint_as_float(v[2 * h + (q >> 4)][2 * (q & 15)]),
                                         __uint_as_float(v[2 * h + (q >> 4)][2 * (q & 15) + 1])), c2, r2);
            e.x = exp2_approx(e.x), e.y = exp2_approx(e.y);
            part[q & 1] = fadd2(part[q & 1], e);
            w[q] = pack_half2(e.x, e.y);
        }
        tc_st32(s_t + 32 * h, w);
    }
    tc_wait_st();
    tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
    sum = fadd2(sum, fadd2(part[0], part[1]));
}

template <int D, class TO>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_attend_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                         const __grid_constant__ CUtensorMap map_v, const PromptParams p, const int pack) {
    using Sh = Shape<D>;
    constexpr int kHalves = D / 64;  // boxes of 64 channels
    extern __shared__ __align__(1024) uint8_t smem_raw[];  // (the swizzle's atoms are 1024 bytes)
    const uint32_t q_a = smem_addr(smem_raw), ring_a = q_a + 2 * Sh::kTile, base_a = q_a + Sh::kTiles;
    uint8_t *base = smem_raw + Sh::kTiles;
    // barriers, 8 bytes each (those of the two tiles side by side)
    const uint32_t full = base_a, ready = full + 8 * kSteps, empty = ready + 8 * kSteps, q_full = empty + 8 * kSteps, q_empty = q_full + 16;
    const uint32_t s_full = q_empty + 16, p_ready = s_full + 16, o_full = p_ready + 16, o_empty = o_full + 16, l_full = o_empty + 16;
    const uint32_t item_full = l_full + 16, item_empty = item_full + 8 * kItems, mfinal = item_empty + 8 * kItems, block_bar = mfinal + 8;
    const uint32_t block_answer = base_a + 592;  // 16 bytes
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(base + 608);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(base + 612);
    volatile Item *items = reinterpret_cast<volatile Item *>(base + 616);
    volatile int *odd = reinterpret_cast<volatile int *>(base + 728);       // [item % 8]: diagonal values that are not finite
    volatile float *sums = reinterpret_cast<volatile float *>(base + 768);  // [tile][row]
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kSteps; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(ready + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(q_full + 8 * x, 1);
            mbar_init(q_empty + 8 * x, 1);
            mbar_init(s_full + 8 * x, 1);
            mbar_init(p_ready + 8 * x, 4);
            mbar_init(o_full + 8 * x, 1);
            mbar_init(o_empty + 8 * x, 4);
            mbar_init(l_full + 8 * x, 4);
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(item_full + 8 * i, 1);
            mbar_init(item_empty + 8 * i, 15);  // every warp but 2
        }
        mbar_init(block_bar, 1);
        mbar_init(mfinal, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        tc_alloc(smem_addr(tmem_slot), kTmemCols);
        tc_relinquish();
    }
    if (warp == 2 && lane < 3) {
        const CUtensorMap *m = lane == 0 ? &map_q : lane == 1 ? &map_k : &map_v;
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int tile_toks = kTileRows / pack;
    pdl_wait_prior_grids();
    pdl_allow_dependents();
    // item k of the block as a consumer: all lanes of the warp (or one thread) call it
    auto wait_item = [&](int k) { return sleep_wait<100>(item_full + 8 * (k % kItems), (k / kItems) & 1, abort_flag); };
    auto read_item = [&](int k) {
        const volatile Item &s = items[k % kItems];
        Item it;
        it.start = s.start, it.end = s.end, it.tok0 = s.tok0, it.head0 = s.head0;
        it.tiles[0] = s.tiles[0], it.tiles[1] = s.tiles[1], it.last = s.last;
        return it;
    };
    // keys of key tile j that some row of tile x of the item sees
    auto live_keys = [&](const Item &it, int x, int j) {
        const int past = min(it.end - it.start, it.tok0 + (x + 1) * tile_toks) - j * kTileKeys;
        return past < kTileKeys ? past : kTileKeys;
    };
    // first key tile that some row of the item does not see in full
    auto first_masked = [&](const Item &it) { return (it.tok0 + 1) / kTileKeys; };

    if (warp < 4) {
        fewer_registers<64>();
        if (warp == 0) {
            // ---------------- copies
            Step<Sh::kSlots> step;
            uint32_t n_free = 0;       // steps known to be used up
            int room = Sh::kSlots;     // free slots
            uint64_t single = 0;       // of the last steps (bit n % 64): only one tile
            int used[2] = {0, 0};      // query tiles loaded
            bool ok = true;
            for (int k = 0; ok; ++k) {
                ok = __all_sync(0xffffffffu, wait_item(k));
                if (!ok) break;
                const Item it = read_item(k);
                __syncwarp();
                if (lane == 0) mbar_arrive(item_empty + 8 * (k % kItems));
                if (it.last) break;
                if (lane == 0) {
                    const int kv_head = it.head0 / p.group, n = max(it.tiles[0], it.tiles[1]);
                    auto load = [&](uint32_t dst, const CUtensorMap *map, int head, int row, uint32_t bar) {
                        for (int h = 0; h < kHalves; ++h) tma_load_3d(dst + h * (128 * 128), map, 64 * h, head, row, bar);
                    };
                    for (int j = 0; ok && j <= n; ++j) {
                        const int tiles = (j > 0) + (j < n);
                        while (ok && room < tiles) {
                            ok = sleep_wait<20>(empty + 8 * (n_free % kSteps), n_free / kSteps & 1u, abort_flag);
                            room += (single >> (n_free % 64)) & 1 ? 1 : 2;
                            ++n_free;
                        }
                        if (!ok) break;
                        room -= tiles;
                        single = (single & ~(1ull << (step.n % 64))) | static_cast<uint64_t>(tiles == 1) << (step.n % 64);
                        const uint32_t bar = step.bar(full);
                        mbar_arrive_expect_tx(bar, tiles * Sh::kTile);
                        if (j > 0) load(ring_a + step.take() * Sh::kTile, &map_v, kv_head, it.start + (j - 1) * kTileKeys, bar);
                        if (j < n) load(ring_a + step.take() * Sh::kTile, &map_k, kv_head, it.start + j * kTileKeys, bar);
                        ++step.n;
                        if (j == 0)
#pragma unroll
                            for (int x = 0; x < 2; ++x) {  // the queries, once the last item's are used up
                                if (!ok || it.tiles[x] == 0) continue;
                                if (used[x] > 0) ok = sleep_wait<20>(q_empty + 8 * x, (used[x] - 1) & 1, abort_flag);
                                if (!ok) continue;
                                ++used[x];
                                mbar_arrive_expect_tx(q_full + 8 * x, pack * tile_toks * D * 2);
                                load(q_a + x * Sh::kTile, &map_q, it.head0, it.start + it.tok0 + x * tile_toks, q_full + 8 * x);
                            }
                    }
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
            }
            if (lane == 0) {
                if (!ok) {
                    record_error(p.err, kErrProducerWait);
                    *abort_flag = 1;
                }
                // Leave no copy in flight into this block's shared memory: warps that gave up waiting for one may be gone
                // before it lands, even if nothing held this one up.
                bool landed = true;
                for (; n_free < step.n; ++n_free) landed = mbar_wait_bounded(full + 8 * (n_free % kSteps), n_free / kSteps & 1u) && landed;
                for (int x = 0; x < 2; ++x)
                    if (used[x] > 0) landed = mbar_wait_bounded(q_full + 8 * x, (used[x] - 1) & 1) && landed;
                if (!landed) record_error(p.err, kErrDrainWait);
            }
            __syncwarp();
        } else if (warp == 2) {
            // ---------------- items
            bool ok = true;
            int index = blockIdx.x;
            uint32_t asked = 0;
            ItemFinder finder;
            finder.start(p, pack);
            auto ask = [&]() {
                if (lane == 0) {
                    fence_proxy_async_smem();  // the last answer has been read
                    mbar_arrive_expect_tx(block_bar, 16);
                    ask_block(block_answer, block_bar);
                }
            };
            auto take_answer = [&]() {  // (waited for in every case: it must not arrive after the block's end)
                ok = __all_sync(0xffffffffu, mbar_wait_bounded(block_bar, asked++ & 1u)) && ok;
                if (ok) index = asked_block(block_answer);
                __syncwarp();
            };
            for (int k = 0; ok; ++k) {
                Item it;
                // The launch has blocks for a tile of every sequence that its rows may not fill; those that turn out to be
                // no items are taken over, too, rather than left to start one after another, for a quarter of the time that
                // the others wait for an item at most.
                uint64_t t0 = 0;
                for (;;) {
                    it.last = index < 0 || !finder.find(p, pack, index, it);
                    if (!it.last || index < 0 || !ok) break;
                    const uint64_t now = global_timer_ns();
                    if (t0 == 0) t0 = now;
                    if (!__shfl_sync(0xffffffffu, now - t0 < kWaitLimitNs / 4, 0)) break;
                    ask();
                    take_answer();
                }
                if (!it.last) ask();
                if (ok && k >= kItems) ok = __all_sync(0xffffffffu, sleep_wait<200>(item_empty + 8 * (k % kItems), ((k / kItems) - 1) & 1, abort_flag));
                if (ok && lane == 0) {
                    volatile Item &dst = items[k % kItems];
                    dst.start = it.start, dst.end = it.end, dst.tok0 = it.tok0, dst.head0 = it.head0;
                    dst.tiles[0] = it.tiles[0], dst.tiles[1] = it.tiles[1], dst.last = it.last;
                    mbar_arrive(item_full + 8 * (k % kItems));
                }
                __syncwarp();
                if (it.last) break;
                take_answer();
            }
            if (!ok) {
                if (lane == 0) record_error(p.err, kErrProducerWait);
                *abort_flag = 1;
            }
            __syncwarp();
        } else if (warp == 3) {
            // ---------------- steps' arrival, and value tiles on the diagonal
            Step<Sh::kSlots> step;
            bool ok = true;
            for (int k = 0; ok; ++k) {
                ok = __all_sync(0xffffffffu, wait_item(k));
                if (!ok) break;
                const Item it = read_item(k);
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(item_empty + 8 * (k % kItems));
                    odd[k % 8] = 0;  // (the storing warps are less than eight items behind)
                }
                if (it.last) break;
                const int n = max(it.tiles[0], it.tiles[1]), masked = first_masked(it);
                for (int j = 0; j <= n; ++j) {
                    ok = __all_sync(0xffffffffu, sleep_wait<20>(step.bar(full), step.parity(), abort_flag));
                    if (!ok) break;
                    if (j > 0) {
                        uint4 *mem = reinterpret_cast<uint4 *>(smem_raw + (2 + step.take()) * Sh::kTile);
                        if (j - 1 >= masked) {
                            uint32_t bad = 0;
#pragma unroll 8
                            for (int q = lane; q < Sh::kTile / 16; q += 32) {
                                const uint4 w = mem[q];
                                bad |= odd_half2(w.x) | odd_half2(w.y) | odd_half2(w.z) | odd_half2(w.w);
                            }
                            if (__any_sync(0xffffffffu, bad != 0)) {
                                __half *h = reinterpret_cast<__half *>(mem);
                                for (int q = lane; q < Sh::kTile / 2; q += 32)
                                    if ((__half_as_ushort(h[q]) & 0x7C00u) == 0x7C00u) h[q] = __ushort_as_half(0);
                                fence_proxy_async_smem();
                                if (lane == 0) odd[k % 8] = 1;
                            }
                            __syncwarp();
                        }
                    }
                    if (j < n) step.take();
                    if (lane == 0) mbar_arrive(step.bar(ready));
                    ++step.n;
                }
            }
            if (!ok) {
                if (lane == 0) record_error(p.err, kErrConsumerWait);
                *abort_flag = 1;
            }
            __syncwarp();
        } else {
            // ---------------- mma issuer (the whole warp, one lane issues). The steps are straight-line code
            // but for branches that are alike in all lanes; what a failed wait leaves is not used.
            const uint32_t issue = lane == 0;
            constexpr uint32_t kIdS = tc_idesc_f16(128, kTileKeys), kIdO = tc_idesc_f16(128, D) | kIdescNMajorB;
            const uint32_t q_desc = desc_lo(q_a, 1), k_desc = desc_lo(ring_a, 1), v_desc = desc_lo(ring_a, 128 * 128 / 16);
            constexpr uint32_t kStep = Sh::kTile / 16;  // from tile to tile in a descriptor
            auto wait = [&](uint32_t bar, uint32_t parity) {
                if (!__all_sync(0xffffffffu, mbar_try_wait(bar, parity & 1u))) wait_slow(bar, parity & 1u, abort_flag, p.err);
            };
            struct Work {
                int t[2], n;     // key tiles of A and B, of the item
                int steps[2];    // of the last one's keys, in steps of 16
                int last;
            };
            // item k, published (through shuffles: the same in every lane for the compiler, too)
            auto take_item = [&](int k) {
                const Item it = read_item(k);
                __syncwarp();
                arrive_if(issue, item_empty + 8 * (k % kItems));
                Work w;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    w.t[x] = __shfl_sync(0xffffffffu, it.tiles[x], 0);
                    w.steps[x] = __shfl_sync(0xffffffffu, (live_keys(it, x, it.tiles[x] - 1) + 15) / 16, 0);
                }
                w.n = max(w.t[0], w.t[1]);
                w.last = __shfl_sync(0xffffffffu, it.last | *abort_flag, 0);
                return w;
            };
            // S of tile x with key tile j of its item, in slot `s`
            auto product_s = [&](const Work &w, int x, int j, uint32_t s) {
                const int t = x == 0 ? w.t[0] : w.t[1];
                const bool final = j + 1 == t;
                const uint32_t id = final ? (kIdS & ~(0x3Fu << 17)) | static_cast<uint32_t>((x == 0 ? w.steps[0] : w.steps[1]) * 2) << 17 : kIdS;
                mma_s<D>(issue, tmem + 128 * x, q_desc + x * kStep, k_desc + s * kStep, id, kDescHi);
                commit(issue, s_full + 8 * x);
                if (final) commit(issue, q_empty + 8 * x);
            };
            Step<Sh::kSlots> step;
            uint32_t par_p = 0, par_q = 0, par_o = 3;  // parities of p_ready, q_full and o_empty, by tile
            uint32_t results = 0;                      // tiles that have had a result
            // One piece of code for an item's first step (keys only), the others and the last (values only): what
            // runs once an item would come from instruction memory each time, and nothing hides that here.
            for (int k = 0;; ++k) {
                wait(item_full + 8 * (k % kItems), k / kItems);
                const Work w = take_item(k);
                if (w.last) break;
                for (int j = -1; j < w.n; ++j) {
                    wait(step.bar(ready), step.parity());
                    const uint32_t sv = j < 0 ? 0 : step.take(), sk = j + 1 < w.n ? step.take() : 0;
#pragma unroll 1
                    for (int x = 0; x < 2; ++x) {
                        const int t = x == 0 ? w.t[0] : w.t[1];
                        if (j >= t) continue;
                        uint32_t bar = q_full + 8 * x, parity = par_q;
                        if (j >= 0) {
                            bar = p_ready + 8 * x, parity = par_p;
                            par_p ^= 1u << x;
                        } else {
                            if (t == 0) continue;
                            par_q ^= 1u << x;
                        }
                        wait(bar, parity >> x);
                        if (j == 0) {
                            if (results >> x & 1u) wait(o_empty + 8 * x, par_o >> x);
                            par_o ^= 1u << x;
                            results |= 1u << x;
                        }
                        tc_fence_after();
                        if (j >= 0) mma_pv(issue, tmem + 256 + 128 * x, tmem + 128 * x, v_desc + sv * kStep, kIdO, j, kDescHi);
                        if (j + 1 < t)
                            product_s(w, x, j + 1, sk);
                        else
                            commit(issue, o_full + 8 * x);
                    }
                    commit(issue, step.bar(empty));
                    ++step.n;
                }
            }
            commit(issue, mfinal);  // every mma complete before tensor memory is freed, after a wait that gave up, too
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(mfinal, 0)) && issue) record_error(p.err, kErrDrainWait);
            __syncwarp();
        }
    } else if (warp < 12) {
        // ---------------- softmax of one tile: thread = row = tensor-memory lane 32 (warp % 4) + lane
        more_registers<192>();
        const int x = (warp - 4) >> 2, row = 32 * (warp & 3) + lane;
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        const uint32_t s_t = tmem + lanes + 128 * x, o_t = tmem + lanes + 256 + 128 * x;
        const float c = fmaxf(fabsf(p.scale) * 1.4426950408889634f, 1e-37f);  // not 0, which times -inf would be NaN
        const bool negate = p.scale < 0.0f;
        int n_s = 0, n_items = 0;  // tiles, items of this tile so far
        bool ok = true;
        for (int k = 0; ok; ++k) {
            ok = __all_sync(0xffffffffu, wait_item(k));
            if (!ok) break;
            const Item item = read_item(k);
            __syncwarp();
            if (lane == 0) mbar_arrive(item_empty + 8 * (k % kItems));
            if (item.last) break;
            const int first_tok = item.tok0 + x * tile_toks, tok = first_tok + row / pack;  // within the sequence
            const int n = x == 0 ? item.tiles[0] : item.tiles[1];
            if (n == 0) continue;
            const float grow = item.start + tok < item.end && row < pack * tile_toks ? kGrow : INFINITY;
            float ref = -INFINITY;
            float2 sum = make_float2(0.0f, 0.0f);
            for (int j = 0; j < n; ++j, ++n_s) {
                ok = __all_sync(0xffffffffu, sleep_wait<20>(s_full + 8 * x, n_s & 1, abort_flag));
                if (!ok) break;
                tc_fence_after();
                // the last column that the warp's first row sees
                const int see_all = first_tok + (row & ~31) / pack - j * kTileKeys;
                softmax_tile<D>(s_t, o_t, p_ready + 8 * x, c, negate, j == 0, tok - j * kTileKeys, see_all, grow, ref, sum);
            }
            if (!ok) break;
            // the storing warps must have taken the item before (one of a single tile can be through here
            // while they are still busy with the other tile), or they would miss a phase of l_full
            if (n_items > 0) ok = __all_sync(0xffffffffu, sleep_wait<20>(o_empty + 8 * x, (n_items - 1) & 1, abort_flag));
            if (!ok) break;
            sums[x * 128 + row] = sum.x + sum.y;
            __syncwarp();
            if (lane == 0) mbar_arrive(l_full + 8 * x);
            ++n_items;
        }
        if (!ok) {
            if (lane == 0) record_error(p.err, kErrConsumerWait);
            *abort_flag = 1;
        }
    } else {
        // ---------------- results: O over the rows' sums
        fewer_registers<64>();
        const int row = 32 * (warp & 3) + lane;
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0;
        int n_items[2] = {0, 0};
        bool ok = true;
        for (int k = 0; ok; ++k) {
            ok = __all_sync(0xffffffffu, wait_item(k));
            if (!ok) break;
            const Item item = read_item(k);
            __syncwarp();
            if (lane == 0) mbar_arrive(item_empty + 8 * (k % kItems));
            if (item.last) break;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                if (!ok || item.tiles[x] == 0) continue;
                const int parity = n_items[x]++ & 1;
                ok = __all_sync(0xffffffffu, sleep_wait<100>(l_full + 8 * x, parity, abort_flag) && sleep_wait<40>(o_full + 8 * x, parity, abort_flag));
                if (!ok) continue;
                tc_fence_after();
                const float inv = 1.0f / sums[x * 128 + row];
                const int tok = item.tok0 + x * tile_toks + row / pack, head = item.head0 + row % pack;
                const bool live = item.start + tok < item.end && row < pack * tile_toks;
                TO *out = static_cast<TO *>(p.out) + (static_cast<int64_t>(item.start + tok) * p.n_heads + head) * D;
                const bool patch = odd[k % 8] != 0;
                const __half *values = static_cast<const __half *>(p.v) + item.head0 / p.group * D;
#pragma unroll 1
                for (int i = 0; i < D; i += 32) {
                    uint32_t o[32];
                    tm_ld32(tmem + lanes + 256 + 128 * x + i, o);
                    tm_wait_ld(o);
                    if (i + 32 == D) {  // all of O has been read
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(o_empty + 8 * x);
                    }
#pragma unroll
                    for (int q = 0; q < 32; q += 16) {
                        if (!live) continue;
                        float y[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) y[e] = __uint_as_float(o[q + e]) * inv;
                        if (patch)  // what warp 3 took out of the tiles on the diagonal, as far as this row sees it
                            for (int key = first_masked(item) * kTileKeys; key <= tok; ++key) {
                                const __half *row_v = values + (item.start + key) * p.v_stride + i + q;
#pragma unroll
                                for (int e = 0; e < 16; ++e)
                                    if ((__half_as_ushort(row_v[e]) & 0x7C00u) == 0x7C00u) y[e] += __half2float(row_v[e]);
                            }
                        store16(out + i + q, y, wide);
                    }
                    __syncwarp();
                }
            }
        }
        if (!ok) {
            if (lane == 0) record_error(p.err, kErrConsumerWait);
            *abort_flag = 1;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tc_dealloc(tmem, kTmemCols);
}

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    }();
    return fn;
}

// f16 [n_tok][heads][D], tokens `stride` elements apart, as a 3-D tensor with
// boxes of 64 channels x box_heads x box_toks (128 rows), 128-byte swizzle;
// tokens past the last read as zeros.
bool encode_rows(CUtensorMap *tm, const void *base, int64_t n_tok, int heads, int d, int64_t stride, int box_heads, int box_toks) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(n_tok)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(stride) * 2};
    const cuuint32_t box[3] = {64u, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_toks)};
    const cuuint32_t estr[3] = {1u, 1u, 1u};
    return enc(tm, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, class TO> cudaError_t launch(const PromptParams &p, int device, cudaStream_t s) {
    // Heads that share a tile: the largest divisor of the group that leaves at most 8 of a tile's rows without a
    // query. (With powers of two only, 9 prompts of 30 .. 200 tokens, 56 heads over 8 of 128: 25.6 us instead of 17.9;
    // 32 prompts of 5 .. 60, 24 heads over 8: 26.9 instead of 14.2.)
    int pack = std::min(p.group, kTileRows);
    while (p.group % pack != 0 || kTileRows / pack * pack < kTileRows - 8) --pack;
    CUtensorMap mq, mk, mv;
    if (!encode_rows(&mq, p.q, p.n_tok, p.n_heads, D, p.q_stride, pack, kTileRows / pack) ||
        !encode_rows(&mk, p.k, p.n_tok, p.n_kv_heads, D, p.k_stride, 1, kTileKeys) ||
        !encode_rows(&mv, p.v, p.n_tok, p.n_kv_heads, D, p.v_stride, 1, kTileKeys)) {
        g_launch_step = "cuTensorMapEncodeTiled";
        return cudaErrorInvalidValue;
    }
    static std::atomic<uint64_t> done{0};
    const uint64_t bit = 1ull << (device & 63);
    if (!(done.load(std::memory_order_acquire) & bit)) {
        const cudaError_t e = cudaFuncSetAttribute(prompt_attend_kernel<D, TO>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   Shape<D>::kSmem);
        if (e != cudaSuccess) return e;
        done.fetch_or(bit, std::memory_order_acq_rel);
    }
    // every sequence has at most one tile that its rows do not fill, and no row is in two
    const int toks = 2 * (kTileRows / pack);
    const int64_t items = (static_cast<int64_t>(p.n_tok) / toks + p.n_seq) * (p.n_heads / pack);
    if (items > INT32_MAX) return cudaErrorInvalidValue;
    return launch_pdl(prompt_attend_kernel<D, TO>, static_cast<int>(items), kThreads, Shape<D>::kSmem, s, mq, mk, mv, p, pack);
}

}  // namespace

cudaError_t launch_prompt_attend(const PromptParams &p, int head_dim, int out_type, int, int device, cudaStream_t s) {
    if (head_dim == 64) return out_type == QG_F32 ? launch<64, float>(p, device, s) : launch<64, __half>(p, device, s);
    return out_type == QG_F32 ? launch<128, float>(p, device, s) : launch<128, __half>(p, device, s);
}

}  // namespace qg
