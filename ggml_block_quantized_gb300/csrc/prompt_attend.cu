// prompt_attend.cu - causal attention over whole packed prompts
// (include/qattn.h, qattn_prompt) on the 5th-generation tensor cores.
//
// A work item is 256 query rows of one key/value head's group: tokens of one
// sequence times `pack` heads (the largest power of two that divides the
// group, at most 128), so that a short prompt's rows fill a tile. Two 128-row
// tiles A and B share every key/value tile of 128 tokens. Per thread block:
//  * warp 0, lane 0: TMA producer. The two query tiles, then key and value
//    tiles in turn into a ring (128-byte swizzle, 64 channels a box).
//  * warp 1, lane 0: issues tcgen05.mma. S = Q K^T into 128 tensor-memory
//    columns a tile, O += P V with P read from tensor memory (f16, over S's
//    columns) and V as it lies in memory (N-major operand). The order
//    PV_A(j) S_A(j+1) PV_B(j) S_B(j+1) keeps the tensor cores on one tile while
//    the other one's softmax runs.
//  * warps 2..5 and 6..9: softmax of tile A and B, a row a thread: S from
//    tensor memory, running maximum, exp2, P back in f16. O is rescaled in
//    place only when a row's maximum has grown by more than 2^8 over the one
//    its weights refer to (weights then stay below 2^8, far from f16's limit);
//    the same threads divide by the sum and store.
// Only tiles on the diagonal are masked. The product P V takes 0 times every
// unseen value, which is NaN for a value that is not finite: a row whose
// result is not finite is computed again, over its own rows alone, by one warp.
#include <cudaTypedefs.h>

#include <atomic>

#include "kv_cache.cuh"
#include "tc_common.cuh"

namespace qg {

namespace {

constexpr int kThreads = 10 * 32;
constexpr int kTileRows = 128, kTileKeys = 128;
constexpr uint32_t kTmemCols = 512;  // S_A, S_B, O_A, O_B at 0, 128, 256, 384
constexpr float kGrow = 8.0f;        // log2 of how far a row's weights may exceed 1

template <int D> struct Shape {
    static constexpr int kTile = 128 * D * 2;  // bytes of a query, key or value tile
    static constexpr int kStages = D == 128 ? 5 : 10;
    static constexpr int kSmem = 1024 + 1024 + (2 + kStages) * kTile;  // alignment, barriers, tiles
    static_assert(kSmem <= kSmemLimit, "shared memory");
};

// Two-operand forms of tcgen05.mma, kind::f16, f32 accumulators.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// Shared-memory descriptor of a 128-byte-swizzled N-major operand (64-element
// rows of N, one row a k): the stride between 64-element parts of N, and
// between groups of 8 k (one atom, 1024 bytes).
__device__ __forceinline__ uint64_t desc_n_major(uint32_t start, uint32_t n_stride) {
    return static_cast<uint64_t>((start >> 4) & 0x3FFFu) | (static_cast<uint64_t>((n_stride >> 4) & 0x3FFFu) << 16) |
           (static_cast<uint64_t>((1024u >> 4) & 0x3FFFu) << 32) | (static_cast<uint64_t>(1) << 46) |
           (static_cast<uint64_t>(2) << 61);
}
constexpr uint32_t kIdescNMajorB = 1u << 16;

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *tm, int c0, int c1, int c2, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}

// 32 columns of this warp's 32 lanes, without the wait.
__device__ __forceinline__ void tm_ld32(uint32_t taddr, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr)
        : "memory");
}
// Waits for this thread's tensor-memory loads; the registers pass through it,
// so that nothing reads them earlier.
__device__ __forceinline__ void tm_wait_ld(uint32_t (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                   "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]),
                   "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]),
                   "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]),
                   "+r"(v[30]), "+r"(v[31])
                 :
                 : "memory");
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// A work item: 2 x 128 rows.
struct Item {
    int start, end;   // the sequence's rows
    int tok0;         // first token of tile A within the sequence
    int head0;        // first query head
    int tiles[2];     // key/value tiles that A and B see (0: no rows)
};

// Sequence s as rows [start, end); empty where its offsets are out of range.
__device__ __forceinline__ int2 seq_rows(const PromptParams &p, int s) {
    const int a = __ldg(p.offsets + s), b = __ldg(p.offsets + s + 1);
    if (a < 0 || b < a || b > p.n_tok) {
        record_error(p.err, kErrBadIndex);
        return make_int2(0, 0);
    }
    return make_int2(a, b);
}

// Item `index` in the order of falling length: items are (token tile l of its
// sequence, sequence, head pack), all tiles of the largest l first, so that the
// longest run first whatever the lengths are. One warp; false past the last.
__device__ __forceinline__ bool find_item(const PromptParams &p, int pack, int index, Item &item) {
    const int lane = threadIdx.x & 31, packs = p.n_heads / pack, toks = 2 * kTileRows / pack;
    const int rank = index / packs;
    // tiles with number >= l
    auto tiles_from = [&](int l) {
        int n = 0;
        for (int s = lane; s < p.n_seq; s += 32) {
            const int2 r = seq_rows(p, s);
            const int t = (r.y - r.x + toks - 1) / toks;
            n += t > l ? t - l : 0;
        }
        return __reduce_add_sync(0xffffffffu, n);
    };
    if (rank >= tiles_from(0)) return false;
    // the level l with tiles_from(l + 1) <= rank < tiles_from(l)
    int lo = 0, hi = (p.n_tok + toks - 1) / toks;  // tiles_from(lo) > rank >= tiles_from(hi)
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (tiles_from(mid) > rank) lo = mid;
        else hi = mid;
    }
    int skip = rank - tiles_from(lo + 1);  // sequences with a tile lo before the item's
    for (int s0 = 0; s0 < p.n_seq; s0 += 32) {
        const int s = s0 + lane;
        int2 r = make_int2(0, 0);
        if (s < p.n_seq) r = seq_rows(p, s);
        uint32_t has = __ballot_sync(0xffffffffu, (r.y - r.x + toks - 1) / toks > lo);
        const int n = __popc(has);
        if (skip >= n) {
            skip -= n;
            continue;
        }
        for (; skip > 0; --skip) has &= has - 1;
        const int at = __ffs(has) - 1;
        item.start = __shfl_sync(0xffffffffu, r.x, at);
        item.end = __shfl_sync(0xffffffffu, r.y, at);
        break;
    }
    item.tok0 = lo * toks;
    item.head0 = (index % packs) * pack;
    const int len = item.end - item.start;
    for (int x = 0; x < 2; ++x) {
        const int first = item.tok0 + x * (toks / 2), past = min(len, first + toks / 2);
        item.tiles[x] = first < len ? (past + kTileKeys - 1) / kTileKeys : 0;
    }
    return true;
}

__device__ __forceinline__ void store8(__half *p, const float (&x)[8]) {
    *reinterpret_cast<uint4 *>(p) =
        make_uint4(pack_half2(x[0], x[1]), pack_half2(x[2], x[3]), pack_half2(x[4], x[5]), pack_half2(x[6], x[7]));
}
__device__ __forceinline__ void store8(float *p, const float (&x)[8]) {
    *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4 *>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}

// One query row over the rows it sees, by one warp, in f32.
template <int D, class TO>
__device__ __noinline__ void attend_row(const PromptParams &p, int start, int row, int head) {
    constexpr int kPer = D / 32;
    const int lane = threadIdx.x & 31, hk = head / p.group;
    const __half *q = static_cast<const __half *>(p.q) + row * p.q_stride + head * D;
    const __half *kb = static_cast<const __half *>(p.k) + hk * D, *vb = static_cast<const __half *>(p.v) + hk * D;
    float m = -INFINITY, l = 0.0f, o[kPer] = {};
    for (int t0 = start; t0 <= row; t0 += 32) {
        const int t = t0 + lane;
        float sc = -INFINITY;
        if (t <= row) {
            sc = 0.0f;
            for (int i = 0; i < D; ++i) sc += __half2float(q[i]) * __half2float(kb[t * p.k_stride + i]);
            sc *= p.scale;
        }
        float mt = sc;
        for (int k = 16; k; k >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, k));
        const float mn = fmaxf(m, mt);
        const float base = mn == -INFINITY ? 0.0f : mn;
        const float keep = expf(m - base);
        const float w = t <= row ? expf(sc - base) : 0.0f;
        m = mn;
        l = l * keep + w;
        for (int k = 0; k < kPer; ++k) o[k] *= keep;
        for (int j = 0; j < 32 && t0 + j <= row; ++j) {
            const float wj = __shfl_sync(0xffffffffu, w, j);
            for (int k = 0; k < kPer; ++k) o[k] += wj * __half2float(vb[(t0 + j) * p.v_stride + 32 * k + lane]);
        }
    }
    for (int k = 16; k; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
    TO *out = static_cast<TO *>(p.out) + (static_cast<int64_t>(row) * p.n_heads + head) * D;
    for (int k = 0; k < kPer; ++k) out[32 * k + lane] = static_cast<TO>(o[k] / l);
}

template <int D, class TO>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_attend_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                         const __grid_constant__ CUtensorMap map_v, const PromptParams p, const int pack) {
    using Sh = Shape<D>;
    constexpr int kHalves = D / 64;  // boxes of 64 channels
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_a = smem_addr(smem_raw), base_a = (raw_a + 1023u) & ~1023u;
    uint8_t *base = smem_raw + (base_a - raw_a);
    // full[stages] | empty[stages] | q | s_full[2] | p_ready[2] | o_full[2] | final | tensor-memory address | abort | item
    const uint32_t full0 = base_a, empty0 = base_a + 8 * Sh::kStages, bar_q = base_a + 16 * Sh::kStages;
    const uint32_t s_full = bar_q + 8, p_ready = bar_q + 24, o_full = bar_q + 40, mfinal = bar_q + 56;
    uint8_t *misc = base + 16 * Sh::kStages + 64;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(misc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(misc + 4);
    volatile int *found = reinterpret_cast<volatile int *>(misc + 8);
    Item *shared_item = reinterpret_cast<Item *>(misc + 16);
    const uint32_t q_a = base_a + 1024, ring_a = q_a + 2 * Sh::kTile;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < Sh::kStages; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        mbar_init(bar_q, 1);
        for (int x = 0; x < 2; ++x) {
            mbar_init(s_full + 8 * x, 1);
            mbar_init(p_ready + 8 * x, 4);
            mbar_init(o_full + 8 * x, 1);
        }
        mbar_init(mfinal, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        tc_alloc(smem_addr(tmem_slot), kTmemCols);
        tc_relinquish();
    }
    pdl_wait_prior_grids();
    pdl_allow_dependents();
    if (warp == 0) {
        Item it;
        const bool ok = find_item(p, pack, blockIdx.x, it);
        if (lane == 0) {
            *found = ok;
            if (ok) *shared_item = it;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if (!*found) {
        if (warp == 1) tc_dealloc(tmem, kTmemCols);
        return;
    }
    const Item item = *shared_item;
    const int n_tiles = max(item.tiles[0], item.tiles[1]);
    const int tile_toks = kTileRows / pack;

    if (warp == 0) {
        // ---------------- producer
        if (lane == 0) {
            const int kv_head = item.head0 / p.group;
            mbar_arrive_expect_tx(bar_q, 2 * Sh::kTile);
            for (int x = 0; x < 2; ++x)
                for (int h = 0; h < kHalves; ++h)
                    tma_load_3d(q_a + x * Sh::kTile + h * (128 * 128), &map_q, 64 * h, item.head0,
                                item.start + item.tok0 + x * tile_toks, bar_q);
            int s = 0, issued = 0;
            uint32_t ph = 0;
            for (int i = 0; i < 2 * n_tiles; ++i) {
                if (issued >= Sh::kStages && !tc_wait(empty0 + 8 * s, ph ^ 1u, abort_flag)) {
                    record_error(p.err, kErrProducerWait);
                    *abort_flag = 1;
                    break;
                }
                mbar_arrive_expect_tx(full0 + 8 * s, Sh::kTile);
                for (int h = 0; h < kHalves; ++h)
                    tma_load_3d(ring_a + s * Sh::kTile + h * (128 * 128), i & 1 ? &map_v : &map_k, 64 * h, kv_head,
                                item.start + (i >> 1) * kTileKeys, full0 + 8 * s);
                ++issued;
                if (++s == Sh::kStages) s = 0, ph ^= 1u;
            }
            // leave no copy in flight into this block's shared memory
            for (int k = issued > Sh::kStages ? issued - Sh::kStages : 0; k < issued; ++k)
                if (!mbar_wait_bounded(full0 + 8 * (k % Sh::kStages), (k / Sh::kStages) & 1)) {
                    record_error(p.err, kErrDrainWait);
                    break;
                }
            if (!mbar_wait_bounded(bar_q, 0u)) record_error(p.err, kErrDrainWait);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------- mma issuer
        if (lane == 0) {
            const uint32_t id_s = tc_idesc_f16(128, kTileKeys), id_o = tc_idesc_f16(128, D) | kIdescNMajorB;
            bool ok = tc_wait(bar_q, 0u, abort_flag);
            auto wait_stage = [&](int i) {  // key tile j is ring entry 2 j, value tile j 2 j + 1
                return tc_wait(full0 + 8 * (i % Sh::kStages), (i / Sh::kStages) & 1, abort_flag);
            };
            auto stage = [&](int i) { return ring_a + (i % Sh::kStages) * Sh::kTile; };
            auto product_s = [&](int x, int j) {
                const uint64_t a = tc_smem_desc(q_a + x * Sh::kTile, 1024), b = tc_smem_desc(stage(2 * j), 1024);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint64_t off = static_cast<uint64_t>((k >> 2) * (128 * 128 / 16) + (k & 3) * 2);
                    mma_ss(tmem + 128 * x, a + off, b + off, id_s, k != 0);
                }
                tc_commit(s_full + 8 * x);
            };
            if (ok) ok = wait_stage(0);
            tc_fence_after();
            if (ok)
                for (int x = 0; x < 2; ++x)
                    if (item.tiles[x] > 0) product_s(x, 0);
            if (ok) tc_commit(empty0);
            for (int j = 0; ok && j < n_tiles; ++j) {
                ok = wait_stage(2 * j + 1);
                if (ok && j + 1 < n_tiles) ok = wait_stage(2 * j + 2);
                for (int x = 0; x < 2 && ok; ++x) {
                    if (j >= item.tiles[x]) continue;
                    ok = tc_wait(p_ready + 8 * x, j & 1, abort_flag);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t v = desc_n_major(stage(2 * j + 1), 128 * 128);
#pragma unroll
                    for (int k = 0; k < kTileKeys / 16; ++k)
                        mma_ts(tmem + 256 + 128 * x, tmem + 128 * x + 8 * k, v + static_cast<uint64_t>(k * (2048 / 16)), id_o,
                               (j | k) != 0);
                    if (j + 1 < item.tiles[x]) product_s(x, j + 1);
                    else tc_commit(o_full + 8 * x);
                }
                if (!ok) break;
                tc_commit(empty0 + 8 * ((2 * j + 1) % Sh::kStages));
                if (j + 1 < n_tiles) tc_commit(empty0 + 8 * ((2 * j + 2) % Sh::kStages));
            }
            if (!ok) {
                record_error(p.err, kErrConsumerWait);
                *abort_flag = 1;
            }
            tc_commit(mfinal);  // every mma complete before tensor memory is freed
            if (!mbar_wait_bounded(mfinal, 0u)) record_error(p.err, kErrDrainWait);
        }
        __syncwarp();
    } else {
        // ---------------- softmax of one tile: thread = row = tensor-memory lane 32 (warp % 4) + lane
        const int x = (warp - 2) >> 2, row = 32 * (warp & 3) + lane;
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        const uint32_t s_t = tmem + lanes + 128 * x, o_t = tmem + lanes + 256 + 128 * x;
        const int tok = item.tok0 + x * tile_toks + row / pack;  // within the sequence
        const int first_tok = item.tok0 + x * tile_toks;
        const float c = fmaxf(fabsf(p.scale) * 1.4426950408889634f, 1e-37f);  // not 0, which times -inf would be NaN
        const bool negate = p.scale < 0.0f;
        float ref = -INFINITY;
        float2 sum = make_float2(0.0f, 0.0f);
        bool ok = true;
        for (int j = 0; j < item.tiles[x]; ++j) {
            ok = __all_sync(0xffffffffu, tc_wait(s_full + 8 * x, j & 1, abort_flag));
            if (!ok) break;
            tc_fence_after();
            uint32_t v[4][32];
#pragma unroll
            for (int i = 0; i < 4; ++i) tm_ld32(s_t + 32 * i, v[i]);
#pragma unroll
            for (int i = 0; i < 4; ++i) tm_wait_ld(v[i]);
            if (negate)
#pragma unroll
                for (int i = 0; i < 128; ++i) v[i >> 5][i & 31] ^= 0x80000000u;
            const int key0 = j * kTileKeys;
            if (key0 + kTileKeys - 1 > first_tok) {  // some row does not see every key
                const int see = tok - key0;          // columns 0 .. see
#pragma unroll
                for (int i = 0; i < 128; ++i)
                    if (i > see) v[i >> 5][i & 31] = 0xFF800000u;
            }
            float mx[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                mx[i] = __uint_as_float(v[i][0]);
#pragma unroll
                for (int k = 1; k < 31; k += 2) mx[i] = fmaxf(fmaxf(mx[i], __uint_as_float(v[i][k])), __uint_as_float(v[i][k + 1]));
                mx[i] = fmaxf(mx[i], __uint_as_float(v[i][31]));
            }
            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
            if (j == 0) {
                ref = top;
            } else if (__any_sync(0xffffffffu, top > ref + kGrow)) {
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
                    for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * keep);
                    tc_st32(o_t + i, o);
                }
            }
            const float2 c2 = make_float2(c, c), r2 = make_float2(-ref, -ref);
            float2 part[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                uint32_t w[32];
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    float2 e = ffma2(make_float2(__uint_as_float(v[i + (k >> 4)][2 * (k & 15)]),
                                                 __uint_as_float(v[i + (k >> 4)][2 * (k & 15) + 1])), c2, r2);
                    e.x = exp2_approx(e.x), e.y = exp2_approx(e.y);
                    part[k & 1] = fadd2(part[k & 1], e);
                    w[k] = pack_half2(e.x, e.y);
                }
                tc_st32(s_t + 16 * i, w);
            }
            sum = fadd2(sum, fadd2(part[0], part[1]));
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_ready + 8 * x);
        }
        // ---- the rows' results
        if (ok && item.tiles[x] > 0) {
            ok = __all_sync(0xffffffffu, tc_wait(o_full + 8 * x, 0u, abort_flag));
            if (ok) {
                tc_fence_after();
                const float inv = 1.0f / (sum.x + sum.y);
                const bool live = item.start + tok < item.end;
                const int head = item.head0 + row % pack;
                TO *out = static_cast<TO *>(p.out) + (static_cast<int64_t>(item.start + tok) * p.n_heads + head) * D;
                float check = 0.0f;  // 0 times every value: NaN if one is not finite
#pragma unroll 1
                for (int i = 0; i < D; i += 32) {
                    uint32_t o[32];
                    tm_ld32(o_t + i, o);
                    tm_wait_ld(o);
#pragma unroll
                    for (int k = 0; k < 32; k += 8) {
                        float y[8];
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            y[q] = __uint_as_float(o[k + q]) * inv;
                            check = fmaf(y[q], 0.0f, check);
                        }
                        if (live) store8(out + i + k, y);
                    }
                }
                uint32_t bad = __ballot_sync(0xffffffffu, live && check != 0.0f);
                for (; bad; bad &= bad - 1) {
                    const int src = __ffs(bad) - 1;
                    attend_row<D, TO>(p, item.start, item.start + __shfl_sync(0xffffffffu, tok, src),
                                      __shfl_sync(0xffffffffu, head, src));
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
    // heads that share a tile: the largest power of two that divides the group
    int pack = p.group & -p.group;
    if (pack > kTileRows) pack = kTileRows;
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
    // every sequence has at most one tile that its rows do not fill
    const int toks = 2 * kTileRows / pack;
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
