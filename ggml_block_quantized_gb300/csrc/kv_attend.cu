// kv_attend.cu - attention of new tokens over the 4-bit paged cache
// (include/qattn.h, qkv_attend), split over the cache's length.
//
// Work. A segment is one (sequence, key/value head, row tile): up to 8 NT query
// rows (token-major over the sequence's queries and the head's group) against
// the sequence's tokens, cut into tiles of 32 tokens (two cache groups). All
// segments' tiles, in order, form one list that the resident thread blocks
// share out in equal contiguous parts (at least one tile a warp), whatever the
// lengths are: they are read on the device. A part that ends inside a segment
// leaves its running maximum, sum and values in the workspace, and a second
// kernel joins the parts of each such segment in order (deterministic).
//
// A block has four consumer warps and one producer warp. The producer walks
// the list, looks the pages up 32 at a time and sends each tile's two groups
// (18 D bytes each, contiguous) into a shared-memory ring with bulk copies;
// consumer w takes tiles w, w + 4, ... of the block's part and keeps its own
// softmax statistics; the four join through shared memory at a segment's end.
//
// Arithmetic, on mma.sync.m16n8k16 (f16 operands, f32 sums), tokens or
// channels as the 16 rows and query rows as the 8 columns, so that a decode
// step's few rows waste little:
//  * codes as A: for f16 queries the key codes themselves. A 4-byte code word
//    masked with 0x000F000F holds two codes as f16 subnormals c 2^-24 (with
//    0x00F000F0, 16 c 2^-24): one logic operation for two elements and no
//    conversion; the queries of low-nibble elements carry the missing 16, and
//    the offset 8 of (code - 8) is the accumulator's start value, -8 sum of the
//    block's q. The tensor cores align subnormals unnormalised, which costs
//    about 7 of the sum's 24 bits: enough for f16 queries, not for f32 ones and
//    not for values (a sum that nearly cancels), so those take code - 8 in f16,
//    exact, for one more packed operation.
//  * scores: per block the f32 sum is multiplied by the token's key scale.
//    Queries are scaled by a power of two to a largest magnitude of 2^10 ..
//    2^11 (exact).
//  * values: B = weight x value scale per token and block (the scale varies
//    along the summed axis), transposed among lanes with movmatrix. The
//    softmax's running reference is not the largest score but the largest sum of
//    a score and the exponent field of its token's largest value scale, less 21,
//    and is raised only when such a sum passes it by 29: every product is then
//    below 2^15 and a row's largest above 2^6, whatever the values' size, so that
//    what f16 loses at its end, 2^-25 of a product, is 2^-31 of the largest.
//    Weights, their sum and the accumulators share that reference, so it cancels.
//    (Raised for every larger score, with a maximum over the lanes each tile,
//    131071 tokens took 50.1 us instead of 48.0. With the largest score and the
//    largest scale of a lane's four tokens, whichever tokens they are of, 24
//    sequences took 58.1 us instead of 59.4, but strong scores of small values
//    beside large ones fell below f16: results off by a third.)
// So codes enter exactly and only q and the weights are rounded: f16 queries
// are exact and the weights take one f16 (2^-11 relative); for f32 both are
// split in two f16 parts and each product is formed twice.
//
// Bound: the cache's bytes would take 58% (f16 queries) and 43% (f32) of the time.
// The rest is the consumers' instructions, about 700 and 900 a tile: the issue
// slots are 56% busy, and a warp that does not issue waits for a result of its
// own, for the math pipes or for its turn, about alike, with the 12 warps a
// multiprocessor that 128 registers allow (14 in two larger blocks were no
// faster). 24 sequences of 200 .. 4096 tokens, 32 heads of 128, f16: 59.3 us, 4.0
// TB/s; one of 131071, 64 query and 8 key heads, f32: 51.5 us, 2.9 TB/s; 777
// tokens, 32 and 8 heads, f32: 8.1 us, of which a tile's work is 1.1: the rest is
// the place in the list (1.0), the queries (1.3), the join (0.5 and 1.1) and the
// launches.
#include <atomic>
#include <cfloat>

#include "kv_cache.cuh"
#include "tc_common.cuh"

namespace qg {

namespace {

constexpr int kWarps = 4;                  // consumer warps
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kTile = 32;                  // tokens of a tile
constexpr int kStart = 11;                 // units of the list that a segment's start counts for: see seq_units
constexpr int kLeast = kWarps;             // units of a part at least
constexpr float kLow = 21.0f, kHigh = 29.0f;  // of the softmax's running reference, above
constexpr int kMaxCtas = 640;              // thread blocks of a launch (workspace is sized for them)

template <int D, int NT, int TERMS> struct Shape {
    using G = KvGroup<D>;
    static constexpr int kTileBytes = 2 * G::kBytes;
    static constexpr int kSlots = D == 128 ? 8 : 16;
    static constexpr int kRows = 8 * NT;
    static constexpr int kRawRow = D * (TERMS == 2 ? 4 : 2);                   // bytes of a query row
    static constexpr int kOffRing = 1024;
    static constexpr int kOffRaw = kOffRing + kSlots * kTileBytes;             // a segment's query rows
    static constexpr int kOffQ = kOffRaw + kRows * kRawRow;                    // [term][nt][block][lane] 16 bytes
    static constexpr int kOffInit = kOffQ + TERMS * NT * G::kNB * 512;         // [nt][block][4 pairs of columns, twice] f32
    static constexpr int kOffRow = kOffInit + NT * G::kNB * 64;                // factor f32, limit and place in out int [rows]
    static constexpr int kOffStat = kOffRow + kRows * 16;                      // [row][warp] reference, sum
    static constexpr int kJoinPitch = D + 4;
    static constexpr int kOffJoin = kOffStat + kWarps * kRows * 8;             // [warp][rows][kJoinPitch]
    static constexpr int kSmem = kOffJoin + kWarps * kRows * kJoinPitch * 4;
    static constexpr int kCtas = NT == 1 ? 3 : 2;                              // resident blocks a multiprocessor
};

// A partial result: rows x D values, then the rows' maxima and sums.
__host__ __device__ constexpr int64_t part_floats(int d, int rows) { return static_cast<int64_t>(rows) * (d + 2); }

// What a thread block leaves for the join: the segment that starts in its part
// and goes on in the next ones. At the workspace's start, one a block.
struct Cut {
    int parts;      // this block's and the following ones'; 0: no such segment
    int rows, row0; // rows of the segment, its first row among the sequence's
    int q0, head;   // first query row of the sequence, key/value head
    int pad[3];
};
static_assert(sizeof(Cut) == 32, "two 16-byte loads");
constexpr int64_t kCutFloats = kMaxCtas * static_cast<int64_t>(sizeof(Cut)) / 4;

struct Seq {
    int len, m, q0;  // tokens in the cache, queries, first query row
};

// Sequence s, checked: no queries (m = 0) where its offsets are out of range.
__device__ __forceinline__ Seq load_seq(const KvAttendParams &p, int s) {
    Seq q;
    q.q0 = s;
    q.m = 1;
    if (p.q_offsets != nullptr) {
        q.q0 = __ldg(p.q_offsets + s);
        const int q1 = __ldg(p.q_offsets + s + 1);
        q.m = q1 - q.q0;
        if (q.q0 < 0 || q1 < q.q0 || q1 > p.n_tok || q.m > p.max_q_len) {
            record_error(p.err, kErrBadIndex);
            q.m = 0;
        }
    }
    q.len = __ldg(p.lengths + s);
    const int64_t room = p.table_stride * p.c.page_size;
    if (q.len < 0 || q.len > room) {
        record_error(p.err, kErrBadIndex);
        q.len = q.len < 0 ? 0 : static_cast<int>(room);
    }
    return q;
}

__device__ __forceinline__ int row_tiles(const KvAttendParams &p, const Seq &q, int rows) {
    return (q.m * p.group + rows - 1) / rows;
}
// Units of a segment: its tiles, and kStart for its queries and its join. (24
// sequences of 200 .. 4096 tokens, 32 heads: 70.0 us at 3, 62.9 at 6, 58.4 to 59.1
// at 8 to 12, 60.9 at 20; 16 of 5 .. 6000, 8 heads, 5 queries: 29.5, 25.0, 22.7 at
// 8, 20.7 at 9, 19.6 at 11, 20.6 at 20. One number for every head size, type and
// row count: only these two were swept, and 131071 tokens in f32 took 49.1 us at 8
// and 50.4 at 11.)
__device__ __forceinline__ int tok_tiles(const Seq &q) { return kStart + (q.len + kTile - 1) / kTile; }
__device__ __forceinline__ int64_t seq_units(const KvAttendParams &p, int s, int rows) {
    const Seq q = load_seq(p, s);
    return q.m == 0 ? 0 : static_cast<int64_t>(p.c.n_heads) * row_tiles(p, q, rows) * tok_tiles(q);
}

// Where a block's part begins: the sequence and the unit within it.
struct Place {
    int seq;
    int64_t at;     // units of this sequence before the part
    int64_t units;  // of all sequences
    int64_t share;  // units of a block's part
};

// The parts' size.
__device__ __forceinline__ int64_t part_share(int64_t units, int ctas) {
    const int64_t share = (units + ctas - 1) / ctas;
    return share < kLeast ? kLeast : share;
}

// Finds the part of block `cta` of `ctas`: up to 32 sequences, every warp by
// itself. seq = n_seq where the part is empty.
__device__ __forceinline__ Place locate_few(const KvAttendParams &p, int rows, int64_t cta, int ctas) {
    const int lane = threadIdx.x & 31;
    const int64_t mine = lane < p.n_seq ? seq_units(p, lane, rows) : 0;
    int64_t past = mine;  // units of the sequences up to this one
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, past, m);
        if (lane >= m) past += o;
    }
    Place r;
    r.units = __shfl_sync(0xffffffffu, past, 31);
    r.share = part_share(r.units, ctas);
    const int64_t u = cta * r.share;
    const uint32_t after = __ballot_sync(0xffffffffu, past > u);
    r.seq = after == 0 ? p.n_seq : __ffs(after) - 1;
    r.at = u - __shfl_sync(0xffffffffu, past - mine, r.seq & 31);
    return r;
}

// The same for any number of sequences, with the whole block (every thread gets
// the result). 32 sequences of 100 tokens take 10.7 us in all with it and 10.3 with
// the one above; 777 tokens of one 8.0 and 7.9.
template <int THREADS> __device__ Place locate(const KvAttendParams &p, int rows, int64_t cta, int ctas) {
    __shared__ int64_t warp_sum[THREADS / 32];
    __shared__ int found_seq;
    __shared__ int64_t found_at;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t first = tid < p.n_seq ? seq_units(p, tid, rows) : 0;
    int64_t v = first;
    for (int s = tid + THREADS; s < p.n_seq; s += THREADS) v += seq_units(p, s, rows);
#pragma unroll
    for (int m = 16; m; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    if (lane == 0) warp_sum[warp] = v;
    if (tid == 0) found_seq = p.n_seq, found_at = 0;
    __syncthreads();
    Place r;
    r.units = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) r.units += warp_sum[w];
    r.share = part_share(r.units, ctas);
    const int64_t u = cta * r.share;
    if (u < r.units) {
        int64_t base = 0;
        for (int s0 = 0; s0 < p.n_seq; s0 += THREADS) {
            const int s = s0 + tid;
            const int64_t mine = s0 == 0 ? first : (s < p.n_seq ? seq_units(p, s, rows) : 0);
            int64_t incl = mine;
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const int64_t o = __shfl_up_sync(0xffffffffu, incl, m);
                if (lane >= m) incl += o;
            }
            __syncthreads();
            if (lane == 31) warp_sum[warp] = incl;
            __syncthreads();
            int64_t before = base;
            for (int w = 0; w < THREADS / 32; ++w) {
                if (w < warp) before += warp_sum[w];
                base += warp_sum[w];
            }
            if (u >= before + incl - mine && u < before + incl) {
                found_seq = s;
                found_at = u - (before + incl - mine);
            }
            if (u < base) break;  // the same for every thread
        }
    }
    __syncthreads();
    r.seq = found_seq;
    r.at = found_at;
    return r;
}

// Walks the segments of a part.
struct Walk {
    Seq q;
    int seq, head, rt;
    int tile, tiles;  // first unit in the segment (kStart is its first tile), the segment's units
    int rts;
    int64_t left;     // units of the part from here on

    __device__ __forceinline__ void start(const KvAttendParams &p, const Place &pl, int rows, int64_t units) {
        left = units;
        seq = pl.seq;
        if (left <= 0) return;
        q = load_seq(p, seq);
        tiles = tok_tiles(q);
        rts = row_tiles(p, q, rows);
        tile = static_cast<int>(pl.at % tiles);
        const int hr = static_cast<int>(pl.at / tiles);
        head = hr / rts;
        rt = hr - head * rts;
    }
    // Units of the part in this segment; of them tiles; the first such tile.
    __device__ __forceinline__ int count() const {
        return left < tiles - tile ? static_cast<int>(left) : tiles - tile;
    }
    __device__ __forceinline__ int first_tile() const { return tile > kStart ? tile - kStart : 0; }
    __device__ __forceinline__ int n_tiles() const {
        const int n = tile + count() - kStart - first_tile();
        return n > 0 ? n : 0;
    }
    __device__ __forceinline__ void next(const KvAttendParams &p, int rows) {
        left -= count();
        tile = 0;
        if (left <= 0) return;
        if (++rt < rts) return;
        rt = 0;
        if (++head < p.c.n_heads) return;
        head = 0;
        do {
            ++seq;
            q = load_seq(p, seq);
        } while (q.m == 0);  // units are left, so there is one
        tiles = tok_tiles(q);
        rts = row_tiles(p, q, rows);
    }
};

// Bounded wait (about 1 s) that suspends the thread between polls and gives up
// once another thread of the block has set the abort flag.
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, const volatile int *abort_flag) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    for (uint32_t i = 1; i < kWaitLimitPolls; ++i) {
        if (mbar_try_wait_hint(bar, parity, 20000u)) return true;
        if ((i & 15u) == 0 && (*abort_flag || global_timer_ns() - t0 > kWaitLimitNs)) return false;
    }
    return false;
}

// d = a b + c
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1, const uint4 &c) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(__uint_as_float(c.x)), "f"(__uint_as_float(c.y)),
          "f"(__uint_as_float(c.z)), "f"(__uint_as_float(c.w)));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// code - 8 in f16 of the low (high) nibbles of bytes 0 and 2; magic = 0x64006400.
__device__ __forceinline__ uint32_t low_codes(uint32_t w, uint32_t magic) {
    return hsub2((w & 0x000F000Fu) | magic, 0x64086408u);  // 1024 + c - 1032
}
__device__ __forceinline__ uint32_t high_codes(uint32_t w, uint32_t magic) {
    return hfma2((w & 0x00F000F0u) | magic, 0x2C002C00u, 0xD480D480u);  // (1024 + 16 c) / 16 - 72
}
// Loads from the tile (plain ones, which the compiler may move among the
// products but not over the waits).
template <int NB> __device__ __forceinline__ void ld_words(const uint8_t *p, uint32_t (&w)[NB]) {
    if (NB == 4) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        w[0] = v.x, w[1] = v.y, w[NB - 2] = v.z, w[NB - 1] = v.w;
    } else {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        w[0] = v.x, w[1] = v.y;
    }
}
// NB f16 (one row's scales, or one value unit of every block) as NB/2 words.
template <int NB> __device__ __forceinline__ void ld_halves(const uint8_t *p, uint32_t (&w)[NB / 2]) {
    if (NB == 4) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        w[0] = v.x, w[NB / 2 - 1] = v.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t *>(p);
    }
}
__device__ __forceinline__ bool not_finite(uint32_t half_bits) { return (half_bits & 0x7C00u) == 0x7C00u; }

// The largest magnitudes among a row's scales (halves apart; NaN has no say).
template <int NB> __device__ __forceinline__ uint32_t max_scales(const uint32_t (&w)[NB / 2]) {
    __half2 m = __habs2(*reinterpret_cast<const __half2 *>(&w[0]));
    if (NB == 4) m = __hmax2(m, __habs2(*reinterpret_cast<const __half2 *>(&w[NB / 2 - 1])));
    return *reinterpret_cast<const uint32_t *>(&m);
}
// The f16 exponent fields of the largest of each of two tokens, from their max_scales: 0 .. 31, the second token's in
// the high half.
__device__ __forceinline__ uint32_t exponent_fields(uint32_t a, uint32_t b) {
    const uint32_t x = __byte_perm(a, b, 0x5410), y = __byte_perm(a, b, 0x7632);
    const __half2 m = __hmax2(*reinterpret_cast<const __half2 *>(&x), *reinterpret_cast<const __half2 *>(&y));
    return (*reinterpret_cast<const uint32_t *>(&m) >> 10) & 0x001F001Fu;
}
// Infinite scales as NaN: times a code less 8 they would be an infinity or NaN by the code.
template <int NB> __device__ __forceinline__ void infinities_to_nan(uint32_t (&w)[NB / 2]) {
#pragma unroll
    for (int i = 0; i < NB / 2; ++i) {
        if (not_finite(w[i])) w[i] |= 0x0200u;
        if (not_finite(w[i] >> 16)) w[i] |= 0x02000000u;
    }
}

// Eight query elements of a row (elements 0..3 and 16..19 from shared address a on) in f32.
template <class T> __device__ __forceinline__ void load_q8(uint32_t a, float (&x)[8]);
template <> __device__ __forceinline__ void load_q8<float>(uint32_t a, float (&x)[8]) {
    const uint4 u = ld_s128(a), v = ld_s128(a + 64);
    x[0] = __uint_as_float(u.x), x[1] = __uint_as_float(u.y), x[2] = __uint_as_float(u.z), x[3] = __uint_as_float(u.w);
    x[4] = __uint_as_float(v.x), x[5] = __uint_as_float(v.y), x[6] = __uint_as_float(v.z), x[7] = __uint_as_float(v.w);
}
template <> __device__ __forceinline__ void load_q8<__half>(uint32_t a, float (&x)[8]) {
    const uint2 u = ld_s64(a), v = ld_s64(a + 32);
    const uint32_t w[4] = {u.x, u.y, v.x, v.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = unpack_half2(w[i]).x, x[2 * i + 1] = unpack_half2(w[i]).y;
}

__device__ __forceinline__ void store2(float *p, float a, float b) { *reinterpret_cast<float2 *>(p) = make_float2(a, b); }
__device__ __forceinline__ void store2(__half *p, float a, float b) { *reinterpret_cast<__half2 *>(p) = __floats2half2_rn(a, b); }

// Whether a row that sees the tokens up to `limit` sees, among those from
// `least` on within the part's tokens first .. past - 1, one whose value scale
// of block b is not finite. Such a token is left out of the products where
// some rows do not see it (0 times its scale would be NaN); the rows that do
// get NaN in the block's channels here.
template <int D> __device__ __noinline__ bool odd_tokens(const KvAttendParams &p, const Walk &seg, int least, int limit, int first, int past, int b) {
    using G = KvGroup<D>;
    if (past > limit) past = limit;
    for (int tok = max(first, least); tok < past; ++tok) {
        const int page = p.table[seg.seq * p.table_stride + tok / p.c.page_size], r = tok % p.c.page_size;
        if (page < 0 || page >= p.c.n_pages) continue;
        const uint8_t *g = p.c.data + ((static_cast<int64_t>(page) * p.c.n_heads + seg.head) * p.c.page_groups + (r >> 4)) * G::kBytes;
        if (not_finite(reinterpret_cast<const unsigned short *>(g + G::kVS + (r & 15) * G::kScaleRow)[b])) return true;
    }
    return false;
}

template <int D, class T, int NT>
__global__ void __launch_bounds__(kThreads, Shape<D, NT, (sizeof(T) == 4 ? 2 : 1)>::kCtas)
    kv_attend_kernel(const KvAttendParams p) {
    using G = KvGroup<D>;
    constexpr int NB = G::kNB, TERMS = sizeof(T) == 4 ? 2 : 1, ROWS = 8 * NT;
    using Sh = Shape<D, NT, TERMS>;
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t base = smem_addr(smem);
    const uint32_t full0 = base, empty0 = base + 8 * Sh::kSlots;
    volatile int *slot_info = reinterpret_cast<volatile int *>(smem + 16 * Sh::kSlots);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + 20 * Sh::kSlots);
    const uint32_t qfull = base + 20 * Sh::kSlots + 16, qempty = qfull + 8;
    __shared__ Walk walks[kWarps];
    // one for each of two segments in turn: see the join
    volatile int *const odd_flags = reinterpret_cast<volatile int *>(smem + 20 * Sh::kSlots + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < Sh::kSlots; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        mbar_init(qfull, 1);
        mbar_init(qempty, kWarps);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    // With p.rest the kernel before does not write what this one reads: it has waited for what came before, and this
    // one's blocks may run beside it; they wait for its end before their own, so that what comes next finds both done.
    if (p.rest == nullptr) pdl_wait_prior_grids();
    pdl_allow_dependents();
    __syncthreads();
    const Place place = p.n_seq <= 32 ? locate_few(p, ROWS, blockIdx.x, gridDim.x) : locate<kThreads>(p, ROWS, blockIdx.x, gridDim.x);
    const int64_t u0 = static_cast<int64_t>(blockIdx.x) * place.share;
    int64_t units = place.units - u0;
    if (units > place.share) units = place.share;
    Cut *const cut = reinterpret_cast<Cut *>(p.partial) + blockIdx.x;
    float *const parts = p.partial + kCutFloats;
    if (threadIdx.x == 0) cut->parts = 0;
    if (units <= 0) {
        if (p.rest != nullptr) pdl_wait_prior_grids();
        return;
    }
    Walk walk;
    walk.start(p, place, ROWS, units);

    if (warp == kWarps) {
        // ---------------- producer
        int slot = 0, seg = 0;
        uint32_t phase = 0;
        int64_t issued = 0;
        bool ok = true;
        for (; walk.left > 0 && ok; ++seg) {
            const int n = walk.n_tiles(), tile0 = walk.first_tile();
            const int groups = (walk.q.len + 15) >> 4;  // of the sequence
            const int32_t *table = p.table + walk.seq * p.table_stride;
            // the segment's query rows: of each token they cover, the heads are contiguous
            {
                const uint32_t raw = base + Sh::kOffRaw, bar = qfull;
                if (seg >= 1) ok = __all_sync(0xffffffffu, wait_bounded(qempty, (seg - 1) & 1, abort_flag));
                if (!ok) break;
                const int row0 = walk.rt * ROWS;
                int row1 = walk.q.m * p.group;
                if (row1 > row0 + ROWS) row1 = row0 + ROWS;
                if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>((row1 - row0) * Sh::kRawRow));
                __syncwarp();
                const int tok = row0 / p.group + lane;
                const int a = max(row0, tok * p.group), z = min(row1, (tok + 1) * p.group);
                if (a < z)
                    bulk_copy_g2s_plain(raw + (a - row0) * Sh::kRawRow,
                                        static_cast<const T *>(p.q) + (walk.q.q0 + tok) * p.q_stride +
                                            (static_cast<int64_t>(walk.head) * p.group + a - tok * p.group) * D,
                                        static_cast<uint32_t>((z - a) * Sh::kRawRow), bar);
            }
            int have = 0;      // first group whose address the lanes hold
            int64_t src = -1;  // byte offset of group have + lane, -1: none
            // up to four tiles at a time, two lanes each (one for each group)
            for (int i = 0; i < n; i += 4) {
                const int g0 = 2 * (tile0 + i), batch = min(4, n - i);
                if (i == 0 || g0 >= have + 32) {
                    have = g0;
                    const int g = have + lane;
                    src = -1;
                    if (g < groups && g < 2 * (tile0 + n)) {
                        const int page = __ldg(table + g / p.c.page_groups);
                        if (page >= 0 && page < p.c.n_pages)
                            src = ((static_cast<int64_t>(page) * p.c.n_heads + walk.head) * p.c.page_groups +
                                   g % p.c.page_groups) * G::kBytes;
                        else
                            record_error(p.err, kErrBadIndex);
                    }
                }
                const int64_t mine = __shfl_sync(0xffffffffu, src, (g0 - have + (lane & 7)) & 31);
                const uint32_t valid = (__ballot_sync(0xffffffffu, mine >= 0) >> (lane & 6)) & 3u;  // of the lane's tile
                int my_slot = slot + (lane >> 1);
                uint32_t my_phase = phase;
                if (my_slot >= Sh::kSlots) my_slot -= Sh::kSlots, my_phase ^= 1u;
                const bool active = lane < 2 * batch;
                if (active && issued + (lane >> 1) >= Sh::kSlots) ok = wait_bounded(empty0 + 8 * my_slot, my_phase ^ 1u, abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (active && (lane & 1) == 0) {
                    slot_info[my_slot] = static_cast<int>(valid);
                    mbar_arrive_expect_tx(full0 + 8 * my_slot, static_cast<uint32_t>(__popc(valid)) * G::kBytes);
                }
                __syncwarp();
                if (active && mine >= 0)
                    bulk_copy_g2s_plain(base + Sh::kOffRing + my_slot * Sh::kTileBytes + (lane & 1) * G::kBytes,
                                        p.c.data + mine, G::kBytes, full0 + 8 * my_slot);
                issued += batch;
                slot += batch;
                if (slot >= Sh::kSlots) slot -= Sh::kSlots, phase ^= 1u;
            }
            if (ok) walk.next(p, ROWS);
        }
        if (!ok) {
            if (lane == 0) record_error(p.err, kErrProducerWait);
            *abort_flag = 1;
        }
        // Leave no copy in flight into this block's shared memory: consumers that gave up waiting for one may be gone
        // before it lands, even if nothing held the producer up.
        for (int64_t k = issued > Sh::kSlots ? issued - Sh::kSlots : 0; k < issued; ++k)
            if (!mbar_wait_bounded(full0 + 8 * static_cast<int>(k % Sh::kSlots),
                                   static_cast<uint32_t>((k / Sh::kSlots) & 1)))
                record_error(p.err, kErrDrainWait);
        if (seg > 0 && !mbar_wait_bounded(qfull, (seg - 1) & 1)) record_error(p.err, kErrDrainWait);
        if (p.rest != nullptr) pdl_wait_prior_grids();
        return;
    }

    // ---------------- consumers
    const int g = lane >> 2, t = lane & 3;
    // 0x64006400, by way of a value the compiler does not know: (word & mask) | magic is then one
    // logic operation (it takes one immediate) and not two
    const uint32_t magic = 0x64006400u | (static_cast<uint32_t>(p.n_tok) >> 31);
    float *row_factor = reinterpret_cast<float *>(smem + Sh::kOffRow);
    int *row_limit = reinterpret_cast<int *>(smem + Sh::kOffRow) + ROWS;
    int *row_out = row_limit + ROWS;  // the row's place in out, in heads; -1: none
    float *stat = reinterpret_cast<float *>(smem + Sh::kOffStat);
    float *join = reinterpret_cast<float *>(smem + Sh::kOffJoin);
    // The walk lies in shared memory, a copy a warp: in registers it cost the loop over the tiles a dozen, which
    // were spilled there.
    Walk &seg = walks[warp];
    if (lane == 0) seg = walk;
    __syncwarp();
    int k = warp;      // this warp's next tile, counted from the segment's first one in the part
    int slot = warp;
    uint32_t phase = 0, phase_q = 0;
    bool ok = true;
    while (seg.left > 0) {
        const int n = seg.n_tiles(), tile0 = seg.first_tile();
        volatile int *const odd_flag = odd_flags + phase_q;
        // ---- the segment's queries, as the mma's B fragments
        if (ok && !__all_sync(0xffffffffu, wait_bounded(qfull, phase_q, abort_flag))) {
            if (lane == 0) record_error(p.err, kErrConsumerWait);
            *abort_flag = 1;
            ok = false;
        }
        {
            const uint32_t raw = base + Sh::kOffRaw;
            const int rows = seg.q.m * p.group, row0 = seg.rt * ROWS, before = seg.q.len - seg.q.m + 1;
            constexpr int kItems = ROWS * NB * 4;
            for (int it = threadIdx.x; it < kItems; it += kWarps * 32) {
                const int r = it / (NB * 4), b = it / 4 % NB, ti = it & 3;
                const int row = row0 + r;
                const bool live = row < rows;
                float x[8] = {};
                if (live) load_q8<T>(raw + r * Sh::kRawRow + (32 * b + 4 * ti) * static_cast<int>(sizeof(T)), x);
                float big = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) big = fmaxf(big, fabsf(x[i]));
#pragma unroll
                for (int m = 1; m < NB * 4; m <<= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, m));
                int e = static_cast<int>(__float_as_uint(big) >> 23) - 127;  // exponent of the largest
                if (e == 128) e = 0;                                          // infinities
                if (e < -117) e = -117;                                       // (2^(10 - e) is an f32)
                const float up = __uint_as_float(static_cast<uint32_t>(10 - e + 127) << 23) * (p.scale < 0.0f ? -1.0f : 1.0f);
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x[i] *= up;
                    if (TERMS == 1) sum += x[i];  // exact in f16
                }
                uint32_t w[TERMS][4];
                // elements of the fragment's words: 0 2 | 1 3 (low nibbles) | 16 18 | 17 19 (high)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int e0 = (i & 2) * 2 + (i & 1);
                    const float f = i < 2 && TERMS == 1 ? 16.0f : 1.0f;  // (subnormal codes: the high nibbles are 16 c)
                    w[0][i] = pack_half2(x[e0] * f, x[e0 + 2] * f);
                    if (TERMS == 2) {
                        const float2 hi = unpack_half2(w[0][i]);
                        w[TERMS - 1][i] = pack_half2(x[e0] * f - hi.x, x[e0 + 2] * f - hi.y);
                    }
                }
                if (TERMS == 1) {
                    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                }
                const int nt = r >> 3, rr = r & 7;
#pragma unroll
                for (int q = 0; q < TERMS; ++q)
                    *reinterpret_cast<uint4 *>(smem + Sh::kOffQ + ((q * NT + nt) * NB + b) * 512 + (rr * 4 + ti) * 16) =
                        make_uint4(w[q][0], w[q][1], w[q][2], w[q][3]);
                if (ti == 0) {
                    float *ini = reinterpret_cast<float *>(smem + Sh::kOffInit) + (nt * NB + b) * 16 + (rr >> 1) * 4 + (rr & 1);
                    ini[0] = ini[2] = sum * -0x1p-17f;  // -8 * 16 * 2^-24, 0 for code - 8
                    if (b == 0) {
                        // 2^(e - 10), for subnormal codes times 2^24 / 16; never 0, which times an unseen
                        // token's -inf would be NaN, nor infinite
                        row_factor[r] = fminf(fmaxf(fabsf(p.scale) * 1.4426950408889634f *
                                                        __uint_as_float(static_cast<uint32_t>(e + 127) << 23) *
                                                        (TERMS == 1 ? 0x1p10f : 0x1p-10f),
                                                    1e-37f),
                                              FLT_MAX);
                        const int tok = row / p.group;
                        row_limit[r] = live ? before + tok : 0;
                        row_out[r] = live ? (seg.q.q0 + tok) * p.n_heads + seg.head * p.group + row - tok * p.group : -1;
                    }
                }
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(qempty);
        if (threadIdx.x == 0) *odd_flag = 0;
        named_barrier(1, kWarps * 32);
        float factor[NT][2];
        // the first row sees least (rows past the last have no say: their result is not stored)
        const int least = row_limit[0];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                factor[nt][c] = row_factor[8 * nt + 2 * t + c];
            }
        float m[NT][2], l[NT][2], o[NT][NB][2][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = -INFINITY;
            l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[nt][b][h][i] = 0.0f;
        }

        for (; k < n; k += kWarps) {
            if (!ok) continue;
            ok = __all_sync(0xffffffffu, wait_bounded(full0 + 8 * slot, phase, abort_flag));
            if (!ok) {
                if (lane == 0) record_error(p.err, kErrConsumerWait);
                *abort_flag = 1;
                continue;
            }
            {
                const uint8_t *const tile_p = smem + Sh::kOffRing + slot * Sh::kTileBytes;
                const int tok0 = (tile0 + k) * kTile;
                const int info = slot_info[slot];
                // ---- scores of 2 x 16 tokens: s[group][nt][0, 1: token g; 2, 3: token g + 8]
                float s[2][NT][4];
                uint32_t dv[2][2][NB / 2];  // value scales of tokens g and g + 8
                {
                    uint32_t w[2][2][NB], dk[2][2][NB / 2];
#pragma unroll
                    for (int gr = 0; gr < 2; ++gr)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint8_t *const ga = tile_p + gr * G::kBytes;
                            ld_words<NB>(ga + (g + 8 * h) * G::kRow + t * (4 * NB), w[gr][h]);
                            ld_halves<NB>(ga + G::kKS + (g + 8 * h) * G::kScaleRow, dk[gr][h]);
                            ld_halves<NB>(ga + G::kVS + (g + 8 * h) * G::kScaleRow, dv[gr][h]);
                        }
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        uint32_t lo[2][4], hi[2][4];
                        float ks[2][2];
#pragma unroll
                        for (int gr = 0; gr < 2; ++gr)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const uint32_t x = w[gr][h][b], y = x >> 8;
                                if (TERMS == 1) {
                                    lo[gr][h] = x & 0x000F000Fu, lo[gr][2 + h] = y & 0x000F000Fu;
                                    hi[gr][h] = x & 0x00F000F0u, hi[gr][2 + h] = y & 0x00F000F0u;
                                } else {
                                    lo[gr][h] = low_codes(x, magic), lo[gr][2 + h] = low_codes(y, magic);
                                    hi[gr][h] = high_codes(x, magic), hi[gr][2 + h] = high_codes(y, magic);
                                }
                                const float2 k2 = unpack_half2(dk[gr][h][b / 2]);
                                ks[gr][h] = b & 1 ? k2.y : k2.x;
                            }
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const uint4 ini = TERMS == 1 ? *reinterpret_cast<const uint4 *>(smem + Sh::kOffInit + (nt * NB + b) * 64 + t * 16)
                                                         : make_uint4(0u, 0u, 0u, 0u);
                            float acc[2][4];
#pragma unroll
                            for (int q = 0; q < TERMS; ++q) {
                                const uint4 bq = *reinterpret_cast<const uint4 *>(smem + Sh::kOffQ + ((q * NT + nt) * NB + b) * 512 + lane * 16);
#pragma unroll
                                for (int gr = 0; gr < 2; ++gr) {
                                    if (q == 0)
                                        mma_f16(acc[gr], lo[gr][0], lo[gr][1], lo[gr][2], lo[gr][3], bq.x, bq.y, ini);
                                    else
                                        mma_f16(acc[gr], lo[gr][0], lo[gr][1], lo[gr][2], lo[gr][3], bq.x, bq.y);
                                    mma_f16(acc[gr], hi[gr][0], hi[gr][1], hi[gr][2], hi[gr][3], bq.z, bq.w);
                                }
                            }
#pragma unroll
                            for (int gr = 0; gr < 2; ++gr)
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    s[gr][nt][i] = b == 0 ? ks[gr][i >> 1] * acc[gr][i]
                                                          : fmaf(ks[gr][i >> 1], acc[gr][i], s[gr][nt][i]);
                        }
                    }
                }
                const bool masked = tok0 + kTile > least || info != 3;
                if (masked) {
                    // tokens that a row does not see, or that lie in no page: whatever
                    // the ring holds there (it may be NaN) is replaced
                    const int len = seg.q.len;
                    bool odd = false;
#pragma unroll
                    for (int gr = 0; gr < 2; ++gr)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int tok = tok0 + 16 * gr + 8 * h + g;
                            const bool in_page = (info >> gr) & 1;
#pragma unroll
                            for (int i = 0; i < NB / 2; ++i) {
                                if (!in_page || tok >= len) dv[gr][h][i] = 0;
                                // a scale that is not finite, of a token that only some rows see: see `odd_tokens`
                                if (tok >= least && not_finite(dv[gr][h][i])) odd = true, dv[gr][h][i] &= 0xFFFF0000u;
                                if (tok >= least && not_finite(dv[gr][h][i] >> 16)) odd = true, dv[gr][h][i] &= 0x0000FFFFu;
                            }
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int c = 0; c < 2; ++c)
                                    if (!in_page || tok >= row_limit[8 * nt + 2 * t + c]) s[gr][nt][2 * h + c] = -INFINITY;
                        }
                    if (odd) *odd_flag = 1;
                }
                // ---- the lane's largest score plus exponent, by column: of each token by itself, since the largest score
                // and the largest scale of different tokens could lie far above every product
                float top[NT][2];
                {
                    float ex[2][2];
                    uint32_t infinite = 0;
#pragma unroll
                    for (int gr = 0; gr < 2; ++gr) {
                        const uint32_t f = exponent_fields(max_scales<NB>(dv[gr][0]), max_scales<NB>(dv[gr][1]));
                        ex[gr][0] = __uint_as_float(__byte_perm(f, 0x4B000000u, 0x7540)) - 8388608.0f;
                        ex[gr][1] = __uint_as_float(__byte_perm(f, 0x4B000000u, 0x7542)) - 8388608.0f;
                        infinite |= f + 0x00010001u;
                    }
                    if (TERMS == 1 && (infinite & 0x00200020u))  // (two terms make NaN of it: infinity less infinity)
#pragma unroll
                        for (int i = 0; i < 4; ++i) infinities_to_nan<NB>(dv[i >> 1][i & 1]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const float f = factor[nt][c];
                            top[nt][c] = fmaxf(fmaxf(fmaf(s[0][nt][c], f, ex[0][0]), fmaf(s[0][nt][2 + c], f, ex[0][1])),
                                               fmaxf(fmaf(s[1][nt][c], f, ex[1][0]), fmaf(s[1][nt][2 + c], f, ex[1][1])));
                        }
                }
                // ---- running reference (raised when a product could pass 2^15), weights
                bool grow = false;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) grow = grow || top[nt][0] - kHigh > m[nt][0] || top[nt][1] - kHigh > m[nt][1];
                if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            float mx = top[nt][c];
#pragma unroll
                            for (int q = 4; q < 32; q <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, q));
                            mx = fmaxf(m[nt][c], mx - kLow);
                            const float keep = exp2_approx(m[nt][c] - (mx == -INFINITY ? 0.0f : mx));
                            m[nt][c] = mx;
                            l[nt][c] *= keep;
#pragma unroll
                            for (int b = 0; b < NB; ++b)
#pragma unroll
                                for (int h = 0; h < 2; ++h) o[nt][b][h][c] *= keep, o[nt][b][h][2 + c] *= keep;
                        }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const float ref = m[nt][c] == -INFINITY ? 0.0f : m[nt][c];
#pragma unroll
                        for (int gr = 0; gr < 2; ++gr)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const float w = exp2_approx(fmaf(s[gr][nt][2 * h + c], factor[nt][c], -ref));
                                s[gr][nt][2 * h + c] = w;
                                l[nt][c] += w;
                            }
                    }
                // ---- values
#pragma unroll
                for (int gr = 0; gr < 2; ++gr) {
                    const uint8_t *const va = tile_p + gr * G::kBytes + G::kV;
                    uint32_t v[4][NB / 2];  // unit g of every block, tokens 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        ld_halves<NB>(va + (4 * i + t) * G::kRow + (g ^ ((t & 2) << 1)) * (2 * NB), v[i]);
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        const uint32_t sel = b & 1 ? 0x7632u : 0x5410u;
                        const uint32_t wa = __byte_perm(v[0][b / 2], v[1][b / 2], sel);
                        const uint32_t wb = __byte_perm(v[2][b / 2], v[3][b / 2], sel);
                        const uint32_t a0 = low_codes(wa, magic), a1 = low_codes(wa >> 8, magic);
                        const uint32_t a2 = low_codes(wb, magic), a3 = low_codes(wb >> 8, magic);
                        const uint32_t h0 = high_codes(wa, magic), h1 = high_codes(wa >> 8, magic);
                        const uint32_t h2 = high_codes(wb, magic), h3 = high_codes(wb >> 8, magic);
                        const float2 f0 = unpack_half2(dv[gr][0][b / 2]), f1 = unpack_half2(dv[gr][1][b / 2]);
                        const float fa = b & 1 ? f0.y : f0.x, fb = b & 1 ? f1.y : f1.x;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const float2 pa = make_float2(s[gr][nt][0] * fa, s[gr][nt][1] * fa);
                            const float2 pb = make_float2(s[gr][nt][2] * fb, s[gr][nt][3] * fb);
                            const uint32_t x = pack_half2(pa.x, pa.y), y = pack_half2(pb.x, pb.y);
                            if (TERMS == 1) {
                                const uint32_t b0 = transpose8(x), b1 = transpose8(y);
                                mma_f16(o[nt][b][0], a0, a1, a2, a3, b0, b1);
                                mma_f16(o[nt][b][1], h0, h1, h2, h3, b0, b1);
                            } else {
                                // sums of 16 tokens, added to the long ones by themselves: the tensor cores cut what
                                // they add off where an ordinary sum rounds, always toward zero, and over 131071
                                // tokens that came to 1.4e-6 of the result
                                const float2 xh = unpack_half2(x), yh = unpack_half2(y);
                                const float2 ra = fadd2(pa, make_float2(-xh.x, -xh.y)), rb = fadd2(pb, make_float2(-yh.x, -yh.y));
                                const uint32_t b0 = transpose8(x), b1 = transpose8(y);
                                const uint32_t b2 = transpose8(pack_half2(ra.x, ra.y)), b3 = transpose8(pack_half2(rb.x, rb.y));
                                const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
                                float lo[4], hi[4];
                                mma_f16(lo, a0, a1, a2, a3, b0, b1, zero);
                                mma_f16(hi, h0, h1, h2, h3, b0, b1, zero);
                                mma_f16(lo, a0, a1, a2, a3, b2, b3);
                                mma_f16(hi, h0, h1, h2, h3, b2, b3);
#pragma unroll
                                for (int i = 0; i < 4; i += 2) {
                                    const float2 u = fadd2(make_float2(o[nt][b][0][i], o[nt][b][0][i + 1]), make_float2(lo[i], lo[i + 1]));
                                    const float2 w2 = fadd2(make_float2(o[nt][b][1][i], o[nt][b][1][i + 1]), make_float2(hi[i], hi[i + 1]));
                                    o[nt][b][0][i] = u.x, o[nt][b][0][i + 1] = u.y;
                                    o[nt][b][1][i] = w2.x, o[nt][b][1][i + 1] = w2.y;
                                }
                            }
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty0 + 8 * slot);
            slot += kWarps;
            if (slot >= Sh::kSlots) slot -= Sh::kSlots, phase ^= 1u;
        }
        // ---- the warps' results become one
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int r = 8 * nt + 2 * t + c;
#pragma unroll
                for (int q = 4; q < 32; q <<= 1) l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], q);
                if (g == 0) *reinterpret_cast<float2 *>(stat + (r * kWarps + warp) * 2) = make_float2(m[nt][c], l[nt][c]);
                float *dst = join + (warp * ROWS + r) * Sh::kJoinPitch + 2 * g;
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        *reinterpret_cast<float2 *>(dst + 32 * b + 16 * h) = make_float2(o[nt][b][h][c], o[nt][b][h][2 + c]);
            }
        const int units = seg.count();
        const bool from = seg.tile == 0, whole = from && units == seg.tiles;
        // A row's channels by 16 / NT threads, four at a time. What the rows' preparation wrote is read before the
        // barrier: a warp that is through with the join prepares the next segment's rows while others still join,
        // and the warp that prepares a row need not be the one that joins it.
        constexpr int kPer = 16 / NT;
        const int r = threadIdx.x / kPer, out_row = row_out[r], limit = row_limit[r];
        named_barrier(1, kWarps * 32);
        {
            if (out_row >= 0) {
                float2 ml[kWarps];
                float top = -INFINITY, den = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; w += 2) {
                    const float4 v = *reinterpret_cast<const float4 *>(stat + (r * kWarps + w) * 2);
                    ml[w] = make_float2(v.x, v.y), ml[w + 1] = make_float2(v.z, v.w);
                }
#pragma unroll
                for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml[w].x);
                const float ref = top == -INFINITY ? 0.0f : top;
                float f[kWarps];
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    f[w] = exp2_approx(ml[w].x - ref);
                    den = fmaf(ml[w].y, f[w], den);
                }
                // a part's result: slot 0 if it enters the segment from outside, slot 1 if the segment starts in it
                float *part = parts + (2 * static_cast<int64_t>(blockIdx.x) + (from ? 1 : 0)) * part_floats(D, ROWS);
                float *part_stats = part + ROWS * D + 2 * r;
                part += r * D;
                const bool to_out = whole && p.rest == nullptr;
                if (whole && !to_out) part = p.rest + static_cast<int64_t>(out_row) * D, part_stats = p.rest_stats + 2 * static_cast<int64_t>(out_row);
                const float inv = !whole ? 1.0f : den == 0.0f ? 0.0f : 1.0f / den;  // no token seen: zeros
                T *out = static_cast<T *>(p.out) + static_cast<int64_t>(out_row) * D;
                const bool odd = *odd_flag != 0;
#pragma unroll
                for (int d0 = 0; d0 < D; d0 += 4 * kPer) {
                    const int d = d0 + 4 * (threadIdx.x % kPer);
                    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) {
                        const float4 v = *reinterpret_cast<const float4 *>(join + (w * ROWS + r) * Sh::kJoinPitch + d);
                        sum.x = fmaf(v.x, f[w], sum.x), sum.y = fmaf(v.y, f[w], sum.y);
                        sum.z = fmaf(v.z, f[w], sum.z), sum.w = fmaf(v.w, f[w], sum.w);
                    }
                    if (odd && odd_tokens<D>(p, seg, least, limit, tile0 * kTile, (tile0 + n) * kTile, d >> 5))
                        sum.x = sum.y = sum.z = sum.w = NAN;
                    if (!to_out) {
                        *reinterpret_cast<float4 *>(part + d) = sum;
                    } else {
                        store2(out + d, sum.x * inv, sum.y * inv);
                        store2(out + d + 2, sum.z * inv, sum.w * inv);
                    }
                }
                if (!to_out && threadIdx.x % kPer == 0) store2(part_stats, top, den);
            }
            if (!whole && from) {
                const int row0 = seg.rt * ROWS, n_parts = 1 + static_cast<int>((seg.tiles - units + place.share - 1) / place.share);
                if (threadIdx.x == 0)  // (thread 0 wrote the 0 above)
                    *cut = Cut{n_parts, min(ROWS, seg.q.m * p.group - row0), row0, seg.q.q0, seg.head, {0, 0, 0}};
                if (p.rest != nullptr && out_row >= 0 && threadIdx.x % kPer == 0)
                    store2(p.rest_stats + 2 * static_cast<int64_t>(out_row), __int_as_float(static_cast<int>(blockIdx.x)), -static_cast<float>(n_parts));
            }
        }
        // The join's areas are written again after the next segment's first barrier, which comes after these reads; its
        // flag is cleared for the next segment but one, after the next one's last barrier.
        phase_q ^= 1u;
        k -= n;
        __syncwarp();
        if (lane == 0) seg.next(p, ROWS);
        __syncwarp();
    }
}

// Joins the parts of the segments that thread blocks of kv_attend_kernel cut:
// block (c, y) rows y, y + gridDim.y, ... of the segment that starts in block c
// and goes on in the next ones, part 0 the second slot of block c, the others the
// first slots of c + 1, c + 2, ... The warps take a row's parts in turn, each lane
// D/32 channels; their sums meet in shared memory in a fixed order. Most blocks
// find nothing to do, so their number counts: 16 sequences, 15 rows: 17.6 us in all
// with 8 blocks of 4 warps a cut, 18.8 with one a row, 19.6 with one of 8 warps a
// row, 22.4 with 2 blocks; 131071 tokens, 8 rows: 50.2, 50.1, 50.2 and 57.0.
constexpr int kJoinWarps = 4, kJoinRows = 8;

template <int D, class T, int NT>
__global__ void __launch_bounds__(32 * kJoinWarps) kv_join_kernel(const KvAttendParams p) {
    constexpr int ROWS = 8 * NT, kPer = D / 32;
    __shared__ float sums[kJoinWarps][D];
    __shared__ float2 stats[kJoinWarps];
    pdl_allow_dependents();
    pdl_wait_prior_grids();  // in every block: what comes next on the stream then waits for the kernel before, too
    const Cut cut = reinterpret_cast<const Cut *>(p.partial)[blockIdx.x];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (cut.parts == 0) return;
    const int64_t pitch = 2 * part_floats(D, ROWS);
    const float *first = p.partial + kCutFloats + blockIdx.x * pitch;  // the parts: first + part_floats, first + i pitch
    for (int r = blockIdx.y; r < cut.rows; r += gridDim.y) {
        const int64_t at = static_cast<int64_t>(r) * D + lane * kPer, st = static_cast<int64_t>(ROWS) * D + 2 * r;
        float top = -INFINITY, den = 0.0f, acc[kPer] = {};
        for (int i0 = warp; i0 < cut.parts; i0 += 4 * kJoinWarps) {
            float2 ml[4];
            float v[4][kPer];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = i0 + j * kJoinWarps;
                ml[j] = make_float2(-INFINITY, 0.0f);
                if (i < cut.parts) {
                    const float *q = i == 0 ? first + part_floats(D, ROWS) : first + i * pitch;
                    ml[j] = __ldcg(reinterpret_cast<const float2 *>(q + st));
#pragma unroll
                    for (int k = 0; k < kPer; k += 2) {
                        const float2 x = __ldcg(reinterpret_cast<const float2 *>(q + at + k));
                        v[j][k] = x.x, v[j][k + 1] = x.y;
                    }
                }
            }
            float nt = top;
#pragma unroll
            for (int j = 0; j < 4; ++j) nt = fmaxf(nt, ml[j].x);
            const float ref = nt == -INFINITY ? 0.0f : nt;  // (nothing seen: zeros; scores that are NaN: NaN)
            const float keep = exp2_approx(top - ref);
            top = nt;
            den *= keep;
#pragma unroll
            for (int k = 0; k < kPer; ++k) acc[k] *= keep;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (i0 + j * kJoinWarps >= cut.parts) break;
                const float f = exp2_approx(ml[j].x - ref);
                den = fmaf(ml[j].y, f, den);
#pragma unroll
                for (int k = 0; k < kPer; ++k) acc[k] = fmaf(v[j][k], f, acc[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < kPer; ++k) sums[warp][lane * kPer + k] = acc[k];
        if (lane == 0) stats[warp] = make_float2(top, den);
        __syncthreads();
        if (threadIdx.x < D / 2) {
            const int d = 2 * threadIdx.x;
            top = -INFINITY, den = 0.0f;
#pragma unroll
            for (int w = 0; w < kJoinWarps; ++w) top = fmaxf(top, stats[w].x);
            const float ref = top == -INFINITY ? 0.0f : top;
            float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int w = 0; w < kJoinWarps; ++w) {
                const float f = exp2_approx(stats[w].x - ref);
                den = fmaf(stats[w].y, f, den);
                sum.x = fmaf(sums[w][d], f, sum.x), sum.y = fmaf(sums[w][d + 1], f, sum.y);
            }
            const int row = cut.row0 + r, tok = row / p.group;
            const float inv = den == 0.0f ? 0.0f : 1.0f / den;
            store2(static_cast<T *>(p.out) +
                       (static_cast<int64_t>(cut.q0 + tok) * p.n_heads + cut.head * p.group + row - tok * p.group) * D + d,
                   sum.x * inv, sum.y * inv);
        }
        __syncthreads();  // sums and stats are the next row's
    }
}

// Query rows a segment takes, in sets of 8: two sets share a tile's loads and
// code conversions, unless the rows make few sets and an odd number of them, whose
// last pair would be half empty. 8 sequences of 3000 .. 6000 tokens, heads of 128,
// f32: 16 rows 34.3 us with two and 34.8 with one, 24 rows 54.2 and 45.9; one of
// 60000, 32 rows: 74.7 and 79.6. (Four sets spill: 67.2 us at 24 rows, 91.8 at 32.)
int row_sets(int64_t rows) {
    const int64_t sets = (rows + 7) / 8;
    return sets % 2 == 1 && sets < 8 ? 1 : 2;
}

cudaError_t launch_join(void (*kernel)(KvAttendParams), dim3 grid, cudaStream_t s, const KvAttendParams &p) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(32 * kJoinWarps);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int D, class T, int NT> cudaError_t launch(const KvAttendParams &p, int sms, int device, cudaStream_t s) {
    using Sh = Shape<D, NT, (sizeof(T) == 4 ? 2 : 1)>;
    static std::atomic<uint64_t> done{0};
    const uint64_t bit = 1ull << (device & 63);
    if (!(done.load(std::memory_order_acquire) & bit)) {
        const cudaError_t e = cudaFuncSetAttribute(kv_attend_kernel<D, T, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem);
        if (e != cudaSuccess) return e;
        done.fetch_or(bit, std::memory_order_acq_rel);
    }
    int ctas = sms * Sh::kCtas;
    if (ctas > kMaxCtas) ctas = kMaxCtas;
    cudaError_t e = launch_pdl(kv_attend_kernel<D, T, NT>, ctas, kThreads, Sh::kSmem, s, p);
    if (e != cudaSuccess || ctas == 1 || p.rest != nullptr) return e;
    const int64_t rows = static_cast<int64_t>(p.max_q_len) * p.group;
    return launch_join(kv_join_kernel<D, T, NT>, dim3(ctas - 1, static_cast<unsigned>(rows < kJoinRows ? rows : kJoinRows)), s, p);
}

template <int D, class T> cudaError_t launch_rows(const KvAttendParams &p, int sms, int device, cudaStream_t s) {
    switch (row_sets(static_cast<int64_t>(p.max_q_len) * p.group)) {
    case 1: return launch<D, T, 1>(p, sms, device, s);
    default: return launch<D, T, 2>(p, sms, device, s);
    }
}

}  // namespace

KvParts kv_attend_parts(int head_dim, int64_t rows) {
    const int n = 8 * row_sets(rows);
    return KvParts{kCutFloats, part_floats(head_dim, n), n};
}

size_t kv_attend_workspace(int head_dim, int rows) {
    return static_cast<size_t>(kCutFloats + 2 * kMaxCtas * part_floats(head_dim, 8 * row_sets(rows))) * sizeof(float);
}

cudaError_t launch_kv_attend(const KvAttendParams &p, int head_dim, int type, int sms, int device, cudaStream_t s) {
    if (head_dim == 64)
        return type == QG_F32 ? launch_rows<64, float>(p, sms, device, s) : launch_rows<64, __half>(p, sms, device, s);
    return type == QG_F32 ? launch_rows<128, float>(p, sms, device, s) : launch_rows<128, __half>(p, sms, device, s);
}

}  // namespace qg
