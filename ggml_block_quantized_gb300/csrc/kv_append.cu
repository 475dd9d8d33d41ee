// kv_append.cu - writing rows to the 4-bit paged cache and reading their
// values back (include/qattn.h: qkv_append, qkv_read).
//
// A row is one head of one token (q, k or v), D elements, four to a lane: D/4
// lanes hold a row, eight lanes a Q4_0 block. A warp's load is 128 elements, one
// row of D = 128 or two of D = 64. The rotation's partner channel is in another
// lane of the row (shuffled as it was loaded: two shuffles for four f16), the
// block's signed maximum takes three butterfly steps among its eight lanes, and
// the four lanes with elements 0..15 of a block take the codes of 16..31 by one
// shuffle and own one 4-byte code word each.
//
// Bound: memory for many rows, latency for few. A prompt of 8191 tokens (32 + 2 x 8
// heads of 128, f16) moves 214 MB and takes 43 us (5.0 TB/s), 13 more with its
// values read back; one token takes 2 us beside the launch. The rest is
// instructions: about 85 a row, of which the bounds, the addresses and the
// rotation's loads are shared by a warp's rows.
#include <algorithm>

#include "kv_cache.cuh"
#include "quant_codes.cuh"

namespace qg {

// Four elements of a row as they lie in memory.
template <class T> struct Four;
template <> struct Four<float> {
    float4 v;
    __device__ __forceinline__ void load(const float *p, bool there) {
        v = there ? *reinterpret_cast<const float4 *>(p) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    __device__ __forceinline__ void get(float (&x)[4]) const { x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w; }
    __device__ __forceinline__ Four from(int lane) const {
        return {make_float4(__shfl_sync(0xffffffffu, v.x, lane), __shfl_sync(0xffffffffu, v.y, lane),
                            __shfl_sync(0xffffffffu, v.z, lane), __shfl_sync(0xffffffffu, v.w, lane))};
    }
};
template <> struct Four<__half> {
    uint2 v;
    __device__ __forceinline__ void load(const __half *p, bool there) {
        v = there ? *reinterpret_cast<const uint2 *>(p) : make_uint2(0u, 0u);
    }
    __device__ __forceinline__ void get(float (&x)[4]) const {
        const float2 a = unpack_half2(v.x), b = unpack_half2(v.y);
        x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
    }
    __device__ __forceinline__ Four from(int lane) const {
        return {make_uint2(__shfl_sync(0xffffffffu, v.x, lane), __shfl_sync(0xffffffffu, v.y, lane))};
    }
};
__device__ __forceinline__ void store4(float *p, const float (&x)[4]) {
    *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void store4(__half *p, const float (&x)[4]) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_half2(x[0], x[1]), pack_half2(x[2], x[3]));
}

// The signed maximum of a block (eight neighbouring lanes, four elements
// each): the first element of strictly largest magnitude, NaN never (the
// quantizer's rule), 0 for a block of zeros. From the block's largest and its
// smallest element; only where both have the same size does the order decide.
__device__ __noinline__ float first_of_largest(const float (&x)[4], int sub) {
    float best = -1.0f, val = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (fabsf(x[i]) > best) best = fabsf(x[i]), val = x[i];
#pragma unroll
    for (int m = 1; m <= 4; m <<= 1) {
        const float ob = __shfl_xor_sync(0xffffffffu, best, m), ov = __shfl_xor_sync(0xffffffffu, val, m);
        // on a tie the lane with the lower elements, whose bit m is clear, keeps its own
        if (ob > best || (ob == best && (sub & m))) best = ob, val = ov;
    }
    return best > 0.0f ? val : 0.0f;
}
__device__ __forceinline__ float signed_max(const float (&x)[4], int sub) {
    float hi = fmaxf(fmaxf(fmaxf(0.0f, x[0]), x[1]), fmaxf(x[2], x[3]));
    float lo = fminf(fminf(fminf(0.0f, x[0]), x[1]), fminf(x[2], x[3]));
#pragma unroll
    for (int m = 1; m <= 4; m <<= 1) {
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, m));
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, m));
    }
    if (__any_sync(0xffffffffu, hi == -lo && hi > 0.0f)) return first_of_largest(x, sub);
    return hi > -lo ? hi : hi < -lo ? lo : 0.0f;
}

// A warp takes ROWS x (32 / kLanes) rows of one token and one kind (q, k or v)
// at a time: their loads are in flight together, and what the token needs (its
// slot, its position's cosines and sines) is loaded and worked out once. TURN:
// 0 no rotation, 1 of halves, 2 of neighbours.
template <int D, class TI, class TO, int ROWS, int TURN>
__global__ void __launch_bounds__(256) kv_append_kernel(const KvAppendParams p) {
    pdl_allow_dependents();
    pdl_wait_prior_grids();
    using G = KvGroup<D>;
    constexpr int kLanes = D / 4, kAside = 32 / kLanes, kBatch = ROWS * kAside;
    const int lane = threadIdx.x & 31, sub = lane % kLanes, aside = lane / kLanes;
    const uint32_t q_batches = (p.n_heads + kBatch - 1) / kBatch, kv_batches = (p.c.n_heads + kBatch - 1) / kBatch;
    const uint32_t batches = q_batches + 2 * kv_batches, total = static_cast<uint32_t>(p.n_tok) * batches;
    const int half = p.rot_dim >> 3;  // lanes of the first halves of the rotated channels
    const bool low = sub < half, turned = sub < 2 * half;
    const uint32_t step = gridDim.x * (blockDim.x >> 5);
    // the bounds are the warp's, so that every lane takes part in the shuffles
    for (uint32_t unit = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); unit < total; unit += step) {
        const int tok = static_cast<int>(unit / batches);
        const uint32_t batch = unit - tok * batches;
        const bool is_q = batch < q_batches, is_k = !is_q && batch < q_batches + kv_batches;
        const int first = static_cast<int>(is_q ? batch : (batch - q_batches) - (is_k ? 0 : kv_batches)) * kBatch + aside;
        const int rows = is_q ? p.n_heads : p.c.n_heads;
        const TI *const src = static_cast<const TI *>(is_q ? p.q : is_k ? p.k : p.v) +
                              tok * (is_q ? p.q_stride : is_k ? p.k_stride : p.v_stride) + first * D + 4 * sub;
        const int slot = is_q ? -1 : p.slots[tok];
        int pos = TURN != 0 ? p.positions[tok] : 0;
        Four<TI> raw[ROWS];
#pragma unroll
        for (int j = 0; j < ROWS; ++j) raw[j].load(src + j * kAside * D, j * kAside < rows - first);
        bool ok = true;
        float c[4], s[4];  // s: less than zero what the first element of a rotated pair takes of the second
        int partner = lane;
        if (TURN != 0) {
            if (pos < 0 || pos >= p.n_pos) {
                if (lane == 0) record_error(p.err, kErrBadIndex);
                ok = false;
                pos = 0;
            }
            if (turned && p.n_pos > 0) {
                const float *row_t = p.rope + static_cast<int64_t>(pos) * p.rot_dim;
                if (TURN == 2) {
                    const float4 v = __ldg(reinterpret_cast<const float4 *>(row_t + 4 * sub));
                    c[0] = c[1] = v.x, c[2] = c[3] = v.z;
                    s[0] = -v.y, s[1] = v.y, s[2] = -v.w, s[3] = v.w;
                } else {
                    partner = low ? lane + half : lane - half;
                    const float4 *at = reinterpret_cast<const float4 *>(row_t) + 2 * (low ? sub : sub - half);
                    const float4 v0 = __ldg(at), v1 = __ldg(at + 1);
                    c[0] = v0.x, c[1] = v0.z, c[2] = v1.x, c[3] = v1.z;
                    s[0] = low ? -v0.y : v0.y, s[1] = low ? -v0.w : v0.w;
                    s[2] = low ? -v1.y : v1.y, s[3] = low ? -v1.w : v1.w;
                }
            }
        }
        const int left = rows - first;  // row j is there if j kAside < left
        TO *out = static_cast<TO *>(is_q ? p.q_out : is_k ? p.k_out : p.v_out);
        const int writes = ok && out != nullptr ? left : 0;
        out += (static_cast<int64_t>(tok) * rows + first) * D + 4 * sub;
        // (each product and the sum rounded by itself)
        auto rotate = [&](const Four<TI> &row, float (&x)[4]) {
            row.get(x);
            if (TURN == 0) return;
            float o[4];
            if (TURN == 2) {
                o[0] = x[1], o[1] = x[0], o[2] = x[3], o[3] = x[2];
            } else {
                row.from(partner).get(o);
            }
            if (turned)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = __fadd_rn(__fmul_rn(x[e], c[e]), __fmul_rn(o[e], s[e]));
        };
        const bool full = left + aside >= kBatch;  // (all rows of the batch are there: alike in every lane)
        if (is_q) {
            if (full && ok) {
#pragma unroll
                for (int j = 0; j < ROWS; ++j) {
                    float x[4];
                    rotate(raw[j], x);
                    store4(out + j * kAside * D, x);
                }
            } else {
#pragma unroll
                for (int j = 0; j < ROWS; ++j) {
                    float x[4];
                    rotate(raw[j], x);
                    if (j * kAside < writes) store4(out + j * kAside * D, x);
                }
            }
            continue;
        }
        if (ok && slot >= p.c.n_slots && lane == 0) record_error(p.err, kErrBadIndex);
        const bool kept = ok && slot >= 0 && slot < p.c.n_slots;
        // the group of the first row, and where in it this lane's codes and scale go: a value row's units hold two
        // bytes of every block, so two blocks' lanes trade halves and each writes four bytes, the lane of the even
        // block unit 2t, the other unit 2t + 1
        const int b = sub >> 3, t = sub & 7;
        uint8_t *group = nullptr;
        uint32_t code_at = 0, scale_at = 0;
        if (kept) {
            group = p.c.group<D>(slot, 0) + static_cast<int64_t>(first) * p.c.page_groups * G::kBytes;
            const int i = (slot % p.c.page_size) & 15, r = kv_value_row(i);
            code_at = is_k ? i * G::kRow + (t * G::kNB + b) * 4
                           : G::kV + r * G::kRow + (kv_value_unit(r, 2 * t + (b & 1)) * G::kNB + (b & ~1)) * 2;
            scale_at = (is_k ? G::kKS : G::kVS) + i * G::kScaleRow + 2 * b;
        }
        const int keeps = kept ? left : 0;
        const int64_t group_step = static_cast<int64_t>(kAside) * p.c.page_groups * G::kBytes;
#pragma unroll
        for (int j = 0; j < ROWS; ++j, group += group_step) {
            if (j * kAside >= left + aside) break;
            float x[4];
            if (is_k)
                rotate(raw[j], x);
            else
                raw[j].get(x);
            if (j * kAside < writes) store4(out + j * kAside * D, x);
            // Q4_0 (each step rounded in f32, as quantize_rows has it)
            const float d = signed_max(x, sub) * -0.125f;
            const float id = d != 0.0f ? __frcp_rn(d) : 0.0f;
            uint32_t e[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) e[i] = q4_0_code(__fadd_rn(__fmul_rn(x[i], id), 8.5f));
            const uint32_t codes = __byte_perm(__byte_perm(e[0], e[1], 0x0040), __byte_perm(e[2], e[3], 0x0040), 0x5410);
            uint32_t w = codes | (__shfl_down_sync(0xffffffffu, codes, 4) << 4);
            if (!is_k) {
                const uint32_t other = __shfl_xor_sync(0xffffffffu, w, 8);
                w = b & 1 ? __byte_perm(other, w, 0x7632) : __byte_perm(w, other, 0x5410);
            }
            if (t < 4 && j * kAside < keeps) {
                *reinterpret_cast<uint32_t *>(group + code_at) = w;
                if (t == 0) *reinterpret_cast<unsigned short *>(group + scale_at) = __half_as_ushort(__float2half_rn(d));
            }
        }
    }
}

// The values of cache rows: a token's k rows, then its v rows, ROWS at a time
// as above. A lane takes one 4-byte word (elements 4t .. 4t + 3 and 16 more of a
// block), D/8 lanes a row.
template <int D, int ROWS>
__global__ void __launch_bounds__(256) kv_read_kernel(const KvCacheView c, const int32_t *__restrict__ slots, int n,
                                                      float *__restrict__ k_out, float *__restrict__ v_out,
                                                      int32_t *err) {
    pdl_allow_dependents();
    pdl_wait_prior_grids();
    using G = KvGroup<D>;
    constexpr int kLanes = D / 8, kAside = 32 / kLanes;
    const int lane = threadIdx.x & 31, b = (lane % kLanes) >> 2, t = lane & 3;
    const int n_k = k_out != nullptr ? c.n_heads : 0, per_tok = n_k + (v_out != nullptr ? c.n_heads : 0);
    const uint32_t batches = (per_tok + ROWS * kAside - 1) / (ROWS * kAside);
    const uint32_t total = static_cast<uint32_t>(n) * batches, step = gridDim.x * (blockDim.x >> 5);
    for (uint32_t unit = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); unit < total; unit += step) {
        const int tok = static_cast<int>(unit / batches);
        const int first = static_cast<int>(unit - tok * batches) * (ROWS * kAside) + lane / kLanes;
        const int slot = slots[tok];
        if (slot >= c.n_slots && lane == 0) record_error(err, kErrBadIndex);
        const bool there = slot >= 0 && slot < c.n_slots;
        const int i = there ? (slot % c.page_size) & 15 : 0, r = kv_value_row(i);
        const uint8_t *const g0 = there ? c.group<D>(slot, 0) : nullptr;
        uint32_t w[ROWS];
        unsigned short d[ROWS];
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            const int h = first + j * kAside;
            w[j] = 0, d[j] = 0;
            if (!there || h >= per_tok) continue;
            const bool is_k = h < n_k;
            const uint8_t *g = g0 + static_cast<int64_t>(is_k ? h : h - n_k) * c.page_groups * G::kBytes;
            if (is_k) {
                w[j] = *reinterpret_cast<const uint32_t *>(g + i * G::kRow + (t * G::kNB + b) * 4);
            } else {
                const unsigned short *vr = reinterpret_cast<const unsigned short *>(g + G::kV + r * G::kRow);
                w[j] = vr[kv_value_unit(r, 2 * t) * G::kNB + b] |
                       static_cast<uint32_t>(vr[kv_value_unit(r, 2 * t + 1) * G::kNB + b]) << 16;
            }
            d[j] = reinterpret_cast<const unsigned short *>(g + (is_k ? G::kKS : G::kVS) + i * G::kScaleRow)[b];
        }
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            const int h = first + j * kAside;
            if (h >= per_tok) break;
            const float ds = f16_bits_to_f32(d[j]);
            float x[2][4];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const uint32_t n = (w[j] >> (4 * q)) & 0x0F0F0F0Fu;
#pragma unroll
                for (int e = 0; e < 4; ++e)  // a code in the low byte of 2^23, less 2^23 + 8: exact, and so is the product
                    x[q][e] = there ? (__uint_as_float(__byte_perm(n, 0x4B000000u, 0x7650 + e)) - 8388616.0f) * ds : 0.0f;
            }
            const bool is_k = h < n_k;
            float *out = (is_k ? k_out : v_out) + (static_cast<int64_t>(tok) * c.n_heads + (is_k ? h : h - n_k)) * D + 32 * b + 4 * t;
            store4(out, x[0]);
            store4(out + 16, x[1]);
        }
    }
}

namespace {

// Rows a warp has in flight: eight where that still leaves a few rounds for
// every warp of the machine, two from one row a warp on, else one (8191 tokens
// of 32 + 2 x 8 heads of 128, written and read: 58.8 us with eight, 62.3 with four,
// 79.9 with two; 64 of 32 + 2 x 32: 6.9 with one, 6.6 with two, 7.6 with four; 1
// of 32 + 2 x 8: 3.7, 4.3, 5.4). Reading is best at two (56.1 us of those 58.8).
int rows_at_once(int64_t warps, int sms) {
    return warps >= static_cast<int64_t>(sms) * 512 ? 8 : warps >= static_cast<int64_t>(sms) * 32 ? 2 : 1;
}

template <int D, class TI, class TO, int ROWS> cudaError_t launch_append_rows(const KvAppendParams &p, int sms, cudaStream_t s) {
    const int rows = ROWS * (128 / D);
    const int64_t warps = static_cast<int64_t>(p.n_tok) * ((p.n_heads + rows - 1) / rows + 2 * ((p.c.n_heads + rows - 1) / rows));
    const int grid = static_cast<int>(std::min<int64_t>((warps + 7) / 8, static_cast<int64_t>(sms) * 8));
    return p.rope == nullptr ? launch_pdl(kv_append_kernel<D, TI, TO, ROWS, 0>, grid, 256, 0, s, p)
           : p.pairs         ? launch_pdl(kv_append_kernel<D, TI, TO, ROWS, 2>, grid, 256, 0, s, p)
                             : launch_pdl(kv_append_kernel<D, TI, TO, ROWS, 1>, grid, 256, 0, s, p);
}

template <int D, class TI, class TO> cudaError_t launch_append(const KvAppendParams &p, int sms, cudaStream_t s) {
    const int per_tok = p.n_heads + 2 * p.c.n_heads;
    switch (rows_at_once(static_cast<int64_t>(p.n_tok) * per_tok / (128 / D), sms)) {
    case 8: return launch_append_rows<D, TI, TO, 8>(p, sms, s);
    case 2: return launch_append_rows<D, TI, TO, 2>(p, sms, s);
    default: return launch_append_rows<D, TI, TO, 1>(p, sms, s);
    }
}

template <int D>
cudaError_t launch_append_types(const KvAppendParams &p, int in_type, int out_type, int sms, cudaStream_t s) {
    if (in_type == QG_F32)
        return out_type == QG_F32 ? launch_append<D, float, float>(p, sms, s) : launch_append<D, float, __half>(p, sms, s);
    return out_type == QG_F32 ? launch_append<D, __half, float>(p, sms, s) : launch_append<D, __half, __half>(p, sms, s);
}

template <int D>
cudaError_t launch_read(const KvCacheView &c, const int32_t *slots, int n, float *k_out, float *v_out, int32_t *err,
                        int sms, cudaStream_t s) {
    const int aside = 256 / D, per_tok = ((k_out != nullptr) + (v_out != nullptr)) * c.n_heads;
    const bool two = rows_at_once(static_cast<int64_t>(n) * per_tok / aside, sms) > 1;
    const int rows = (two ? 2 : 1) * aside;
    const int64_t warps = static_cast<int64_t>(n) * ((per_tok + rows - 1) / rows);
    const int grid = static_cast<int>(std::min<int64_t>((warps + 7) / 8, static_cast<int64_t>(sms) * 8));
    return two ? launch_pdl(kv_read_kernel<D, 2>, grid, 256, 0, s, c, slots, n, k_out, v_out, err)
               : launch_pdl(kv_read_kernel<D, 1>, grid, 256, 0, s, c, slots, n, k_out, v_out, err);
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendParams &p, int head_dim, int in_type, int out_type, int sms, cudaStream_t s) {
    return head_dim == 64 ? launch_append_types<64>(p, in_type, out_type, sms, s)
                          : launch_append_types<128>(p, in_type, out_type, sms, s);
}

cudaError_t launch_kv_read(const KvCacheView &c, int head_dim, const int32_t *slots, int64_t n, float *k_out,
                           float *v_out, int32_t *err, int sms, cudaStream_t s) {
    return head_dim == 64 ? launch_read<64>(c, slots, static_cast<int>(n), k_out, v_out, err, sms, s)
                          : launch_read<128>(c, slots, static_cast<int>(n), k_out, v_out, err, sms, s);
}

}  // namespace qg
