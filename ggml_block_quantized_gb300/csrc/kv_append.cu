// kv_append.cu - writing rows to the 4-bit paged cache and reading their
// values back (include/qattn.h: qkv_append, qkv_read).
//
// A row is one head of one token (q, k or v), D elements, four to a lane: D/4
// lanes hold a row, eight lanes a Q4_0 block. A warp holds 128 elements, that
// is one row of D = 128 or two of D = 64; the rows of q, k and v of a token
// follow one another. The rotation's partner channel is in another lane of the
// row (one shuffle an element), the block's signed maximum takes three
// butterfly steps among its eight lanes, and the four lanes with elements 0..15
// of a block take the codes of 16..31 by one shuffle and own one 4-byte code
// word each.
#include "kv_cache.cuh"
#include "quant_codes.cuh"

namespace qg {

template <class T> __device__ __forceinline__ void load4(const T *p, float (&x)[4]);
template <> __device__ __forceinline__ void load4<float>(const float *p, float (&x)[4]) {
    const float4 v = *reinterpret_cast<const float4 *>(p);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
}
template <> __device__ __forceinline__ void load4<__half>(const __half *p, float (&x)[4]) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    x[0] = f16_bits_to_f32(v.x), x[1] = f16_bits_to_f32(v.x >> 16);
    x[2] = f16_bits_to_f32(v.y), x[3] = f16_bits_to_f32(v.y >> 16);
}
__device__ __forceinline__ void store4(float *p, const float (&x)[4]) {
    *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void store4(__half *p, const float (&x)[4]) {
    const __half2 a = __floats2half2_rn(x[0], x[1]), b = __floats2half2_rn(x[2], x[3]);
    *reinterpret_cast<uint2 *>(p) =
        make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
}

// The signed maximum of a block (eight neighbouring lanes, four elements
// each): the first element of strictly largest magnitude, NaN never (the
// quantizer's rule), +0 for a block of zeros.
__device__ __forceinline__ float block_signed_max(const float (&x)[4], int sub) {
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

template <int D, class TI, class TO>
__global__ void __launch_bounds__(256) kv_append_kernel(const KvAppendParams p) {
    pdl_allow_dependents();
    pdl_wait_prior_grids();
    using G = KvGroup<D>;
    constexpr int kLanes = D / 4, kRows = 32 / kLanes;
    const int lane = threadIdx.x & 31, sub = lane % kLanes;
    const int per_tok = p.n_heads + 2 * p.c.n_heads;
    const int total = p.n_tok * per_tok;
    const int half = p.rot_dim >> 3;  // lanes of the first halves of the rotated channels
    const int step = static_cast<int>(gridDim.x * (blockDim.x >> 5)) * kRows;
    // the bound is the warp's (its first row), so that every lane takes part in the shuffles
    for (int first = static_cast<int>(blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)) * kRows; first < total;
         first += step) {
        const int row = first + lane / kLanes;
        const bool live = row < total;
        const int tok = live ? row / per_tok : 0;
        const int h = live ? row - tok * per_tok : 0;
        const bool is_q = h < p.n_heads, is_k = !is_q && h < p.n_heads + p.c.n_heads;
        const int hk = is_q ? 0 : (is_k ? h - p.n_heads : h - p.n_heads - p.c.n_heads);
        float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        bool ok = live;
        if (live) {
            const TI *src = is_q ? static_cast<const TI *>(p.q) + tok * p.q_stride + h * D
                            : is_k ? static_cast<const TI *>(p.k) + tok * p.k_stride + hk * D
                                   : static_cast<const TI *>(p.v) + tok * p.v_stride + hk * D;
            load4(src + 4 * sub, x);
        }
        if (p.rope != nullptr) {
            int pos = live ? p.positions[tok] : 0;
            if (pos < 0 || pos >= p.n_pos) {
                if (sub == 0) record_error(p.err, kErrBadIndex);
                ok = false;
                pos = 0;
            }
            const float *row_t = p.rope + static_cast<int64_t>(pos) * p.rot_dim;
            const bool turned = (is_q || is_k) && sub < 2 * half;
            if (p.pairs) {
                if (turned) {
                    const float4 cs = __ldg(reinterpret_cast<const float4 *>(row_t + 4 * sub));
                    const float a0 = x[0], b0 = x[1], a1 = x[2], b1 = x[3];
                    x[0] = __fsub_rn(__fmul_rn(a0, cs.x), __fmul_rn(b0, cs.y));
                    x[1] = __fadd_rn(__fmul_rn(a0, cs.y), __fmul_rn(b0, cs.x));
                    x[2] = __fsub_rn(__fmul_rn(a1, cs.z), __fmul_rn(b1, cs.w));
                    x[3] = __fadd_rn(__fmul_rn(a1, cs.w), __fmul_rn(b1, cs.z));
                }
            } else {
                const bool low = sub < half;
                const int at = low ? sub : sub - half;
                const int partner = (lane - sub) + (turned ? (low ? sub + half : at) : sub);
                float o[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) o[i] = __shfl_sync(0xffffffffu, x[i], partner);
                if (turned) {
                    const float4 c0 = __ldg(reinterpret_cast<const float4 *>(row_t + 8 * at));
                    const float4 c1 = __ldg(reinterpret_cast<const float4 *>(row_t + 8 * at) + 1);
                    const float c[4] = {c0.x, c0.z, c1.x, c1.z}, s[4] = {c0.y, c0.w, c1.y, c1.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        x[i] = low ? __fsub_rn(__fmul_rn(x[i], c[i]), __fmul_rn(o[i], s[i]))
                                   : __fadd_rn(__fmul_rn(o[i], s[i]), __fmul_rn(x[i], c[i]));
                }
            }
        }
        // f32 rows out
        if (ok) {
            const int64_t at = is_q ? (static_cast<int64_t>(tok) * p.n_heads + h) * D
                                    : (static_cast<int64_t>(tok) * p.c.n_heads + hk) * D;
            TO *out = static_cast<TO *>(is_q ? p.q_out : is_k ? p.k_out : p.v_out);
            if (out != nullptr) store4(out + at + 4 * sub, x);
        }
        if (__all_sync(0xffffffffu, is_q)) continue;
        // Q4_0 (each step rounded in f32, as quantize_rows has it)
        const float d = block_signed_max(x, sub) / -8.0f;
        const float id = d != 0.0f ? 1.0f / d : 0.0f;
        uint32_t codes = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = java_f2i(__fadd_rn(__fmul_rn(x[i], id), 8.5f));
            codes |= (static_cast<uint32_t>(c < 15 ? c : 15) & 0xFu) << (8 * i);
        }
        const uint32_t upper = __shfl_down_sync(0xffffffffu, codes, 4);
        const int slot = live && !is_q ? p.slots[tok] : -1;
        if (!ok || is_q || slot < 0) continue;
        if (slot >= p.c.n_slots) {
            if (sub == 0) record_error(p.err, kErrBadIndex);
            continue;
        }
        uint8_t *g = p.c.group<D>(slot, hk);
        const int i = (slot % p.c.page_size) & 15, b = sub >> 3, t = sub & 7;
        if (t < 4) {
            const uint32_t w = codes | (upper << 4);
            if (is_k) {
                *reinterpret_cast<uint32_t *>(g + i * G::kRow + (t * G::kNB + b) * 4) = w;
            } else {
                const int r = kv_value_row(i);
                unsigned short *vr = reinterpret_cast<unsigned short *>(g + G::kV + r * G::kRow);
                vr[kv_value_unit(r, 2 * t) * G::kNB + b] = static_cast<unsigned short>(w & 0xFFFFu);
                vr[kv_value_unit(r, 2 * t + 1) * G::kNB + b] = static_cast<unsigned short>(w >> 16);
            }
            if (t == 0)
                reinterpret_cast<unsigned short *>(g + (is_k ? G::kKS : G::kVS) + i * G::kScaleRow)[b] =
                    __half_as_ushort(__float2half_rn(d));
        }
    }
}

// The values of a cache row, four elements to a lane as above: the k rows of a
// token, then its v rows.
template <int D>
__global__ void __launch_bounds__(256) kv_read_kernel(const KvCacheView c, const int32_t *__restrict__ slots, int n,
                                                      float *__restrict__ k_out, float *__restrict__ v_out,
                                                      int32_t *err) {
    pdl_allow_dependents();
    pdl_wait_prior_grids();
    using G = KvGroup<D>;
    constexpr int kLanes = D / 4;
    const int kinds = (k_out != nullptr) + (v_out != nullptr);
    const int per_tok = kinds * c.n_heads;
    const int64_t lanes = static_cast<int64_t>(n) * per_tok * kLanes;
    for (int64_t at = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; at < lanes;
         at += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t row = at / kLanes;
        const int sub = static_cast<int>(at % kLanes);
        const int64_t tok = row / per_tok;
        int h = static_cast<int>(row - tok * per_tok);
        const bool is_k = k_out != nullptr && h < c.n_heads;
        if (!is_k && k_out != nullptr) h -= c.n_heads;
        const int slot = slots[tok];
        float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (slot >= c.n_slots) {
            if (sub == 0) record_error(err, kErrBadIndex);
        } else if (slot >= 0) {
            const uint8_t *g = c.group<D>(slot, h);
            const int i = (slot % c.page_size) & 15, b = sub >> 3, t = sub & 3;
            uint32_t w;
            if (is_k) {
                w = *reinterpret_cast<const uint32_t *>(g + i * G::kRow + (t * G::kNB + b) * 4);
            } else {
                const int r = kv_value_row(i);
                const unsigned short *vr = reinterpret_cast<const unsigned short *>(g + G::kV + r * G::kRow);
                w = vr[kv_value_unit(r, 2 * t) * G::kNB + b] |
                    static_cast<uint32_t>(vr[kv_value_unit(r, 2 * t + 1) * G::kNB + b]) << 16;
            }
            if (sub & 4) w >>= 4;
            const float d = f16_bits_to_f32(
                reinterpret_cast<const unsigned short *>(g + (is_k ? G::kKS : G::kVS) + i * G::kScaleRow)[b]);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                x[e] = static_cast<float>(static_cast<int>((w >> (8 * e)) & 0xFu) - 8) * d;  // exact
        }
        store4((is_k ? k_out : v_out) + (tok * c.n_heads + h) * D + 4 * sub, x);
    }
}

namespace {

template <int D, class TI, class TO>
cudaError_t launch_append(const KvAppendParams &p, int sms, cudaStream_t s) {
    const int64_t warps = (static_cast<int64_t>(p.n_tok) * (p.n_heads + 2 * p.c.n_heads) * (D / 4) + 31) / 32;
    int64_t grid = (warps + 7) / 8;
    if (grid > static_cast<int64_t>(sms) * 8) grid = static_cast<int64_t>(sms) * 8;
    return launch_pdl(kv_append_kernel<D, TI, TO>, static_cast<int>(grid), 256, 0, s, p);
}

template <int D>
cudaError_t launch_append_types(const KvAppendParams &p, int in_type, int out_type, int sms, cudaStream_t s) {
    if (in_type == QG_F32)
        return out_type == QG_F32 ? launch_append<D, float, float>(p, sms, s) : launch_append<D, float, __half>(p, sms, s);
    return out_type == QG_F32 ? launch_append<D, __half, float>(p, sms, s) : launch_append<D, __half, __half>(p, sms, s);
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendParams &p, int head_dim, int in_type, int out_type, int sms, cudaStream_t s) {
    return head_dim == 64 ? launch_append_types<64>(p, in_type, out_type, sms, s)
                          : launch_append_types<128>(p, in_type, out_type, sms, s);
}

cudaError_t launch_kv_read(const KvCacheView &c, int head_dim, const int32_t *slots, int64_t n, float *k_out,
                           float *v_out, int32_t *err, int sms, cudaStream_t s) {
    const int kinds = (k_out != nullptr) + (v_out != nullptr);
    int64_t grid = (n * kinds * c.n_heads * (head_dim / 4) + 255) / 256;
    if (grid > static_cast<int64_t>(sms) * 16) grid = static_cast<int64_t>(sms) * 16;
    return head_dim == 64 ? launch_pdl(kv_read_kernel<64>, static_cast<int>(grid), 256, 0, s, c, slots,
                                       static_cast<int>(n), k_out, v_out, err)
                          : launch_pdl(kv_read_kernel<128>, static_cast<int>(grid), 256, 0, s, c, slots,
                                       static_cast<int>(n), k_out, v_out, err);
}

}  // namespace qg
