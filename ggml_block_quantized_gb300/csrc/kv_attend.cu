// kv_attend.cu - attention of new tokens over the 4-bit paged cache
// (include/qattn.h, qkv_attend).
//
// One warp for one query row (a token's head): 32 cache tokens at a time, a
// lane each for the scores, then the running maximum and sum of the softmax,
// then four (or two) channels a lane for the weighted values.
#include "kv_cache.cuh"

namespace qg {

template <int D, class T>
__global__ void __launch_bounds__(128) kv_attend_kernel(const KvAttendParams p) {
    pdl_allow_dependents();
    pdl_wait_prior_grids();
    using G = KvGroup<D>;
    constexpr int kPer = D / 32;
    __shared__ float qs[4][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int s = blockIdx.x, h = blockIdx.y * 4 + warp;
    if (h >= p.n_heads) return;
    int q0 = s, q1 = s + 1;
    if (p.q_offsets != nullptr) q0 = p.q_offsets[s], q1 = p.q_offsets[s + 1];
    if (q0 < 0 || q1 < q0 || q1 > p.n_tok || q1 - q0 > p.max_q_len) {
        if (lane == 0) record_error(p.err, kErrBadIndex);
        return;
    }
    int len = p.lengths[s];
    const int64_t room = p.table_stride * p.c.page_size;
    if (len < 0 || len > room) {
        if (lane == 0) record_error(p.err, kErrBadIndex);
        len = len < 0 ? 0 : static_cast<int>(room);
    }
    const int hk = h / p.group;
    for (int tok = q0; tok < q1; ++tok) {
        const T *q = static_cast<const T *>(p.q) + tok * p.q_stride + h * D;
        __syncwarp();
        for (int i = lane; i < D; i += 32) qs[warp][i] = static_cast<float>(q[i]) * p.scale;
        __syncwarp();
        const int seen = len - (q1 - tok) + 1;
        float m = -INFINITY, l = 0.0f, o[kPer] = {};
        for (int t0 = 0; t0 < seen; t0 += 32) {
            const int t = t0 + lane;
            float sc = -INFINITY;
            const uint8_t *g = nullptr;
            if (t < seen) {
                const int page = p.table[s * p.table_stride + t / p.c.page_size];
                if (page < 0 || page >= p.c.n_pages) {
                    record_error(p.err, kErrBadIndex);
                } else {
                    g = p.c.data + ((static_cast<int64_t>(page) * p.c.n_heads + hk) * p.c.page_groups +
                                    ((t % p.c.page_size) >> 4)) * G::kBytes;
                    const int i = t & 15;
                    float sum = 0.0f;
                    for (int b = 0; b < G::kNB; ++b) {
                        float part = 0.0f;
                        for (int w4 = 0; w4 < 4; ++w4) {
                            const uint32_t w =
                                *reinterpret_cast<const uint32_t *>(g + i * G::kRow + (w4 * G::kNB + b) * 4);
                            for (int e = 0; e < 4; ++e) {
                                part += qs[warp][32 * b + 4 * w4 + e] * (static_cast<int>((w >> (8 * e)) & 15u) - 8);
                                part += qs[warp][32 * b + 16 + 4 * w4 + e] *
                                        (static_cast<int>((w >> (8 * e + 4)) & 15u) - 8);
                            }
                        }
                        sum += part * f16_bits_to_f32(
                                          reinterpret_cast<const unsigned short *>(g + G::kKS + i * G::kScaleRow)[b]);
                    }
                    sc = sum;
                }
            }
            float mt = sc;
            for (int k = 16; k; k >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, k));
            const float mn = fmaxf(m, mt);
            if (mn == -INFINITY) continue;
            const float keep = expf(m - mn);
            const float w = g != nullptr ? expf(sc - mn) : 0.0f;
            m = mn;
            l = l * keep + w;
            for (int k = 0; k < kPer; ++k) o[k] *= keep;
            for (int j = 0; j < 32; ++j) {
                const float wj = __shfl_sync(0xffffffffu, w, j);
                const uint8_t *gj = reinterpret_cast<const uint8_t *>(
                    __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(g), j));
                if (gj == nullptr) continue;
                const int i = (t0 + j) & 15, r = kv_value_row(i);
                for (int k = 0; k < kPer; ++k) {
                    const int e = lane;  // element of block k
                    const int byte = e & 15, u = kv_value_unit(r, byte >> 1);
                    const int c = (gj[G::kV + r * G::kRow + (u * G::kNB + k) * 2 + (byte & 1)] >> (e & 16 ? 4 : 0)) & 15;
                    o[k] += wj * ((c - 8) *
                                  f16_bits_to_f32(
                                      reinterpret_cast<const unsigned short *>(gj + G::kVS + i * G::kScaleRow)[k]));
                }
            }
        }
        for (int k = 16; k; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
        T *out = static_cast<T *>(p.out) + (static_cast<int64_t>(tok) * p.n_heads + h) * D;
        for (int k = 0; k < kPer; ++k) out[32 * k + lane] = static_cast<T>(l > 0.0f || l != l ? o[k] / l : 0.0f);
    }
}

size_t kv_attend_workspace(int, int) { return 16; }

cudaError_t launch_kv_attend(const KvAttendParams &p, int head_dim, int type, int, int, cudaStream_t s) {
    const dim3 grid(p.n_seq, (p.n_heads + 3) / 4);
    if (head_dim == 64) {
        if (type == QG_F32) kv_attend_kernel<64, float><<<grid, 128, 0, s>>>(p);
        else kv_attend_kernel<64, __half><<<grid, 128, 0, s>>>(p);
    } else {
        if (type == QG_F32) kv_attend_kernel<128, float><<<grid, 128, 0, s>>>(p);
        else kv_attend_kernel<128, __half><<<grid, 128, 0, s>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace qg
