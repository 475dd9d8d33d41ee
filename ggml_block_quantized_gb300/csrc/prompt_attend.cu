// prompt_attend.cu - causal attention over whole packed prompts
// (include/qattn.h, qattn_prompt).
//
// One warp for one query row: 32 keys at a time, a lane each for the scores,
// the running maximum and sum of the softmax, then D/32 channels a lane.
#include "kv_cache.cuh"

namespace qg {

template <int D, class TO>
__global__ void __launch_bounds__(128) prompt_row_kernel(const PromptParams p) {
    pdl_allow_dependents();
    pdl_wait_prior_grids();
    constexpr int kPer = D / 32;
    __shared__ float qs[4][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row = blockIdx.x, h = blockIdx.y * 4 + warp;
    if (h >= p.n_heads) return;
    int start = -1;
    for (int s = 0; s < p.n_seq; ++s) {
        const int a = p.offsets[s], b = p.offsets[s + 1];
        if (a < 0 || b < a || b > p.n_tok) {
            if (lane == 0) record_error(p.err, kErrBadIndex);
            continue;
        }
        if (row >= a && row < b) start = a;
    }
    if (start < 0) return;
    const int hk = h / p.group;
    const __half *q = static_cast<const __half *>(p.q) + row * p.q_stride + h * D;
    const __half *kb = static_cast<const __half *>(p.k) + hk * D, *vb = static_cast<const __half *>(p.v) + hk * D;
    for (int i = lane; i < D; i += 32) qs[warp][i] = __half2float(q[i]) * p.scale;
    __syncwarp();
    float m = -INFINITY, l = 0.0f, o[kPer] = {};
    for (int t0 = start; t0 <= row; t0 += 32) {
        const int t = t0 + lane;
        float sc = -INFINITY;
        if (t <= row) {
            sc = 0.0f;
            for (int i = 0; i < D; ++i) sc += qs[warp][i] * __half2float(kb[t * p.k_stride + i]);
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
    TO *out = static_cast<TO *>(p.out) + (static_cast<int64_t>(row) * p.n_heads + h) * D;
    for (int k = 0; k < kPer; ++k) out[32 * k + lane] = static_cast<TO>(l > 0.0f || l != l ? o[k] / l : 0.0f);
}

cudaError_t launch_prompt_attend(const PromptParams &p, int head_dim, int out_type, int, int, cudaStream_t s) {
    const dim3 grid(p.n_tok, (p.n_heads + 3) / 4);
    if (head_dim == 64) {
        if (out_type == QG_F32) prompt_row_kernel<64, float><<<grid, 128, 0, s>>>(p);
        else prompt_row_kernel<64, __half><<<grid, 128, 0, s>>>(p);
    } else {
        if (out_type == QG_F32) prompt_row_kernel<128, float><<<grid, 128, 0, s>>>(p);
        else prompt_row_kernel<128, __half><<<grid, 128, 0, s>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace qg
