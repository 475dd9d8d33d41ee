// step_kernels.cuh - launch interface of the kernels behind include/qstep.h.
#pragma once
#include "qg_common.cuh"
#include "qstep.h"

namespace qg {

// Whether a matrix's rows can be read and written 16 bytes at a time; of one that is not there its stride says nothing.
inline bool rows_on_16(const void *p, int64_t stride, int type) {
    return p == nullptr || ((reinterpret_cast<uintptr_t>(p) & 15u) == 0 && stride % (type == QG_F32 ? 4 : 8) == 0);
}

// All of a norm's. (The rows of x_out are contiguous; with xq, whose blocks are made from such rows alone, d is a multiple of 32.)
inline bool norm_rows_on_16(const qnorm_args &a) {
    return a.d % 8 == 0 && rows_on_16(a.h, a.h_stride, a.h_type) && rows_on_16(a.y, a.y_stride, a.y_type) &&
           rows_on_16(a.gate, a.gate_stride, QG_F32) && rows_on_16(a.post_w, 0, QG_F32) && rows_on_16(a.post_b, 0, QG_F32) &&
           rows_on_16(a.w, 0, QG_F32) && rows_on_16(a.b, 0, QG_F32) && rows_on_16(a.h_out, a.h_out_stride, a.h_type) &&
           rows_on_16(a.x_out, a.d, a.x_type);
}

cudaError_t launch_norm(const qnorm_args &a, cudaStream_t s);

struct SampleParams {
    const void *logits;
    const float *temperature, *top_p, *min_p, *uniform;
    const int32_t *top_k;
    int32_t *token;
    float *prob;
    int64_t stride;
    int vocab;
    int n, blocks, slice;  // rows; blocks of a row; logits of a block (these and what follows: the launch's)
    float2 power[64];
};

cudaError_t launch_sample(SampleParams p, int type, int n, int sms, int device, cudaStream_t s);

}  // namespace qg
