// step_kernels.cuh - launch interface of the kernels behind include/qstep.h.
#pragma once
#include "qg_common.cuh"
#include "qstep.h"

namespace qg {

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
