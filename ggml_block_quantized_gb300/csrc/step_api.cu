// step_api.cu - the C ABI declared in include/qstep.h: argument validation and
// kernel launches. Nothing here allocates device memory or synchronizes.
#include "api_common.h"
#include "step_kernels.cuh"

using namespace qg;

namespace {

bool float_type(int t) { return t == QG_F32 || t == QG_F16; }
bool aligned(const void *p, int type) { return (reinterpret_cast<uintptr_t>(p) & (type == QG_F32 ? 3u : 1u)) == 0; }
constexpr int64_t kMaxStride = int64_t(1) << 40;
bool stride_ok(int64_t stride) { return stride >= 0 && stride <= kMaxStride; }
bool finite(float x) { return x - x == 0.0f; }

}  // namespace

extern "C" {

int qnorm_residual(const qnorm_args *a, qg_stream_t stream) {
    if (!a) return QG_ERR_NULL;
    if (!float_type(a->h_type) || !float_type(a->y_type) || !float_type(a->x_type)) return QG_ERR_TYPE;
    if (a->xq && a->act_type != QG_Q8_0 && a->act_type != QG_Q8_1 && a->act_type != QG_Q8_K) return QG_ERR_TYPE;
    if (a->n < 0 || a->n > (1 << 30) || a->d < 1 || a->d > 16384 || !stride_ok(a->h_stride) || !stride_ok(a->y_stride) ||
        !stride_ok(a->gate_stride) || (a->h_out && (!stride_ok(a->h_out_stride) || (a->n > 1 && a->h_out_stride < a->d))) ||
        !finite(a->scale) || !finite(a->eps) || a->eps < 0.0f || (a->xq && a->d % (a->act_type == QG_Q8_K ? 256 : 32) != 0))
        return QG_ERR_SHAPE;
    if (a->n == 0) return QG_OK;
    if (!a->h || (!a->h_out && !a->x_out && !a->xq)) return QG_ERR_NULL;
    if (!aligned(a->h, a->h_type) || !aligned(a->y, a->y_type) || !aligned(a->post_w, QG_F32) || !aligned(a->post_b, QG_F32) ||
        !aligned(a->gate, QG_F32) || !aligned(a->w, QG_F32) || !aligned(a->b, QG_F32) || !aligned(a->h_out, a->h_type) ||
        !aligned(a->x_out, a->x_type))
        return QG_ERR_ALIGN;
    if (a->xq && (!aligned16(a->xq) || !norm_rows_on_16(*a))) return QG_ERR_ALIGN;
    DeviceInfo dev;
    const int st = current_device(&dev);
    if (st != QG_OK) return st;
    const cudaError_t e = launch_norm(*a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? QG_OK : cuda_fail(e, "norm launch");
}

int qsample(int type, const void *logits, int64_t stride, int64_t n, int64_t vocab, const float *temperature,
            const int32_t *top_k, const float *top_p, const float *min_p, const float *uniform, int32_t *token, float *prob,
            qg_stream_t stream) {
    if (!float_type(type)) return QG_ERR_TYPE;
    if (n < 0 || n > (1 << 24) || vocab < 1 || vocab > (1 << 19) || !stride_ok(stride)) return QG_ERR_SHAPE;
    if (n == 0) return QG_OK;
    if (!logits || !uniform || !token) return QG_ERR_NULL;
    if (!aligned(logits, type) || !aligned(temperature, QG_F32) || !aligned(top_k, QG_F32) || !aligned(top_p, QG_F32) ||
        !aligned(min_p, QG_F32) || !aligned(uniform, QG_F32) || !aligned(token, QG_F32) || !aligned(prob, QG_F32))
        return QG_ERR_ALIGN;
    DeviceInfo dev;
    const int st = current_device(&dev);
    if (st != QG_OK) return st;
    SampleParams p = {};
    p.logits = logits;
    p.temperature = temperature;
    p.top_k = top_k;
    p.top_p = top_p;
    p.min_p = min_p;
    p.uniform = uniform;
    p.token = token;
    p.prob = prob;
    p.stride = stride;
    p.vocab = static_cast<int>(vocab);
    const cudaError_t e = launch_sample(p, type, static_cast<int>(n), dev.sms, dev.device, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? QG_OK : cuda_fail(e, "sample launch");
}

}  // extern "C"
