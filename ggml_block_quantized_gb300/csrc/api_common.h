// api_common.h - host helpers that the C entry points of api.cu and
// attn_api.cu share (defined in api.cu).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace qg {

struct DeviceInfo {
    int device;
    int sms;
    int smem_optin;  // opt-in dynamic shared memory per CTA (bytes)
    int32_t *err;    // device address of g_device_error on this device
};

// The current device's properties, looked up once per device.
int current_device(DeviceInfo *info);

// Keeps the error's text for qg_last_cuda_error and returns QG_ERR_CUDA.
int cuda_fail(cudaError_t e, const char *where = "");

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace qg
