// quant_act.cuh - the activation quantizers' rules (quantize_act, see
// quantize.cu) for values that a kernel holds in registers: a lane's eight
// consecutive ones, a block in consecutive lanes of a warp.
#pragma once
#include "qg_common.cuh"

namespace qg {

// The row's block that holds elements 8c .. 8c + 7 (this lane's v); every lane
// of a block's calls together. row: the row's first byte.
template <int TYPE> __device__ __forceinline__ void quantize_held(const float (&v)[8], uint8_t *row, int c) {
    constexpr int kLanes = TYPE == QG_Q8_K ? 32 : 4, kLeast = TYPE == QG_Q8_K ? -127 : -128;
    constexpr int kBytes = TYPE == QG_Q8_K ? 292 : TYPE == QG_Q8_1 ? 36 : 34;
    // (a warp may hold the row's end: its last lanes are then not here, but blocks are whole)
    const uint32_t lanes = kLanes == 32 ? 0xffffffffu : ((1u << (kLanes & 31)) - 1) << (threadIdx.x & 28);
    // fmaxf ignores NaN, as the scalar rule's comparison does (a block of 32 that holds nothing else has d = NaN)
    float amax = TYPE == QG_Q8_K ? 0.0f : fabsf(v[0]);
#pragma unroll
    for (int i = TYPE == QG_Q8_K ? 0 : 1; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
#pragma unroll
    for (int m = 1; m < kLanes; m <<= 1) amax = fmaxf(amax, __shfl_xor_sync(lanes, amax, m));
    const float d = amax / 127.0f, id = d != 0.0f ? 1.0f / d : 0.0f;
    uint32_t w[2] = {0u, 0u};
    int sum = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int q = code_from_rounded(roundf(__fmul_rn(v[i], id)), kLeast, 127);
        sum += q;
        w[i >> 2] |= (static_cast<uint32_t>(q) & 0xFFu) << (8 * (i & 3));
    }
    uint8_t *block = row + static_cast<int64_t>(c / kLanes) * kBytes;
    const int part = c % kLanes;
    if (TYPE == QG_Q8_K) {
        uint32_t *q = reinterpret_cast<uint32_t *>(block + 4 + 8 * part);
        q[0] = w[0], q[1] = w[1];
        sum += __shfl_xor_sync(lanes, sum, 1);  // of 16 elements
        if ((part & 1) == 0) reinterpret_cast<int16_t *>(block + 260)[part >> 1] = static_cast<int16_t>(sum);
        if (part == 0) *reinterpret_cast<float *>(block) = d;
        return;
    }
    unsigned short *q = reinterpret_cast<unsigned short *>(block + (TYPE == QG_Q8_1 ? 4 : 2) + 8 * part);  // 2-byte aligned
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = static_cast<unsigned short>(w[i >> 1] >> (16 * (i & 1)));
    if (TYPE == QG_Q8_1) {
        sum += __shfl_xor_sync(lanes, sum, 1);
        sum += __shfl_xor_sync(lanes, sum, 2);
    }
    if (part == 0) {
        *reinterpret_cast<unsigned short *>(block) = __half_as_ushort(__float2half_rn(d));
        if (TYPE == QG_Q8_1) {
            const float s = __fmul_rn(static_cast<float>(sum), d);  // a block holding inf: 0 * inf, one fixed quiet NaN
            reinterpret_cast<unsigned short *>(block)[1] = s != s ? 0x7E00u : __half_as_ushort(__float2half_rn(s));
        }
    }
}

}  // namespace qg
