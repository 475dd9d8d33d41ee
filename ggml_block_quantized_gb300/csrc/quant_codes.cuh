// quant_codes.cuh - the code arithmetic of the 32-element weight types that
// the quantizers (quantize.cu) and the 4-bit cache (kv_append.cu) share.
#pragma once
#include <stdint.h>

namespace qg {

// Float to int as the lesson's Java code casts it: truncation toward zero,
// 0 for NaN, the int range's end beyond it (a NaN element, or a scale so
// small that 1/d overflows, reaches those cases). Written out rather than
// left to the conversion instruction's own NaN and overflow rules.
__device__ __forceinline__ int java_f2i(float t) {
    if (t != t) return 0;
    if (t >= 2147483648.0f) return 2147483647;
    if (t <= -2147483648.0f) return -2147483647 - 1;
    return static_cast<int>(t);
}

// min(java_f2i(t), 15) & 15 for t = x (1/d) + 8.5 of a Q4_0 block, in three
// operations. There t is in 0.4 .. 16.6 or, where 1/d overflows or x is not
// finite, an infinity or NaN: clamped (NaN becomes 0, as the cast has it), then
// truncated by an addition of 2^23 that rounds toward zero. The code is the
// result's low byte; its high bytes are those of 2^23.
__device__ __forceinline__ uint32_t q4_0_code(float t) {
    return __float_as_uint(__fadd_rz(fminf(fmaxf(t, 0.0f), 15.5f), 8388608.0f));
}

}  // namespace qg
