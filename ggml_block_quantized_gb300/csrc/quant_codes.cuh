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

}  // namespace qg
