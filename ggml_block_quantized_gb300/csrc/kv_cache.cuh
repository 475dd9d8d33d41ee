// kv_cache.cuh - the layout of the 4-bit paged cache (include/qattn.h,
// qkv_cache) for its kernels, and their launch interface.
#pragma once
#include "qattn.h"
#include "qg_common.cuh"

namespace qg {

constexpr int32_t kErrBadIndex = 4;  // device error word: a page, slot, position, length or offset out of range

// A group: 16 tokens of one head. Key codes | value codes | key scales | value scales.
template <int D> struct KvGroup {
    static constexpr int kNB = D / 32;       // Q4_0 blocks of a row
    static constexpr int kRow = D / 2;       // code bytes of a row
    static constexpr int kScaleRow = D / 16; // scale bytes of a row
    static constexpr int kV = 8 * D, kKS = 16 * D, kVS = 17 * D, kBytes = 18 * D;
};

// The row in which the value codes of token i of a group lie: 0 2 4 6 1 3 5 7
// and the same of the upper eight, so that the tokens 2t (t = 0..3) that the
// four lanes of a tensor-core fragment read together are neighbours.
__host__ __device__ constexpr int kv_value_row(int i) { return (i & 8) | ((i & 1) << 2) | ((i >> 1) & 3); }
// Which of a value row's eight 2-byte units (of every block) holds unit u: the
// halves are swapped in rows 2, 3, 6, 7, which puts the four neighbours' reads
// into different shared-memory banks.
__host__ __device__ constexpr int kv_value_unit(int row, int u) { return u ^ ((row & 2) << 1); }

// Two f16 as one word, the first in the low half.
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float2 unpack_half2(uint32_t v) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&v));
}

// A cache as its kernels take it.
struct KvCacheView {
    uint8_t *data;
    int64_t n_slots;  // n_pages * page_size
    int n_pages, n_heads, page_size, page_groups;

    // The group of `slot` (in range) and head h.
    template <int D> __device__ __forceinline__ uint8_t *group(int slot, int h) const {
        const int page = slot / page_size, r = slot - page * page_size;
        return data + ((static_cast<int64_t>(page) * n_heads + h) * page_groups + (r >> 4)) * KvGroup<D>::kBytes;
    }
};

struct KvAppendParams {
    KvCacheView c;
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;
    const int32_t *slots, *positions;
    const float *rope;
    void *q_out, *k_out, *v_out;
    int32_t *err;
    int n_tok, n_heads, n_pos, rot_dim, pairs;
};

cudaError_t launch_kv_append(const KvAppendParams &p, int head_dim, int in_type, int out_type, int sms, cudaStream_t s);
cudaError_t launch_kv_read(const KvCacheView &c, int head_dim, const int32_t *slots, int64_t n, float *k_out,
                           float *v_out, int32_t *err, int sms, cudaStream_t s);

struct KvAttendParams {
    KvCacheView c;
    const void *q;
    void *out;
    const int32_t *table, *lengths, *q_offsets;
    int64_t q_stride, table_stride;
    float *partial;
    int32_t *err;
    float scale;
    int n_seq, n_tok, n_heads, group, max_q_len;
};

size_t kv_attend_workspace(int head_dim, int rows);
cudaError_t launch_kv_attend(const KvAttendParams &p, int head_dim, int type, int sms, int device, cudaStream_t s);

struct PromptParams {
    const void *q, *k, *v;
    void *out;
    const int32_t *offsets;
    int64_t q_stride, k_stride, v_stride;
    int32_t *err;
    float scale;
    int n_seq, n_tok, n_heads, n_kv_heads, group;
};

cudaError_t launch_prompt_attend(const PromptParams &p, int head_dim, int out_type, int sms, int device,
                                 cudaStream_t s);

}  // namespace qg
