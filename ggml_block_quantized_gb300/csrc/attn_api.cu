// attn_api.cu - the C ABI declared in include/qattn.h: argument validation and
// kernel launches. Nothing here allocates device memory or synchronizes.
#include "api_common.h"
#include "kv_cache.cuh"

using namespace qg;

namespace {

bool float_type(int t) { return t == QG_F32 || t == QG_F16; }
bool head_dim_ok(int d) { return d == 64 || d == 128; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
// A token stride in elements: at least the row, whole 16 bytes.
bool stride_ok(int64_t stride, int64_t row, int type) {
    return stride >= row && stride % (type == QG_F32 ? 4 : 8) == 0 && stride <= (int64_t(1) << 40);
}

// The cache's geometry (its data pointer is checked by the caller).
int check_cache(const qkv_cache *c, KvCacheView *v) {
    if (!c) return QG_ERR_NULL;
    if (qkv_cache_bytes(c->n_pages, c->n_kv_heads, c->head_dim, c->page_size) < 0) return QG_ERR_SHAPE;
    v->data = static_cast<uint8_t *>(c->data);
    v->n_slots = c->n_pages * c->page_size;
    v->n_pages = static_cast<int>(c->n_pages);
    v->n_heads = c->n_kv_heads;
    v->page_size = c->page_size;
    v->page_groups = c->page_size / 16;
    return QG_OK;
}

// Rows of one key/value head that a sequence's queries make: at most
// max_q_len * group, within what the kernels index.
constexpr int64_t kMaxRows = 1 << 20;

int check_heads(int n_heads, int n_kv_heads) {
    return n_heads >= 1 && n_kv_heads >= 1 && n_heads % n_kv_heads == 0 && n_heads <= 65536 ? QG_OK : QG_ERR_SHAPE;
}

}  // namespace

extern "C" {

int64_t qkv_cache_bytes(int64_t n_pages, int n_kv_heads, int head_dim, int page_size) {
    if (n_pages < 0 || n_kv_heads < 1 || n_kv_heads > 65536 || !head_dim_ok(head_dim) || page_size < 16 ||
        page_size % 16 != 0 || n_pages > INT32_MAX / page_size)
        return -1;
    return n_pages * page_size * n_kv_heads * (head_dim / 8 * 9);
}

int qkv_append(const qkv_cache *cache, const qkv_append_args *a, qg_stream_t stream) {
    KvAppendParams p = {};
    int st = check_cache(cache, &p.c);
    if (st != QG_OK) return st;
    if (!a) return QG_ERR_NULL;
    if (!float_type(a->in_type) || !float_type(a->out_type)) return QG_ERR_TYPE;
    const int d = cache->head_dim, n_heads = a->q ? a->n_heads : 0;
    if (a->n_tok < 0 || a->n_tok > (1 << 30) || (a->q && (check_heads(n_heads, cache->n_kv_heads) != QG_OK)) ||
        a->n_tok * (n_heads + 2 * static_cast<int64_t>(cache->n_kv_heads)) > (1 << 30))
        return QG_ERR_SHAPE;
    if (a->rope && (a->rot_dim < 8 || a->rot_dim % 8 != 0 || a->rot_dim > d || a->n_pos < 0)) return QG_ERR_SHAPE;
    if (a->n_tok == 0) return QG_OK;
    if (!a->k || !a->v || !a->slots || (a->q && !a->q_out) || (a->rope && !a->positions)) return QG_ERR_NULL;
    if (!cache->data && cache->n_pages > 0) return QG_ERR_NULL;
    const int64_t kv_row = static_cast<int64_t>(cache->n_kv_heads) * d, q_row = static_cast<int64_t>(n_heads) * d;
    if (!aligned16(cache->data) || !aligned16(a->q) || !aligned16(a->k) || !aligned16(a->v) || !aligned16(a->rope) ||
        !aligned16(a->q_out) || !aligned16(a->k_out) || !aligned16(a->v_out) || !aligned4(a->slots) ||
        !aligned4(a->positions))
        return QG_ERR_ALIGN;
    if ((a->q && !stride_ok(a->q_stride, q_row, a->in_type)) || !stride_ok(a->k_stride, kv_row, a->in_type) ||
        !stride_ok(a->v_stride, kv_row, a->in_type))
        return QG_ERR_SHAPE;
    DeviceInfo dev;
    st = current_device(&dev);
    if (st != QG_OK) return st;
    p.q = a->q;
    p.k = a->k;
    p.v = a->v;
    p.q_stride = a->q_stride;
    p.k_stride = a->k_stride;
    p.v_stride = a->v_stride;
    p.slots = a->slots;
    p.positions = a->positions;
    p.rope = a->rope;
    p.q_out = a->q_out;
    p.k_out = a->k_out;
    p.v_out = a->v_out;
    p.err = dev.err;
    p.n_tok = static_cast<int>(a->n_tok);
    p.n_heads = n_heads;
    p.n_pos = a->n_pos;
    p.rot_dim = a->rope ? a->rot_dim : 0;
    p.pairs = a->rope_pairs;
    const cudaError_t e =
        launch_kv_append(p, d, a->in_type, a->out_type, dev.sms, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? QG_OK : cuda_fail(e, "kv_append launch");
}

int qkv_read(const qkv_cache *cache, const int32_t *slots, int64_t n, float *k_out, float *v_out, qg_stream_t stream) {
    KvCacheView c;
    int st = check_cache(cache, &c);
    if (st != QG_OK) return st;
    if (n < 0 || n > (1 << 30) || n * c.n_heads > (1 << 30)) return QG_ERR_SHAPE;
    if (n == 0 || (!k_out && !v_out)) return QG_OK;
    if (!slots || (!cache->data && cache->n_pages > 0)) return QG_ERR_NULL;
    if (!aligned16(cache->data) || !aligned16(k_out) || !aligned16(v_out) || !aligned4(slots)) return QG_ERR_ALIGN;
    DeviceInfo dev;
    st = current_device(&dev);
    if (st != QG_OK) return st;
    const cudaError_t e = launch_kv_read(c, cache->head_dim, slots, n, k_out, v_out, dev.err, dev.sms,
                                         reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? QG_OK : cuda_fail(e, "kv_read launch");
}

size_t qkv_attend_workspace_bytes(int head_dim, int n_kv_heads, int n_heads, int max_q_len) {
    if (!head_dim_ok(head_dim) || check_heads(n_heads, n_kv_heads) != QG_OK || max_q_len < 1) return 0;
    const int64_t rows = static_cast<int64_t>(n_heads / n_kv_heads) * max_q_len;
    return rows > kMaxRows ? 0 : kv_attend_workspace(head_dim, static_cast<int>(rows));
}

int qkv_attend(const qkv_cache *cache, int type, const void *q, int64_t q_stride, void *out, const int32_t *table,
               int64_t table_stride, const int32_t *lengths, const int32_t *q_offsets, int64_t n_seq, int64_t n_tok,
               int n_heads, int max_q_len, float scale, void *workspace, size_t workspace_bytes, qg_stream_t stream) {
    KvAttendParams p = {};
    int st = check_cache(cache, &p.c);
    if (st != QG_OK) return st;
    if (!float_type(type)) return QG_ERR_TYPE;
    const int d = cache->head_dim;
    if (check_heads(n_heads, cache->n_kv_heads) != QG_OK || n_seq < 0 || n_tok < 0 || max_q_len < 1 ||
        n_seq > (1 << 24) || n_tok > (1 << 30) || table_stride < 0 || table_stride > INT32_MAX || (!q_offsets && n_tok < n_seq) ||
        !(scale == scale) || scale - scale != 0.0f)
        return QG_ERR_SHAPE;
    const size_t need = qkv_attend_workspace_bytes(d, cache->n_kv_heads, n_heads, max_q_len);
    if (need == 0) return QG_ERR_SHAPE;
    if (n_seq == 0 || n_tok == 0) return QG_OK;
    if (!q || !out || !lengths || (!table && table_stride > 0) || (!cache->data && cache->n_pages > 0))
        return QG_ERR_NULL;
    if (!aligned16(cache->data) || !aligned16(q) || !aligned16(out) || !aligned16(workspace) || !aligned4(table) ||
        !aligned4(lengths) || !aligned4(q_offsets))
        return QG_ERR_ALIGN;
    if (!stride_ok(q_stride, static_cast<int64_t>(n_heads) * d, type)) return QG_ERR_SHAPE;
    if (!workspace || workspace_bytes < need) return QG_ERR_WORKSPACE;
    DeviceInfo dev;
    st = current_device(&dev);
    if (st != QG_OK) return st;
    p.q = q;
    p.out = out;
    p.table = table;
    p.lengths = lengths;
    p.q_offsets = q_offsets;
    p.q_stride = q_stride;
    p.table_stride = table_stride;
    p.partial = static_cast<float *>(workspace);
    p.err = dev.err;
    p.scale = scale;
    p.n_seq = static_cast<int>(n_seq);
    p.n_tok = static_cast<int>(n_tok);
    p.n_heads = n_heads;
    p.group = n_heads / cache->n_kv_heads;
    p.max_q_len = max_q_len;
    const cudaError_t e = launch_kv_attend(p, d, type, dev.sms, dev.device, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? QG_OK : cuda_fail(e, "kv_attend launch");
}

int qattn_prompt(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                 int out_type, void *out, const int32_t *offsets, int64_t n_seq, int64_t n_tok, int n_heads,
                 int n_kv_heads, int head_dim, float scale, qg_stream_t stream) {
    if (!float_type(out_type)) return QG_ERR_TYPE;
    if (!head_dim_ok(head_dim) || check_heads(n_heads, n_kv_heads) != QG_OK || n_seq < 0 || n_tok < 0 ||
        n_seq > (1 << 24) || n_tok > (1 << 28) || !(scale == scale) || scale - scale != 0.0f)
        return QG_ERR_SHAPE;
    if (n_seq == 0 || n_tok == 0) return QG_OK;
    if (!q || !k || !v || !out || !offsets) return QG_ERR_NULL;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned4(offsets)) return QG_ERR_ALIGN;
    const int64_t kv_row = static_cast<int64_t>(n_kv_heads) * head_dim;
    if (!stride_ok(q_stride, static_cast<int64_t>(n_heads) * head_dim, QG_F16) ||
        !stride_ok(k_stride, kv_row, QG_F16) || !stride_ok(v_stride, kv_row, QG_F16))
        return QG_ERR_SHAPE;
    DeviceInfo dev;
    const int st = current_device(&dev);
    if (st != QG_OK) return st;
    PromptParams p = {};
    p.q = q;
    p.k = k;
    p.v = v;
    p.out = out;
    p.offsets = offsets;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.err = dev.err;
    p.scale = scale;
    p.n_seq = static_cast<int>(n_seq);
    p.n_tok = static_cast<int>(n_tok);
    p.n_heads = n_heads;
    p.n_kv_heads = n_kv_heads;
    p.group = n_heads / n_kv_heads;
    const cudaError_t e =
        launch_prompt_attend(p, head_dim, out_type, dev.sms, dev.device, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? QG_OK : cuda_fail(e, "prompt_attend launch");
}

}  // extern "C"
