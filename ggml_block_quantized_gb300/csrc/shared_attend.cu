// shared_attend.cu - attention of new tokens of sequences that share a prefix,
// over the 4-bit paged cache (include/qattn.h, qkv_attend_shared).
//
// All query rows of a key/value head see the whole prefix, so it is taken once
// for all of them: an item is one key/value head and 128 of its rows (token-major
// over the call's tokens and the head's group), its units tiles of 128 prefix
// tokens. The items' units form one list that the thread blocks share out in
// equal contiguous parts; each stretch of an item in a part leaves its rows'
// values, reference and sum in the workspace. Each sequence's own tokens go
// through kv_attend's kernels, which leave theirs there, too, and a last kernel
// joins a row's results in a fixed order.
#include <atomic>
#include <cfloat>

#include "kv_cache.cuh"

namespace qg {

namespace {

constexpr int kRows = 128;   // of an item
constexpr int kTokens = 128; // of a unit
constexpr int kMaxParts = 160;

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The prefix's length, checked, and the list of units.
struct Units {
    int len, tiles;      // tokens, units of an item
    int64_t all, share;  // of all items, of a part
    __device__ __forceinline__ Units(const SharedParams &p, int parts) {
        len = __ldg(p.prefix_len);
        const int64_t room = p.prefix_pages * static_cast<int64_t>(p.own.c.page_size);
        if (len < 0 || len > room) {
            record_error(p.own.err, kErrBadIndex);
            len = len < 0 ? 0 : static_cast<int>(room);
        }
        tiles = (len + kTokens - 1) / kTokens;
        all = static_cast<int64_t>(p.own.c.n_heads) * p.row_tiles * tiles;
        share = (all + parts - 1) / parts;
        if (share < 1) share = 1;
    }
};
// A stretch's place: parts and items both rise along the list, one of them at least from stretch to stretch.
__host__ __device__ constexpr int64_t stretch_floats(int d) { return static_cast<int64_t>(kRows) * (d + 2); }

// The channel whose value lies at place `at` of a stretch's row.
template <int D> __device__ __forceinline__ int channel_at(int at) { return at; }

// A thread a row.
template <int D, class T> __global__ void __launch_bounds__(kRows) prefix_kernel(const SharedParams p) {
    using G = KvGroup<D>;
    __shared__ float k_row[D], v_row[D];
    pdl_allow_dependents();
    pdl_wait_prior_grids();
    const KvAttendParams &a = p.own;
    const Units units(p, gridDim.x);
    int64_t u = blockIdx.x * units.share;
    const int64_t past = min(u + units.share, units.all);
    const float c = a.scale * 1.4426950408889634f;
    while (u < past) {
        const int64_t item = u / units.tiles;
        const int tile0 = static_cast<int>(u - item * units.tiles), n = static_cast<int>(min(past - u, static_cast<int64_t>(units.tiles - tile0)));
        u += n;
        const int head = static_cast<int>(item / p.row_tiles), row = static_cast<int>(item % p.row_tiles) * kRows + threadIdx.x;
        const int tok = row / a.group;
        const bool live = tok < a.n_tok;
        float q[D], o[D];
        for (int i = 0; i < D; ++i) {
            q[i] = live ? static_cast<float>(static_cast<const T *>(a.q)[tok * a.q_stride + (static_cast<int64_t>(head) * a.group + row - tok * a.group) * D + i]) : 0.0f;
            o[i] = 0.0f;
        }
        float ref = -INFINITY, sum = 0.0f;
        for (int t = tile0 * kTokens; t < min((tile0 + n) * kTokens, units.len); ++t) {
            const int page = __ldg(p.prefix_table + t / a.c.page_size);
            if (page < 0 || page >= a.c.n_pages) {
                if (threadIdx.x == 0) record_error(a.err, kErrBadIndex);
                continue;
            }
            const uint8_t *g = a.c.template group<D>(page * a.c.page_size + t % a.c.page_size, head);
            const int i = t & 15, vr = kv_value_row(i), j = threadIdx.x & 15;
            __syncthreads();
            if (threadIdx.x < D / 2) {
                const int b = threadIdx.x >> 4;
                const uint8_t kb = g[i * G::kRow + ((j / 4) * G::kNB + b) * 4 + j % 4];
                const uint8_t vb = g[G::kV + vr * G::kRow + (kv_value_unit(vr, j / 2) * G::kNB + b) * 2 + j % 2];
                const float ks = f16_bits_to_f32(reinterpret_cast<const unsigned short *>(g + G::kKS + i * G::kScaleRow)[b]);
                const uint32_t bits = reinterpret_cast<const unsigned short *>(g + G::kVS + i * G::kScaleRow)[b];
                const float vs = (bits & 0x7C00u) == 0x7C00u ? NAN : f16_bits_to_f32(bits);
                k_row[32 * b + j] = ((kb & 15) - 8) * ks, k_row[32 * b + 16 + j] = ((kb >> 4) - 8) * ks;
                v_row[32 * b + j] = ((vb & 15) - 8) * vs, v_row[32 * b + 16 + j] = ((vb >> 4) - 8) * vs;
            }
            __syncthreads();
            float s = 0.0f;
            for (int d = 0; d < D; ++d) s = fmaf(q[d], k_row[d], s);
            s *= c;
            const float next = fmaxf(ref, s), keep = exp2_approx(ref - (next == -INFINITY ? 0.0f : next)), w = exp2_approx(s - (next == -INFINITY ? 0.0f : next));
            ref = next;
            sum = fmaf(sum, keep, w);
            for (int d = 0; d < D; ++d) o[d] = fmaf(o[d], keep, w * v_row[d]);
        }
        float *out = p.stretches + (blockIdx.x + item) * stretch_floats(D);
        for (int d = 0; d < D; ++d) out[threadIdx.x * D + d] = o[d];
        reinterpret_cast<float2 *>(out + kRows * D)[threadIdx.x] = make_float2(ref, sum);
    }
}

// Joins each row's results: of its stretches of the prefix, and of its own tokens. Block (s, i): query i of sequence
// s; a warp a head.
template <int D, class T> __global__ void __launch_bounds__(256) shared_join_kernel(const SharedParams p, const int parts) {
    constexpr int kPer = D / 32;
    pdl_allow_dependents();
    pdl_wait_prior_grids();
    const KvAttendParams &a = p.own;
    const int lane = threadIdx.x & 31;
    int q0 = blockIdx.x, m = 1;
    if (a.q_offsets != nullptr) {
        q0 = __ldg(a.q_offsets + blockIdx.x);
        const int q1 = __ldg(a.q_offsets + blockIdx.x + 1);
        m = q0 < 0 || q1 < q0 || q1 > a.n_tok || q1 - q0 > a.max_q_len ? 0 : q1 - q0;
    }
    const Units units(p, parts);
    for (int i = blockIdx.y; i < m; i += gridDim.y) {
        const int tok = q0 + i;
        for (int h = threadIdx.x >> 5; h < a.n_heads; h += blockDim.x >> 5) {
            const int kv = h / a.group, row = tok * a.group + h - kv * a.group;
            const int64_t item = static_cast<int64_t>(kv) * p.row_tiles + row / kRows;
            const int64_t rest = static_cast<int64_t>(tok) * a.n_heads + h;
            float2 ml = reinterpret_cast<const float2 *>(a.rest_stats)[rest];
            float top = ml.x, den = ml.y, acc[kPer];
#pragma unroll
            for (int k = 0; k < kPer; ++k) acc[k] = __ldcg(a.rest + rest * D + channel_at<D>(lane * kPer + k));
            if (units.tiles > 0) {
                const int64_t c0 = item * units.tiles / units.share, c1 = ((item + 1) * units.tiles - 1) / units.share;
                for (int64_t c = c0; c <= c1; ++c) {
                    const float *part = p.stretches + (c + item) * stretch_floats(D);
                    ml = __ldcg(reinterpret_cast<const float2 *>(part + kRows * D) + row % kRows);
                    const float next = fmaxf(top, ml.x), ref = next == -INFINITY ? 0.0f : next;
                    const float keep = exp2_approx(top - ref), f = exp2_approx(ml.x - ref);
                    top = next;
                    den = den * keep + ml.y * f;
#pragma unroll
                    for (int k = 0; k < kPer; ++k)
                        acc[k] = acc[k] * keep + f * __ldcg(part + row % kRows * D + lane * kPer + k);
                }
            }
            const float inv = den == 0.0f ? 0.0f : 1.0f / den;  // no token seen: zeros
#pragma unroll
            for (int k = 0; k < kPer; ++k)
                static_cast<T *>(a.out)[rest * D + channel_at<D>(lane * kPer + k)] = static_cast<T>(acc[k] * inv);
        }
    }
}

int64_t row_tiles(int64_t n_tok, int group) { return (n_tok * group + kRows - 1) / kRows; }
size_t align(size_t n) { return (n + 255) / 256 * 256; }

template <int D, class T> cudaError_t launch(SharedParams &p, int sms, int device, cudaStream_t s) {
    const int parts = sms < kMaxParts ? sms : kMaxParts;
    cudaError_t e = launch_pdl(prefix_kernel<D, T>, parts, kRows, 0, s, p);
    if (e == cudaSuccess) e = launch_kv_attend(p.own, D, sizeof(T) == 4 ? QG_F32 : QG_F16, sms, device, s);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.own.n_seq), static_cast<unsigned>(p.own.max_q_len < 64 ? p.own.max_q_len : 64));
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, shared_join_kernel<D, T>, static_cast<const SharedParams>(p), static_cast<const int>(parts));
}

}  // namespace

// The workspace: kv_attend's own, the rows' results of their own tokens, the stretches.
size_t shared_attend_workspace(int head_dim, int n_kv_heads, int group, int64_t n_tok, int max_q_len) {
    const size_t rows = static_cast<size_t>(n_tok) * group * n_kv_heads;
    return align(kv_attend_workspace(head_dim, group * max_q_len)) + align(rows * head_dim * 4) + align(rows * 8) +
           static_cast<size_t>(kMaxParts + n_kv_heads * row_tiles(n_tok, group)) * stretch_floats(head_dim) * 4;
}

cudaError_t launch_shared_attend(SharedParams p, int head_dim, int type, int sms, int device, cudaStream_t s) {
    KvAttendParams &a = p.own;
    uint8_t *at = reinterpret_cast<uint8_t *>(a.partial);
    const size_t rows = static_cast<size_t>(a.n_tok) * a.n_heads;
    at += align(kv_attend_workspace(head_dim, a.group * a.max_q_len));
    a.rest = reinterpret_cast<float *>(at);
    at += align(rows * head_dim * 4);
    a.rest_stats = reinterpret_cast<float *>(at);
    at += align(rows * 8);
    p.stretches = reinterpret_cast<float *>(at);
    p.row_tiles = static_cast<int>(row_tiles(a.n_tok, a.group));
    if (head_dim == 64) return type == QG_F32 ? launch<64, float>(p, sms, device, s) : launch<64, __half>(p, sms, device, s);
    return type == QG_F32 ? launch<128, float>(p, sms, device, s) : launch<128, __half>(p, sms, device, s);
}

}  // namespace qg
