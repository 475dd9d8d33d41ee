// norm.cu - the norms before and after a block with its gate and residual
// (include/qstep.h, qnorm_residual).
//
// A row lies in the registers of its threads from the first load to the last
// store: with u = N(y), h' = h + scale gate u and x = N(h') every input is read
// once and every output written once, whatever norms there are. A norm's sums
// are formed by shuffles and, for rows of several warps, one barrier each; with
// `layer` the mean is known before the squares are summed, from the registers,
// so that a large mean costs no bits.
//
// Threads hold eight consecutive elements at a time (rows on 16-byte
// boundaries: one 32-byte load or two of 16; a block of the activation types is
// then 4 lanes or one warp, and xq needs no memory), or four single ones a row's
// threads apart (any alignment; eight took a fifth longer for 1037 rows of 1283).
// Up to 8192 (4096) elements a thread has one such set, so that a single row is
// read by as many threads as there can be.
//
// Memory bounds it where there is work for every multiprocessor: 8191 rows of
// 4096, f16 h, f32 y, f16 x take 52.6 us (335 MB at 6.4 TB/s), close to a copy's
// 49.4; there the instructions of an element count next (38 of them took 57.7 us;
// a layer norm takes 57.0, activation blocks instead of x 59 to 64). 1037 rows of
// 1283 in f32 take 9.8 us, 48 rows of 5120 with both norms 4.2, one row of 4096 3.0:
// the chain of launch, load, two sums by shuffles and barrier, store. Rows off
// 16-byte boundaries of more than 8192 elements spill 52 to 60 bytes a thread
// (2048 of 16383 in f32 136 us, of 16384 90).
#include "quant_act.cuh"
#include "step_kernels.cuh"

namespace qg {

namespace {

constexpr int kMaxThreads = 1024;

// Sum over a row's threads; `part` alternates so that one barrier a sum is enough.
struct RowSum {
    float *buf;  // [2][warps of the row, 32 at most]
    int warps, warp, barrier, part = 0;
    __device__ __forceinline__ float operator()(float v) {
#pragma unroll
        for (int m = 16; m; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
        if (warps == 1) return v;
        float *b = buf + part * 32;
        part ^= 1;
        const int lane = threadIdx.x & 31;
        if (lane == 0) b[warp] = v;
        named_barrier(barrier, warps * 32);
        v = lane < warps ? b[lane] : 0.0f;
#pragma unroll
        for (int m = 16; m; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
        return v;
    }
};

__device__ __forceinline__ void load8(const float *p, float (&v)[8], bool wide32) {
    if (wide32) {
        asm volatile("ld.global.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                     : "l"(p)
                     : "memory");
    } else {
        const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
}
__device__ __forceinline__ void load8(const __half *p, float (&v)[8], bool) {
    const uint4 a = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ void store8(float *p, const float (&v)[8], bool wide32) {
    if (wide32) {
        asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]),
                     "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                     : "memory");
    } else {
        reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
}
__device__ __forceinline__ void store8(__half *p, const float (&v)[8], bool) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// The elements that a thread holds of a row. WIDE: SETS x 8, set k is elements
// 8 (t + k T) on; else SETS x 4, element i of them is t + i T (T threads a row).
template <bool WIDE, int SETS> struct Held {
    static constexpr int W = WIDE ? 8 : 4;
    using Values = float[SETS][W];
    int t, threads, d;
    bool wide32;  // rows of f32 lie on 32-byte boundaries
    template <class F> __device__ __forceinline__ void each(F f) const {  // f(set, first element) or f(i, element)
        if (WIDE) {
#pragma unroll
            for (int k = 0; k < SETS; ++k) {
                const int e = 8 * (t + k * threads);
                if (e < d) f(k, e);
            }
        } else {
#pragma unroll
            for (int i = 0; i < W * SETS; ++i) {
                const int e = t + i * threads;
                if (e < d) f(i, e);
            }
        }
    }
    template <class T> __device__ __forceinline__ void load(const T *p, Values &v) const {
        each([&](int i, int e) {
            if constexpr (WIDE) load8(p + e, v[i], wide32);
            else v[i / W][i % W] = static_cast<float>(p[e]);
        });
    }
    template <class T> __device__ __forceinline__ void store(T *p, const Values &v) const {
        each([&](int i, int e) {
            if constexpr (WIDE) store8(p + e, v[i], wide32);
            else p[e] = static_cast<T>(v[i / W][i % W]);
        });
    }
    // f(value, vector's element) over all held elements; p a [d] vector (nullptr: `none`)
    template <class T, class F> __device__ __forceinline__ void with(const T *p, float none, Values &v, F f) const {
        if (p == nullptr) {
#pragma unroll
            for (int k = 0; k < SETS; ++k)
#pragma unroll
                for (int i = 0; i < W; ++i) v[k][i] = f(v[k][i], none);
            return;
        }
        each([&](int i, int e) {
            if constexpr (WIDE) {
                float w[8];
                load8(p + e, w, wide32);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = f(v[i][j], w[j]);
            } else {
                v[i / W][i % W] = f(v[i / W][i % W], static_cast<float>(p[e]));
            }
        });
    }
    __device__ __forceinline__ float sum(const Values &v) const {  // (elements past the row's end are 0)
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < SETS; ++k)
#pragma unroll
            for (int i = 0; i < W; ++i) s += v[k][i];
        return s;
    }
    __device__ __forceinline__ float squares(const Values &v) const {
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < SETS; ++k)
#pragma unroll
            for (int i = 0; i < W; ++i) s = fmaf(v[k][i], v[k][i], s);
        return s;
    }
    __device__ __forceinline__ void clear(Values &v) const {
#pragma unroll
        for (int k = 0; k < SETS; ++k)
#pragma unroll
            for (int i = 0; i < W; ++i) v[k][i] = 0.0f;
    }
    // v becomes N(v; w, b)
    __device__ __forceinline__ void norm(Values &v, const float *w, const float *b, bool layer, float eps, float per,
                                         RowSum &row_sum) const {
        if (layer) {
            const float mean = row_sum(sum(v)) * per;
            each([&](int i, int) {
                if constexpr (WIDE) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[i][j] -= mean;
                } else {
                    v[i / W][i % W] -= mean;
                }
            });
        }
        const float inv = rsqrtf(row_sum(squares(v)) * per + eps);  // (off by 2^-22 at most)
        with(w, 1.0f, v, [&](float x, float y) { return x * inv * y; });
        if (b != nullptr) with(b, 0.0f, v, [](float x, float y) { return x + y; });
    }
};

// blockDim.x threads a row, a multiple of 32, blockDim.y rows; per: 1 / d.
// MOST: threads of a block at most. With rows on 16-byte boundaries registers are kept few enough for 1280 threads and
// more a multiprocessor: what is on its way from memory counts (8191 rows of 4096, f16 and f32, before later steps: 57.4 us with
// three blocks of 512, 69.5 with two, 57.6 with four).
template <class TH, class TY, bool WIDE, int SETS, int MOST>
__global__ void __launch_bounds__(MOST, MOST == 1024 || !WIDE ? 1 : MOST == 512 ? 3 : 5) norm_kernel(const qnorm_args a, const float per, const bool wide32) {
    __shared__ float sums[8 * 64];
    pdl_allow_dependents();
    pdl_wait_prior_grids();
    const int t = threadIdx.x, threads = blockDim.x;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    if (row >= a.n) return;
    const Held<WIDE, SETS> held{t, threads, static_cast<int>(a.d), wide32};
    RowSum row_sum{sums + threadIdx.y * 64, threads / 32, t / 32, 1 + static_cast<int>(threadIdx.y)};
    const bool layer = a.layer != 0;
    const TH *const h = static_cast<const TH *>(a.h) + row * a.h_stride;
    typename Held<WIDE, SETS>::Values v;
    held.clear(v);
    if (a.y != nullptr) {
        held.load(static_cast<const TY *>(a.y) + row * a.y_stride, v);
        typename Held<WIDE, SETS>::Values early;  // (of more sets h is read when u is done: both would not fit the registers)
        if constexpr (SETS == 1) {
            held.clear(early);
            held.load(h, early);
        }
        if (a.post_w != nullptr) held.norm(v, a.post_w, a.post_b, layer, a.eps, per, row_sum);
        if (a.gate != nullptr) held.with(a.gate + row * a.gate_stride, 1.0f, v, [](float x, float y) { return x * y; });
        if constexpr (SETS == 1) {
#pragma unroll
            for (int i = 0; i < held.W; ++i) v[0][i] = fmaf(a.scale, v[0][i], early[0][i]);
        } else {
            held.with(h, 0.0f, v, [&](float x, float y) { return fmaf(a.scale, x, y); });
        }
    } else {
        held.load(h, v);
    }
    if (a.h_out != nullptr) held.store(static_cast<TH *>(a.h_out) + row * a.h_out_stride, v);
    if (a.x_out == nullptr && a.xq == nullptr) return;
    held.norm(v, a.w, a.b, layer, a.eps, per, row_sum);
    if (a.x_out != nullptr) {
        if (a.x_type == QG_F32) held.store(static_cast<float *>(a.x_out) + row * a.d, v);
        else held.store(static_cast<__half *>(a.x_out) + row * a.d, v);
    }
    if constexpr (WIDE) {
        if (a.xq != nullptr) {
            const int64_t bytes = a.act_type == QG_Q8_K ? a.d / 256 * 292 : a.d / 32 * (a.act_type == QG_Q8_1 ? 36 : 34);
            uint8_t *xq = static_cast<uint8_t *>(a.xq) + row * bytes;
            held.each([&](int k, int e) {
                if (a.act_type == QG_Q8_K) quantize_held<QG_Q8_K>(v[k], xq, e / 8);
                else if (a.act_type == QG_Q8_1) quantize_held<QG_Q8_1>(v[k], xq, e / 8);
                else quantize_held<QG_Q8_0>(v[k], xq, e / 8);
            });
        }
    }
}

bool on32(const void *p, int64_t stride) { return p == nullptr || ((reinterpret_cast<uintptr_t>(p) & 31u) == 0 && stride % 8 == 0); }

template <class TH, class TY, bool WIDE> cudaError_t launch(const qnorm_args &a, cudaStream_t s) {
    constexpr int kWidth = WIDE ? 8 : 4;
    const int units = static_cast<int>((a.d + kWidth - 1) / kWidth);
    const int sets = units <= kMaxThreads ? 1 : units <= 2 * kMaxThreads ? 2 : 4;
    const int threads = ((units + sets - 1) / sets + 31) / 32 * 32;
    const int rows = threads >= 256 ? 1 : 256 / threads;
    // (of f16 matrices it says nothing)
    const bool wide32 = on32(a.h, a.h_stride) && on32(a.y, a.y_stride) && on32(a.gate, a.gate_stride) && on32(a.post_w, 0) && on32(a.post_b, 0) &&
                        on32(a.w, 0) && on32(a.b, 0) && on32(a.h_out, a.h_out_stride) && on32(a.x_out, a.d);
    auto kernel = norm_kernel<TH, TY, WIDE, 2, 1024>;
    if constexpr (!WIDE)
        if (sets == 4) kernel = norm_kernel<TH, TY, WIDE, 4, 1024>;
    if (sets == 1) kernel = threads * rows <= 256 ? norm_kernel<TH, TY, WIDE, 1, 256> : threads <= 512 ? norm_kernel<TH, TY, WIDE, 1, 512> : norm_kernel<TH, TY, WIDE, 1, 1024>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((a.n + rows - 1) / rows));
    cfg.blockDim = dim3(threads, rows);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    g_launch_step = "cudaLaunchKernelEx";
    return cudaLaunchKernelEx(&cfg, kernel, a, 1.0f / static_cast<float>(a.d), wide32);
}

template <class TH, class TY> cudaError_t launch_types(const qnorm_args &a, cudaStream_t s) {
    return norm_rows_on_16(a) ? launch<TH, TY, true>(a, s) : launch<TH, TY, false>(a, s);
}

}  // namespace

cudaError_t launch_norm(const qnorm_args &a, cudaStream_t s) {
    if (a.h_type == QG_F32) return a.y_type == QG_F32 ? launch_types<float, float>(a, s) : launch_types<float, __half>(a, s);
    return a.y_type == QG_F32 ? launch_types<__half, float>(a, s) : launch_types<__half, __half>(a, s);
}

}  // namespace qg
