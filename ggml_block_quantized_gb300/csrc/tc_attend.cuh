// tc_attend.cuh - what the attention kernels on the 5th-generation tensor cores
// share: products S = Q K^T and O = P V with P in tensor memory, descriptors,
// tensor-memory loads, waits that leave shared memory to the operands.
#pragma once
#include "kv_cache.cuh"
#include "tc_common.cuh"

namespace qg {

// tcgen05.mma, kind::f16, f32 accumulators, and its commit, issued where
// `issue` is not 0 (one lane). The whole warp runs the code around them: its
// addresses and descriptors then stay in uniform registers, which the
// instructions take their operands from. The issuing warp is bound by its
// instructions' latency, not by their number on the multiprocessor, so the
// products come as blocks with one predicate and a constant high descriptor
// word: with descriptors added up in 64 bits and a predicate each, 32 products
// took about 3800 cycles to issue, 60% more than the tensor cores need.
// S (+)= Q K^T: 16 channels a product, the 64-channel halves 16 KB apart.
template <int D> __device__ __forceinline__ void mma_s(uint32_t issue, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t hi, uint32_t acc = 0) {
    if (D == 64)
        asm volatile(
            "{\n\t.reg .pred p0, p1, q;\n\t.reg .b64 da, db;\n\t.reg .b32 a, b;\n\tsetp.ne.u32 q, %4, 0;\n\tsetp.ne.u32 p0, %6, 0;\n\tsetp.eq.u32 p1, 0, 0;\n\t"
            "mov.b32 a, %1;\n\tmov.b32 b, %2;\n\t"
            "mov.b64 da, {a, %5};\n\tmov.b64 db, {b, %5};\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p0;\n\t"
            "add.u32 a, %1, 2;\n\tadd.u32 b, %2, 2;\n\t"
            "mov.b64 da, {a, %5};\n\tmov.b64 db, {b, %5};\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p1;\n\t"
            "add.u32 a, %1, 4;\n\tadd.u32 b, %2, 4;\n\t"
            "mov.b64 da, {a, %5};\n\tmov.b64 db, {b, %5};\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p1;\n\t"
            "add.u32 a, %1, 6;\n\tadd.u32 b, %2, 6;\n\t"
            "mov.b64 da, {a, %5};\n\tmov.b64 db, {b, %5};\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p1;\n\t"
            "}" ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(issue), "r"(hi), "r"(acc)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p0, p1, q;\n\t.reg .b64 da, db;\n\t.reg .b32 a, b;\n\tsetp.ne.u32 q, %4, 0;\n\tsetp.ne.u32 p0, %6, 0;\n\tsetp.eq.u32 p1, 0, 0;\n\t"
            "mov.b32 a, %1;\n\tmov.b32 b, %2;\n\t"
            "mov.b64 da, {a, %5};\n\tmov.b64 db, {b, %5};\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p0;\n\t"
            "add.u32 a, %1, 2;\n\tadd.u32 b, %2, 2;\n\t"
            "mov.b64 da, {a, %5};\n\tmov.b64 db, {b, %5};\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p1;\n\t"
            "add.u32 a, %1, 4;\n\tadd.u32 b, %2, 4;\n\t"
            "mov.b64 da, {a, %5};\n\tmov.b64 db, {b, %5};\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p1;\n\t"
            "add.u32 a, %1, 6;\n\tadd.u32 b, %2, 6;\n\t"
            "mov.b64 da, {a, %5};\n\tmov.b64 db, {b, %5};\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p1;\n\t"
            "add.u32 a, %1, 1024;\n\tadd.u32 b, %2, 1024;\n\t"
            "mov.b64 da, {a, %5};\n\tmov.b64 db, {b, %5};\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p1;\n\t"
            "add.u32 a, %1, 1026;\n\tadd.u32 b, %2, 1026;\n\t"
            "mov.b64 da, {a, %5};\n\tmov.b64 db, {b, %5};\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p1;\n\t"
            "add.u32 a, %1, 1028;\n\tadd.u32 b, %2, 1028;\n\t"
            "mov.b64 da, {a, %5};\n\tmov.b64 db, {b, %5};\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p1;\n\t"
            "add.u32 a, %1, 1030;\n\tadd.u32 b, %2, 1030;\n\t"
            "mov.b64 da, {a, %5};\n\tmov.b64 db, {b, %5};\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p1;\n\t"
            "}" ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(issue), "r"(hi), "r"(acc)
            : "memory");
}
// The same with Q in tensor memory, 8 columns a product.
template <int D> __device__ __forceinline__ void mma_s_tm(uint32_t issue, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t hi, uint32_t acc) {
#pragma unroll
    for (int h = 0; h < D / 64; ++h)
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t.reg .b64 db;\n\t.reg .b32 a, b;\n\tsetp.ne.u32 q, %5, 0;\n\tsetp.ne.u32 p, %4, 0;\n\t"
            "mov.b32 a, %1;\n\tmov.b32 b, %2;\n\t"
            "mov.b64 db, {b, %6};\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], db, %3, p;\n\t"
            "setp.ne.u32 p, 1, 0;\n\t"
            "add.u32 a, %1, 8;\n\tadd.u32 b, %2, 2;\n\t"
            "mov.b64 db, {b, %6};\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], db, %3, p;\n\t"
            "add.u32 a, %1, 16;\n\tadd.u32 b, %2, 4;\n\t"
            "mov.b64 db, {b, %6};\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], db, %3, p;\n\t"
            "add.u32 a, %1, 24;\n\tadd.u32 b, %2, 6;\n\t"
            "mov.b64 db, {b, %6};\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], db, %3, p;\n\t"
            "}" ::"r"(d), "r"(a + 32 * h), "r"(b + 1024 * h), "r"(idesc), "r"(h == 0 ? acc : 1u), "r"(issue), "r"(hi)
            : "memory");
}
// O (+)= P V: 16 keys a product, 8 columns of P and 2 KB of V; 128 keys, or 64.
template <int KEYS = 128> __device__ __forceinline__ void mma_pv(uint32_t issue, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc, uint32_t hi) {
    if (KEYS == 64)
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t.reg .b64 db;\n\t.reg .b32 a, b;\n\tsetp.ne.u32 q, %5, 0;\n\tsetp.ne.u32 p, %4, 0;\n\t"
            "mov.b32 a, %1;\n\tmov.b32 b, %2;\n\t"
            "mov.b64 db, {b, %6};\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], db, %3, p;\n\t"
            "setp.ne.u32 p, 1, 0;\n\t"
            "add.u32 a, %1, 8;\n\tadd.u32 b, %2, 128;\n\t"
            "mov.b64 db, {b, %6};\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], db, %3, p;\n\t"
            "add.u32 a, %1, 16;\n\tadd.u32 b, %2, 256;\n\t"
            "mov.b64 db, {b, %6};\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], db, %3, p;\n\t"
            "add.u32 a, %1, 24;\n\tadd.u32 b, %2, 384;\n\t"
            "mov.b64 db, {b, %6};\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], db, %3, p;\n\t"
            "}" ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(issue), "r"(hi)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t.reg .b64 db;\n\t.reg .b32 a, b;\n\tsetp.ne.u32 q, %5, 0;\n\tsetp.ne.u32 p, %4, 0;\n\t"
            "mov.b32 a, %1;\n\tmov.b32 b, %2;\n\t"
            "mov.b64 db, {b, %6};\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], db, %3, p;\n\t"
            "setp.ne.u32 p, 1, 0;\n\t"
            "add.u32 a, %1, 8;\n\tadd.u32 b, %2, 128;\n\t"
            "mov.b64 db, {b, %6};\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], db, %3, p;\n\t"
            "add.u32 a, %1, 16;\n\tadd.u32 b, %2, 256;\n\t"
            "mov.b64 db, {b, %6};\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], db, %3, p;\n\t"
            "add.u32 a, %1, 24;\n\tadd.u32 b, %2, 384;\n\t"
            "mov.b64 db, {b, %6};\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], db, %3, p;\n\t"
            "add.u32 a, %1, 32;\n\tadd.u32 b, %2, 512;\n\t"
            "mov.b64 db, {b, %6};\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], db, %3, p;\n\t"
            "add.u32 a, %1, 40;\n\tadd.u32 b, %2, 640;\n\t"
            "mov.b64 db, {b, %6};\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], db, %3, p;\n\t"
            "add.u32 a, %1, 48;\n\tadd.u32 b, %2, 768;\n\t"
            "mov.b64 db, {b, %6};\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], db, %3, p;\n\t"
            "add.u32 a, %1, 56;\n\tadd.u32 b, %2, 896;\n\t"
            "mov.b64 db, {b, %6};\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], db, %3, p;\n\t"
            "}" ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(issue), "r"(hi)
            : "memory");
}
__device__ __forceinline__ void commit(uint32_t issue, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar), "r"(issue)
        : "memory");
}
__device__ __forceinline__ void arrive_if(uint32_t issue, uint32_t bar) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t@q mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar),
                 "r"(issue)
                 : "memory");
}
// Bounded wait (about 1 s) that sleeps about NS nanoseconds between polls and
// gives up once another thread of the block has set the abort flag. Polling
// without a pause takes shared-memory cycles from the tensor cores' operands.
template <int NS> __device__ __forceinline__ bool sleep_wait(uint32_t bar, uint32_t parity, const volatile int *abort_flag) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    for (uint32_t i = 1; i < kWaitLimitPolls; ++i) {
        __nanosleep(NS);
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 63u) == 0 && (*abort_flag || global_timer_ns() - t0 > kWaitLimitNs)) return false;
    }
    return false;
}

// Shared-memory descriptors, 128-byte swizzle: low word the address and the
// leading stride, high word the stride between groups of 8 rows (K-major) or of
// 8 k (N-major), one atom of 1024 bytes, version 1, swizzle mode 2. K-major has
// no leading stride (1); N-major operands lie as 64-element rows of N, one row
// a k, and their leading stride is the one between 64-element parts of N.
constexpr uint32_t kDescHi = (1024u >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_lo(uint32_t start, uint32_t leading) { return ((start >> 4) & 0x3FFFu) | leading << 16; }
constexpr uint32_t kIdescNMajorB = 1u << 16, kIdescMinusB = 1u << 14;  // (of the instruction descriptor)

// 32 columns of this warp's 32 lanes, without the wait.
__device__ __forceinline__ void tm_ld32(uint32_t taddr, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr)
        : "memory");
}
// 32 lanes x 16 columns from this warp's 16 registers each.
__device__ __forceinline__ void tc_st16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
// Waits for this thread's tensor-memory loads; the registers pass through it,
// so that nothing reads them earlier.
__device__ __forceinline__ void tm_wait_ld(uint32_t (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                   "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]),
                   "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]),
                   "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]),
                   "+r"(v[30]), "+r"(v[31])
                 :
                 : "memory");
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 32 bytes in one store, or in two where `out` (and with it every row, a multiple
// of 32 bytes) lies only on the 16-byte boundary that the interface asks for: a
// 32-byte store there would fault.
__device__ __forceinline__ void store32(void *p, const uint32_t (&w)[8], bool wide) {
    if (wide)
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                     "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    else {
        uint4 *q = static_cast<uint4 *>(p);
        q[0] = make_uint4(w[0], w[1], w[2], w[3]);
        q[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}
template <int R> __device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R> __device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }

}  // namespace qg
