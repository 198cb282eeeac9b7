// tensor.cuh -- PTX wrappers of the attention kernel: mbarriers with bounded
// waits, TMA tile loads, tcgen05 products and TMEM accesses, and the
// shared-memory matrix descriptors.  Not a public header.
#pragma once

#include <cuda.h>

#include <cstdint>

namespace specv {

__device__ __forceinline__ uint32_t smem_addr(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// ------------------------------------------------------------- mbarriers

__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count));
}

__device__ __forceinline__ void bar_arrive(uint32_t bar, uint32_t count = 1) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void bar_arrive_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

constexpr uint32_t kTries = 1u << 21;  // a wait gives up after this many (each may suspend): seconds

// Waits for the phase `parity`; false when the tries ran out: *dead is set and
// the caller leaves its loops (others then run out of theirs).  The loop is one
// asm statement: the thread that issues the products is bound by its own
// instructions, and this is most of what it does.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int *dead) {
    uint32_t tries;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mov.u32 %0, 0;\n"
        "AGAIN:\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "@p bra DONE;\n\t"
        "add.u32 %0, %0, 1;\n\t"
        "setp.lt.u32 p, %0, %3;\n\t"
        "@p bra AGAIN;\n"
        "DONE:\n\t}"
        : "=&r"(tries)
        : "r"(bar), "r"(parity), "n"(kTries)
        : "memory");
    if (tries < kTries) return true;
    *dead = 1;
    return false;
}

// The same without the flag.
__device__ __forceinline__ void bar_drain(uint32_t bar, uint32_t parity) {
    for (uint32_t i = 0; i < kTries && !bar_try(bar, parity); ++i) {
    }
}

// True in one lane of a converged warp.  Code under it counts as one thread's
// to the compiler, which then keeps descriptors in uniform registers: under
// `lane == 0` a product took over 100 cycles to issue.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

// `threads` threads, whole warps, meet at hardware barrier `id`; whether any of
// them came with x.
__device__ __forceinline__ bool any_of(int id, int threads, bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.aligned.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(x ? 1u : 0u), "r"(id), "r"(threads)
        : "memory");
    return r != 0;
}

// Generic-proxy writes to shared memory, made visible to TMA and the tensor cores.
__device__ __forceinline__ void fence_async_proxy() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// ------------------------------------------------------------------ TMA

__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap *map, uint32_t bar, int x,
                                         int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// Four bytes (zeros where not `on`), and their arrival at `bar` once this
// thread's copies so far are there (the barrier's count includes it).
__device__ __forceinline__ void copy4(uint32_t dst, const void *src, bool on) {
    asm volatile("cp.async.ca.shared::cta.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(on ? 4u : 0u) : "memory");
}

__device__ __forceinline__ void copies_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// -------------------------------------------------------------- tcgen05

__device__ __forceinline__ void tmem_alloc(uint32_t where, uint32_t columns) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(where),
                 "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_free(uint32_t base, uint32_t columns) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(columns)
                 : "memory");
}

__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                     bar)
                 : "memory");
}

__device__ __forceinline__ void fence_before_sync() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}

__device__ __forceinline__ void fence_after_sync() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// D[tmem] (+)= A B with A and B in shared memory.  F8: both
// operands e4m3, 32 deep; else both bf16, 16 deep.  A matrix descriptor comes
// as its low word (which moves along the matrix) and its high word.
template <bool F8>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t a_hi, uint32_t b, uint32_t b_hi,
                                       uint32_t idesc, bool add) {
    if (F8)
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.u32 p, %6, 0;\n\t"
            "mov.b64 x, {%1, %2};\n\tmov.b64 y, {%3, %4};\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %5, p;\n\t}" ::"r"(d),
            "r"(a), "r"(a_hi), "r"(b), "r"(b_hi), "r"(idesc), "r"(add ? 1u : 0u));
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.u32 p, %6, 0;\n\t"
            "mov.b64 x, {%1, %2};\n\tmov.b64 y, {%3, %4};\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %5, p;\n\t}" ::"r"(d),
            "r"(a), "r"(a_hi), "r"(b), "r"(b_hi), "r"(idesc), "r"(add ? 1u : 0u));
}

// Both bf16, A in TMEM.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t b_hi, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tsetp.ne.u32 p, %5, 0;\n\tmov.b64 y, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(b_hi), "r"(idesc), "r"(add ? 1u : 0u));
}

// 32 consecutive TMEM columns of this thread's lane (a warp reads its own 32
// lanes); complete after tmem_load_wait.
__device__ __forceinline__ void tmem_load32(uint32_t addr, float *v) {
    uint32_t *r = reinterpret_cast<uint32_t *>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr)
        : "memory");
}

__device__ __forceinline__ void tmem_store32(uint32_t addr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
        "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
        "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

__device__ __forceinline__ void tmem_load16(uint32_t addr, float *v) {
    uint32_t *r = reinterpret_cast<uint32_t *>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr)
        : "memory");
}

__device__ __forceinline__ void tmem_store16(uint32_t addr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void tmem_load_wait() {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_store_wait() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Shared-memory matrix descriptor of rows of `kRow` bytes (128, 64 or 32), each
// swizzled over its whole width, eight rows to a pattern: the low word holds
// the address and `lead`, the bytes between column blocks of kRow bytes where
// the matrix's columns are taken along memory and there is more than one.
__device__ __forceinline__ uint32_t matrix_lo(uint32_t addr, uint32_t lead) { return addr >> 4 | (lead >> 4) << 16; }

template <int kRow>
constexpr uint32_t kMatrixHi = static_cast<uint32_t>((8 * kRow) >> 4) | 1u << 14 |
                               (kRow == 128 ? 2u : kRow == 64 ? 4u : 6u) << 29;

// Byte offset of (row, byte) in such a matrix: 16-byte units are permuted
// within a row by the row's place in its pattern of eight rows.
template <int kRow>
__device__ __forceinline__ uint32_t swizzled(uint32_t row, uint32_t byte) {
    static_assert(kRow == 128 || kRow == 64 || kRow == 32, "swizzled rows");
    const uint32_t o = row * kRow + byte;
    return o ^ ((o >> 7 & (kRow / 16 - 1)) << 4);
}

// Instruction descriptor: fp32 accumulators, M = 128, N = n columns, both
// operands of one type (bf16, or e4m3); a_along / b_along: the operand's M or N
// runs along memory (else its K does).
__host__ __device__ constexpr uint32_t mma_desc(bool f8, int n, bool a_along, bool b_along) {
    return 1u << 4 | (f8 ? 0u : 1u << 7 | 1u << 10) | (a_along ? 1u << 15 : 0u) | (b_along ? 1u << 16 : 0u) |
           static_cast<uint32_t>(n >> 3) << 17 | (128u >> 4) << 24;
}

}  // namespace specv
