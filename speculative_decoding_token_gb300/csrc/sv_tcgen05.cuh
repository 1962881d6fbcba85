// sv_tcgen05.cuh -- the fifth-generation tensor core's instructions as the
// tree kernels use them: tensor-memory allocation, loads and stores, matrix
// products with operands in shared memory or tensor memory, tiled copies, and
// their descriptors (PTX ISA, "tcgen05" and "cp.async.bulk.tensor").
#pragma once

#include <cstdint>
#include <cuda.h>

#include "sv_stream.cuh"
#include "sv_tree.h"

namespace sv {

// What a look at a barrier takes that does not open meanwhile (measured: 1.0 us,
// whatever time it is asked to take).
constexpr uint64_t kLookNs = 1000;

// A whole warp's wait, the same outcome for every lane (what follows a wait are
// instructions of whole warps). It gives up after `limit` nanoseconds, or once
// another of the CTA has (`abort`, in shared memory), and the status says so. A
// warp that gave up touches nothing that is shared and arrives at no barrier of
// this kind any more: whoever needs it gives up in turn, and nobody takes for
// done what was not. What a CTA waits for before it exits (its copies and products
// in flight) has the fixed bound of mbar_wait_bounded.
__device__ __forceinline__ bool wait_on(uint64_t &bar, uint32_t parity, int32_t &abort,
                                        int32_t *status, uint64_t limit) {
    constexpr uint32_t all = 0xffffffffu;
    const uint32_t at = smem_u32(&bar);
    if (__all_sync(all, mbar_try_wait(at, parity))) return true;
    const uint64_t t0 = global_ns() - kLookNs;
    while (!__any_sync(all, global_ns() - t0 > limit)) {
        if (__all_sync(all, mbar_try_wait(at, parity))) return true;
        if (__any_sync(all, *(volatile int32_t *)&abort)) return false;
    }
    *(volatile int32_t *)&abort = 1;
    atomicOr(status, SPECVERIFY_STATUS_TIMEOUT);
    return false;
}

// --- tensor memory -----------------------------------------------------------
// One warp; the address of column 0 goes to shared memory at `dst`.
__device__ __forceinline__ void tmem_alloc(uint32_t dst, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}

__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}

__device__ __forceinline__ void tc_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}

__device__ __forceinline__ void tc_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

__device__ __forceinline__ void tmem_wait_ld() {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_wait_st() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// 32 columns of the warp's 32 lanes: r[i] is column i of the thread's lane.
// The warp reads lanes 32 (warp % 4) and up; `addr` carries that lane in its
// upper half. The values are there after tmem_wait_ld.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}

__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}

__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
        "r"(addr)
        : "memory");
}

template <int N>
__device__ __forceinline__ void tmem_ld_n(uint32_t addr, uint32_t *r) {
    static_assert(N == 16 || N == 32, "columns of a load");
    if (N == 32)
        tmem_ld32(addr, r);
    else
        tmem_ld16(addr, r);
}

// --- matrix products ----------------------------------------------------------
// Shared-memory matrix descriptor of a tile in 128-byte rows with the 128-byte
// swizzle, groups of 8 rows 1024 bytes apart. `lead`: for an operand whose
// contiguous dimension is not the summed one, the bytes between its blocks of
// 64 elements (ignored otherwise).
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead) {
    return (uint64_t)((addr & 0x3FFFF) >> 4) | ((uint64_t)(lead >> 4) << 16) |
           ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// Instruction descriptor of kind::f16 with fp32 sums: both operands binary16
// or both bfloat16; A has the summed dimension contiguous, B too unless b_mn.
__host__ __device__ constexpr uint32_t mma_desc(bool fp16, bool b_mn, int m, int n) {
    return (1u << 4) | ((fp16 ? 0u : 1u) << 7) | ((fp16 ? 0u : 1u) << 10) |
           ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// Whether this lane is the one that issues its warp's products. The warp runs
// the issuing code as a whole, so that descriptors stay in uniform registers;
// code under `if (lane == 0)` takes about 100 cycles a product instead of 64.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}

// D (tensor memory) = A B (+ D), 16 steps of the summed dimension, issued by
// the lane whose `on` is set.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, bool add,
                                       bool on) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(desc), "r"((uint32_t)add), "r"((uint32_t)on)
        : "memory");
}

// The same with A in tensor memory, two elements a column.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t desc, bool add,
                                       bool on) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(desc), "r"((uint32_t)add), "r"((uint32_t)on)
        : "memory");
}

// One arrival on `bar` once every product that the lane issued has completed.
__device__ __forceinline__ void mma_commit(uint32_t bar, bool on) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
            bar),
        "r"((uint32_t)on)
        : "memory");
}

// --- tiled copies ---------------------------------------------------------------
// A box of a [page][head][token][element] map, first element `x` (a multiple of 8).
__device__ __forceinline__ void tile_load(uint32_t dst, const CUtensorMap *map, int x, int token,
                                          int head, int page, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(map), "r"(x), "r"(token), "r"(head), "r"(page), "r"(bar)
        : "memory");
}

// Generic writes to shared memory before, asynchronous reads of it after.
__device__ __forceinline__ void fence_async_smem() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ void mbar_fence_init() {
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

// --- host: maps of a cache's keys or values --------------------------------------
constexpr int kTile = kTileSlots;  // of a tile, and its rows of 128 bytes

// Tokens of one copy: the largest power of two that divides the page size and a tile.
int cache_box(int page);

// A [page][head][token][element] map in boxes of 64 elements by `box` tokens;
// false where the layout cannot be described.
bool cache_map(const CacheParams &c, const char *base, int box, CUtensorMap *map);

}  // namespace sv
