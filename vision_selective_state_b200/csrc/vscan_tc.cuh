// 5th-generation tensor core (tcgen05) building blocks: tensor memory, products with
// the left operand in tensor memory and the right one in swizzled shared memory,
// and waits that give up instead of hanging.
//
// Shared-memory tiles are 64 rows of 64 bf16 (128 bytes a row), with the 16-byte
// pieces of row r exchanged by r mod 8 (the 128-byte swizzle); a wider tile is
// several of them, one after the other. Read with the row index as the product's
// column (K-major) or with the row index as its summed index (MN-major), the same
// tile serves as B and as its transpose.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace vscan {

constexpr int TC_TILE = 64 * 128;  // bytes of a 64 x 64 tile

// Byte offset of 16-byte piece c of row r in a tile (c < 8), or in a row of tiles.
__device__ __forceinline__ int tc_swizzle(int r, int c) { return (c >> 3) * TC_TILE + r * 128 + (((c & 7) ^ (r & 7)) << 4); }

// Descriptor of a tile: start address, 1024 bytes from one group of eight rows to
// the next, 128-byte swizzle. A product sums 16 at a time: a K-major tile steps 32
// bytes, an MN-major one 16 rows = 2048 bytes.
__device__ __forceinline__ uint64_t tc_desc(uint32_t smem)
{
    return (uint64_t)((smem >> 4) & 0x3fff) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
           (uint64_t)2 << 61;
}

// Instruction descriptor: bf16 x bf16 into float32, 128 rows, n columns.
__host__ __device__ constexpr uint32_t tc_idesc(int n, bool b_mn_major)
{
    return 1u << 4 | 1u << 7 | 1u << 10 | (b_mn_major ? 1u << 16 : 0u) | (uint32_t)(n >> 3) << 17 | (128u >> 4) << 24;
}

// One lane of a converged warp. A branch on this predicate keeps the operands of the
// products in uniform registers: a 64-column product then issues in its 32 cycles, behind a
// branch on the thread index it took 47.
__device__ __forceinline__ bool tc_elect()
{
    uint32_t p;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.b32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0;
}

// d[128][n] (+)= a[128][16] b[16][n]; d and a are tensor-memory addresses. One thread.
__device__ __forceinline__ void tc_mma(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile("{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d), "r"(a), "l"(b), "r"(idesc),
                 "r"((uint32_t)add)
                 : "memory");
}

// The same with the left operand in shared memory, in the right one's form.
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile("{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
                 "r"((uint32_t)add)
                 : "memory");
}

// The barrier completes when all products issued so far by this thread have.
__device__ __forceinline__ void tc_commit(uint32_t mbar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(mbar) : "memory");
}

__device__ __forceinline__ void tc_alloc(uint32_t smem_out)  // one warp; all 512 columns
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(smem_out) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
}
// At the end of a kernel, by one warp, behind a barrier of the block. Where a wait gave up, products and copies
// into shared memory may still be on their way: they get a millisecond to end before the block gives its memory back.
__device__ __forceinline__ void tc_free(uint32_t addr, const volatile int* dead)
{
    if (*dead)
#pragma unroll 1
        for (int i = 0; i < 1000; ++i) __nanosleep(1000);
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(addr));
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }
// Shared memory written by ordinary stores and copies, seen by the tensor core.
__device__ __forceinline__ void tc_fence_smem() { asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory"); }

// This warp's 32 rows, 32 (16) neighbouring columns: one row a lane.
__device__ __forceinline__ void tc_ld32(uint32_t addr, float* v)
{
    uint32_t* r = reinterpret_cast<uint32_t*>(v);
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
                   "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
                   "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(addr));
}
__device__ __forceinline__ void tc_ld16(uint32_t addr, float* v)
{
    uint32_t* r = reinterpret_cast<uint32_t*>(v);
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(addr));
}
__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t* r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(addr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
                 "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
                 : "memory");
}

// ---- launches that follow one another ------------------------------------------------
// A call's kernels each start while the one before ends (launch_after): start_next lets the next
// one's blocks come as soon as all of this one's have got that far, and wait_previous, which
// every block executes before it reads what the one before wrote or returns, waits for its end.
__device__ __forceinline__ void start_next() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }
__device__ __forceinline__ void wait_previous() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }

// ---- barriers ------------------------------------------------------------------------
__device__ __forceinline__ void mbar_init(uint32_t mbar, int count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(mbar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_fence_init() { asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory"); }
__device__ __forceinline__ bool mbar_test(uint32_t mbar, uint32_t parity)
{
    uint32_t done;
    asm volatile("{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000;\nselp.b32 %0, 1, 0, p;\n}\n"
                 : "=r"(done) : "r"(mbar), "r"(parity) : "memory");
    return done != 0;
}
// 16 bytes into shared memory, or zeros. (The copy with a source size in a register has to be
// ready for any size.)
__device__ __forceinline__ void copy16(void* smem, const void* gmem, bool valid)
{
    asm volatile("{\n.reg .pred p;\nsetp.eq.b32 p, %2, 0;\ncp.async.cg.shared.global [%0], [%1], 16, p;\n}\n" ::"r"(
                     static_cast<unsigned>(__cvta_generic_to_shared(smem))), "l"(gmem), "r"((int)valid));
}

// Copies by the bulk engine: 16-byte aligned, a multiple of 16 bytes, counted by a barrier.
__device__ __forceinline__ void mbar_expect(uint32_t mbar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(mbar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_in(uint32_t smem, const void* gmem, uint32_t bytes, uint32_t mbar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(smem), "l"(gmem),
                 "r"(bytes), "r"(mbar) : "memory");
}
__device__ __forceinline__ void bulk_out(void* gmem, const void* smem, uint32_t bytes)
{
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\n" ::"l"(gmem),
                 "r"(static_cast<uint32_t>(__cvta_generic_to_shared(smem))), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_out_read()  // this thread's copies have read shared memory
{
    asm volatile("cp.async.bulk.commit_group;\ncp.async.bulk.wait_group.read 0;\n" ::: "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t mbar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(mbar) : "memory");
}
// Named barriers: some threads only arrive, the others wait for them.
__device__ __forceinline__ void bar_arrive(int id, int threads) { asm volatile("bar.arrive %0, %1;\n" ::"r"(id), "r"(threads) : "memory"); }
__device__ __forceinline__ void bar_sync(int id, int threads) { asm volatile("bar.sync %0, %1;\n" ::"r"(id), "r"(threads) : "memory"); }
// Tries until `ready` says so, TC_WAIT_TRIES times at most. Then `dead` is set: the CTA's other waits give
// up within 256 tries, every later one after its first, and the kernel runs to its end with invalid
// results instead of hanging.
constexpr int TC_WAIT_TRIES = 1 << 20;
template <typename READY>
__host__ __device__ __forceinline__ void tc_bounded_wait(READY ready, volatile int* dead)
{
    int i = 0;
    while (i < TC_WAIT_TRIES && !ready())  // looks at `dead` after the first try and every 256th
        i = (i & 255) == 0 && *dead ? TC_WAIT_TRIES : i + 1;
    if (i == TC_WAIT_TRIES) *dead = 1;
}
// Wait for a phase, at most about a second in all: each try sleeps for up to 1000 ns.
__device__ __forceinline__ void mbar_wait(uint32_t mbar, uint32_t parity, volatile int* dead)
{
    tc_bounded_wait([&] { return mbar_test(mbar, parity); }, dead);
    __syncwarp();
}

}  // namespace vscan
