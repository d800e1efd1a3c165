// tcgen05.cuh -- inline-PTX wrappers of sm_103a's fifth-generation tensor cores as the attention
// kernels use them: tensor memory, matrix products of 16-bit elements into fp32, their operand
// descriptors, and moves between tensor memory and registers.
//
// Tensor memory has 128 lanes (accumulator rows) of 512 32-bit columns an SM; an address holds
// the lane in its upper half and the column in its lower one, and warp w of a warpgroup reaches
// lanes 32 w .. 32 w + 31 only. Operands in shared memory are tiles of 64 elements (128 bytes) by
// any number of rows, as a tensor map with the 128-byte swizzle lands them: the 16-byte word c of
// row r sits at word c ^ (r mod 8) of that row, tiles start on 1,024-byte boundaries.
#pragma once
#include <cstdint>

#include "ptx.cuh"

namespace uly {

constexpr int kTmemColumns = 512;

// True in one lane of a converged warp, the same one every time. Products, their commits and tensor
// copies are issued behind it: the compiler then knows that a single lane runs and keeps their
// operands in uniform registers (behind `lane == 0` each product took about 100 cycles to issue).
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(p));
    return p != 0;
}

// One warp allocates all of an SM's tensor memory; the base address arrives in shared memory.
__device__ __forceinline__ void tmem_alloc(uint32_t* where)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(where)),
                 "n"(kTmemColumns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_free(uint32_t base)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base),
                 "n"(kTmemColumns)
                 : "memory");
}

// Order this thread's tensor-memory work before (after) a barrier that it passes next (has passed).
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// An arrival on `bar` once every product this thread has issued so far is complete.
__device__ __forceinline__ void tc_commit(uint64_t* bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                     smem_u32(bar))
                 : "memory");
}

// Instruction descriptor: fp32 accumulator of 128 rows x n columns, A and B both bf16 or both
// fp16; b_mn: B's rows in shared memory run along K (its columns, N, are contiguous).
__host__ __device__ constexpr uint32_t tc_idesc(bool f16, int n, bool b_mn)
{
    return (1u << 4) | (f16 ? 0u : (1u << 7) | (1u << 10)) | (b_mn ? 1u << 16 : 0u) |
           (uint32_t(n >> 3) << 17) | (uint32_t(128 >> 4) << 24);
}

constexpr uint64_t kDescSwizzle128 = (uint64_t(2) << 61) | (uint64_t(1) << 46);

// Shared-memory operand whose rows are contiguous along K (64 elements a tile row): eight rows
// every 1,024 bytes. A step of 16 elements along K is 32 bytes, four steps a tile.
__device__ __forceinline__ uint64_t tc_desc_k(uint32_t addr)
{
    return kDescSwizzle128 | (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 16) |
           uint64_t((addr >> 4) & 0x3FFF);
}

// Shared-memory operand whose rows run along K: 64 columns of N contiguous, the next 64 at
// `tile_bytes`; eight rows of K every 1,024 bytes. A step of 16 along K is 2,048 bytes.
__device__ __forceinline__ uint64_t tc_desc_mn(uint32_t addr, uint32_t tile_bytes)
{
    return kDescSwizzle128 | (uint64_t(1024 >> 4) << 32) | (uint64_t(tile_bytes >> 4) << 16) |
           uint64_t((addr >> 4) & 0x3FFF);
}

// D[tmem] (+)= A[smem] B[smem], one step of 16 along K, by one thread.
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          bool accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u)
        : "memory");
}

// The same with A in tensor memory (two 16-bit elements a column: 8 columns a step).
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                          bool accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u)
        : "memory");
}

// 32 consecutive columns of this thread's lane. The values are there after tmem_wait_ld, which
// takes the registers so that no use of them moves ahead of it.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32])
{
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

// The same for 16 columns.
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}

__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[16])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                   "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                   "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}

__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                   "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                   "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                   "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                   "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                   "+r"(r[30]), "+r"(r[31])::"memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32])
{
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

__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The largest of three in one instruction.
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

// Registers a thread from here on, for every warp of a warpgroup (the shares of all warpgroups
// add up to what the block was launched with).
template <int N>
__device__ __forceinline__ void regs_grow()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

template <int N>
__device__ __forceinline__ void regs_shrink()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Asks for the place of a CTA of this launch that has not started yet; its answer (16 bytes at
// `answer`, 16-byte aligned) is counted on `bar`. Not to be called again after a refusal.
__device__ __forceinline__ void steal_cta(void* answer, uint64_t* bar)
{
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::
            "r"(smem_u32(answer)),
        "r"(smem_u32(bar))
        : "memory");
}

// The stolen CTA's blockIdx.x, or -1 when none was left.
__device__ __forceinline__ int64_t stolen_cta(const void* answer)
{
    uint32_t x, got;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b128 a;\n\tld.shared.b128 a, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n\t"
        "selp.u32 %1, 1, 0, p;\n\tmov.u32 %0, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, a;\n\t}"
        : "=r"(x), "=r"(got)
        : "r"(smem_u32(answer))
        : "memory");
    return got ? int64_t(x) : -1;
}

// Programmatic launches: what comes before this kernel in its stream (and launched it early) is
// complete and its writes are visible; the kernel behind it may start where there is room.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// A kernel that started early and has not waited yet may see only what it acquires: a word that the
// kernel in front of it released after its own wait, which carries everything that one had seen.
__device__ __forceinline__ void release_word(uint32_t* p, uint32_t v)
{
    asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t acquire_word(const uint32_t* p)
{
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
// Orders earlier ordinary accesses to global memory before later tensor and bulk copies of it.
__device__ __forceinline__ void fence_proxy_async_global() { asm volatile("fence.proxy.async.global;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// 2^x (subnormal results flushed to zero).
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// How the warps of a CTA give up: together, and only when nothing moves. One warp, which works the units
// out and stays until the others are done, watches: its own waits run out once the loading warp's count
// has not gone on for `limit_us`, so that it does not matter how long a unit is or how many units without
// work come one after the other. Every other wait ends with it. (There are dozens of them: a clock and
// a count in each made units of few key blocks 9 % slower.)
struct CtaLife {
    int dead;           // a wait has run out: every warp finishes what it has in flight and ends
    int stuck;          // a copy in flight did not land either
    uint32_t loads;     // copies issued
    uint32_t limit_us;  // 0: whatever is not there at the second look has run out (self-test)
    uint64_t done;      // barrier: the other warps
};

__device__ __forceinline__ void life_init(CtaLife& l, uint32_t limit_us, int warps)
{
    l.dead = l.stuck = 0;
    l.loads = 0;
    l.limit_us = limit_us;
    mbar_init(&l.done, warps - 1);
}

// Bits of the status word that a CTA's end leaves.
__device__ __forceinline__ unsigned life_status(const CtaLife& l)
{
    return (l.dead ? kStatusWaitTimeout : 0u) | (l.stuck ? kStatusDrainTimeout : 0u);
}

// A wait inside such a CTA: false once the CTA has given up. A waiting thread is parked by the hardware
// (up to 10 us at a time) instead of polling: the warps at work need the issue slots. (The first try
// apart from the loop: as one loop, 75,600 tokens x 8 heads of 128 took 16.1 ms in place of 13.8.)
__device__ __forceinline__ bool wait_or_dead(uint64_t* bar, uint32_t parity, volatile CtaLife* life)
{
    if (mbar_try_wait_hint<10000>(bar, parity)) return true;
    while (!mbar_try_wait_hint<10000>(bar, parity)) {
        if (life->dead) return false;
    }
    return true;
}

// The same by the warp that watches.
__device__ __forceinline__ bool wait_watching(uint64_t* bar, uint32_t parity, volatile CtaLife* life)
{
    if (mbar_try_wait_hint<10000>(bar, parity)) return true;
    uint64_t t0 = global_timer_ns();
    uint32_t moved = life->loads;
    while (!mbar_try_wait_hint<10000>(bar, parity)) {
        const uint64_t limit = uint64_t(life->limit_us) * 1000u, now = global_timer_ns();
        const uint32_t at = life->loads;
        if (at != moved && limit > 0) {
            moved = at;
            t0 = now;
        } else if (now - t0 >= limit) {
            life->dead = 1;
        }
        if (life->dead) return false;
    }
    return true;
}

// A warp's end: the watching one waits for the others.
__device__ __forceinline__ void life_end(CtaLife& l, bool watching)
{
    __syncwarp();
    if (watching)
        wait_watching(&l.done, 0, &l);
    else if ((threadIdx.x & 31) == 0)
        mbar_arrive(&l.done);
}

}  // namespace uly
