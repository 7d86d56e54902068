// tensor.cuh -- the pieces of sm_103a that the attention kernels are built from:
// barriers in shared memory, bulk tensor copies, tensor-core products with
// operands in shared or tensor memory, and tensor memory itself.
//
// Operand tiles.  A tile is rows of 64 elements (128 bytes) in the 128-byte
// swizzle, 8 rows to a 1 KB atom; wider rows are several such blocks one behind
// the other.  The same tile serves as an operand whose contraction runs along
// the row (major_k: 32 bytes further per 16 elements) and as one whose
// contraction runs across the rows (major_mn: 2 KB further per 16 rows).
#pragma once

#include <cuda.h>

#include <type_traits>

#include "decoder.cuh"

namespace gsr {

constexpr int kBlockBytes = 128 * 128;   // 128 rows of 64 16-bit elements

__device__ __forceinline__ uint32_t smem_address(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t pred;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(pred));
    return pred != 0;
}

// ---- barriers -----------------------------------------------------------------

__device__ __forceinline__ void barrier_init(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void barrier_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void barrier_expect(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ bool barrier_try(uint32_t bar, uint32_t parity)
{
    uint32_t done;
    asm volatile(
        "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}

// Waits end: one that has run for kWaitCycles (seconds; a step takes
// microseconds) marks the block as aborted and reports to the host's status
// word, and every later wait of the block returns at once: the copying thread
// then stops (its barriers could not count copies that nothing waits for), the
// others run through the rest of their loops, and the results are not valid.  The
// context's next call of a decoder operator or gsr_synchronize says so.
constexpr long long kWaitCycles = 4000000000ll;

struct WaitGuard {
    volatile uint32_t *aborted;   // shared
    uint32_t *status;             // the context's status word (host memory)

    __device__ __forceinline__ bool stop() const { return *aborted != 0; }
};

__device__ __forceinline__ void barrier_wait(uint32_t bar, uint32_t parity, const WaitGuard &g)
{
    if (barrier_try(bar, parity)) return;
    const long long start = clock64();
    while (!barrier_try(bar, parity)) {
        if (*g.aborted) return;
        if (clock64() - start > kWaitCycles) {
            *g.aborted = 1;
            *(volatile uint32_t *)g.status = 1;
            return;
        }
    }
}

// The same for a whole warp, which leaves it converged: its lanes may see the
// barrier turn at different tries, and warp-wide instructions on tensor memory or
// matrix fragments are undefined for lanes that have come apart.  So may a lane
// fall two phases behind, and wait for one that has gone.
__device__ __forceinline__ void barrier_wait_warp(uint32_t bar, uint32_t parity, const WaitGuard &g)
{
    barrier_wait(bar, parity, g);
    __syncwarp();
}

// At the end of an aborted block: time for copies and products in flight to land
// before its shared memory is given to another block.
__device__ __forceinline__ void drain_if_aborted(const WaitGuard &g)
{
    if (!*g.aborted) return;
    const long long start = clock64();
    while (clock64() - start < 20000000ll) {
    }
}

// ---- copies ----------------------------------------------------------------------

// The box at (x, row, head, item) of a [item, head, row, x] tensor map into
// shared memory; elements outside the tensor arrive as zeros.
__device__ __forceinline__ void copy_box(uint32_t to, const CUtensorMap *map, uint32_t bar, int x, int row, int head,
                                         int item)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], "
        "[%2];" ::"r"(to),
        "l"(map), "r"(bar), "r"(x), "r"(row), "r"(head), "r"(item)
        : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// Makes this thread's ordinary writes to shared memory visible to copies and products.
__device__ __forceinline__ void fence_async()
{
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// ---- tensor memory ------------------------------------------------------------------

__device__ __forceinline__ void tmem_alloc(uint32_t to, uint32_t columns)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(to), "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_free(uint32_t base, uint32_t columns)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(columns) : "memory");
}

__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// (The registers of a load hold their values only behind this wait: `pin` keeps
// their uses there.)
__device__ __forceinline__ void tmem_wait_load() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void pin(uint32_t (&r)[32])
{
#pragma unroll
    for (int i = 0; i < 32; i += 8)
        asm volatile(""
                     : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                       "+r"(r[i + 6]), "+r"(r[i + 7]));
}

// 32 columns of the calling thread's lane.
__device__ __forceinline__ void tmem_load32(uint32_t (&r)[32], uint32_t at)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(at)
        : "memory");
}

__device__ __forceinline__ void tmem_store32(uint32_t at, const uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
        "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
        "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(at)
        : "memory");
}

// ---- products -------------------------------------------------------------------------

// Shared-memory operand descriptors (128-byte swizzle, 8-row atoms 1 KB apart).
// The low word holds the address, which alone changes from one to the next, and
// the distance of blocks of 64 along the free dimension (for a contraction
// across the rows; 1 where there is none), both in units of 16 bytes.
constexpr uint32_t kOperandHigh = (1u << 14) | (2u << 29) | (1024 >> 4);

__device__ __forceinline__ uint32_t operand_rows(uint32_t address) { return (1u << 16) | (address >> 4); }

__device__ __forceinline__ uint32_t operand_across(uint32_t address)
{
    return ((uint32_t)(kBlockBytes >> 4) << 16) | (address >> 4);
}

// Instruction descriptor: f32 sums of 16-bit operands of one type, M = 128.
template <typename T>
__device__ __forceinline__ uint32_t product_form(int n, bool b_major_mn)
{
    constexpr uint32_t kType = sizeof(T) == 2 && std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
    return (1u << 4) | (kType << 7) | (kType << 10) | ((b_major_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
           ((128u >> 4) << 24);
}

// d (128 x n, tensor memory) = a b (+ d), one instruction's 16 terms.  Called by a
// whole converged warp, issued by its leader.
__device__ __forceinline__ void product_ss(bool leader, uint32_t d, uint32_t a, uint32_t b, uint32_t form, bool add)
{
    asm volatile(
        "{\n.reg .pred p, q;\n.reg .b64 a, b;\nsetp.ne.u32 p, %4, 0;\nsetp.ne.u32 q, %5, 0;\n"
        "mov.b64 a, {%1, %6};\nmov.b64 b, {%2, %6};\n"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(form), "r"((uint32_t)add), "r"((uint32_t)leader), "n"(kOperandHigh)
        : "memory");
}

__device__ __forceinline__ void product_ts(bool leader, uint32_t d, uint32_t a, uint32_t b, uint32_t form, bool add)
{
    asm volatile(
        "{\n.reg .pred p, q;\n.reg .b64 b;\nsetp.ne.u32 p, %4, 0;\nsetp.ne.u32 q, %5, 0;\n"
        "mov.b64 b, {%2, %6};\n"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n}\n" ::"r"(d),
        "r"(a), "r"(b), "r"(form), "r"((uint32_t)add), "r"((uint32_t)leader), "n"(kOperandHigh)
        : "memory");
}

// Arrives on the barrier once every product the leader has issued is complete.
__device__ __forceinline__ void product_commit(bool leader, uint32_t bar)
{
    asm volatile(
        "{\n.reg .pred q;\nsetp.ne.u32 q, %1, 0;\n"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar),
        "r"((uint32_t)leader)
        : "memory");
}

// d = a b^T over `steps` x 16 elements along both tiles' rows of a (128 rows) and b.
template <int HD>
__device__ __forceinline__ void product_rows(bool leader, uint32_t d, uint32_t a, uint32_t b, uint32_t form, int steps)
{
    const uint32_t a0 = operand_rows(a), b0 = operand_rows(b);
    if (steps == HD / 16) {
#pragma unroll
        for (int k = 0; k < HD / 16; ++k) {
            const uint32_t at = ((k >> 2) * kBlockBytes + (k & 3) * 32) >> 4;
            product_ss(leader, d, a0 + at, b0 + at, form, k != 0);
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < HD / 16; ++k) {
        const uint32_t at = ((k >> 2) * kBlockBytes + (k & 3) * 32) >> 4;
        if (k < steps) product_ss(leader, d, a0 + at, b0 + at, form, k != 0);
    }
}

// d (+)= a b with a (128 rows, 16-bit pairs in tensor memory) against the 128
// rows of tile b.  a's 128 terms lie in `groups` runs, each at the start of its
// own 128 / groups columns (1: one run of 64 columns).  (Fewer steps for a tile's
// tail made every product's issue slower: 184 us where these take 165.)
__device__ __forceinline__ void product_across(bool leader, uint32_t d, uint32_t a, uint32_t b, uint32_t form, bool add,
                                               int groups = 1)
{
    const uint32_t b0 = operand_across(b);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int each = 8 / groups;
        product_ts(leader, d, a + k / each * (128 / groups) + k % each * 8, b0 + (k * 2048 >> 4), form, add || k != 0);
    }
}

// ---- registers ------------------------------------------------------------------------------

// A block has two warpgroups that compute, each thread with a row of scores or half
// of one, and one whose warps copy and issue products and give most of their
// registers to the others.
constexpr int kStartRegisters = 168, kFewRegisters = 72, kManyRegisters = 216;
static_assert(kFewRegisters + 2 * kManyRegisters <= 3 * kStartRegisters, "the shares must fit what the block starts with");

__device__ __forceinline__ void give_registers()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegisters));
}

__device__ __forceinline__ void take_registers()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kManyRegisters));
}

// ---- host ------------------------------------------------------------------------------------

// Tensor map of a [batch, tokens, heads, dim] array for boxes of 64 elements of
// `rows` tokens of one head.  A stride of 0 (one array for all items or heads)
// becomes an extent of 1; the kernels multiply such a coordinate by 0.
// (A kernel compiled to start with fewer registers than the shares add up to
// would wait for them forever: refuse to launch it.)
int check_registers(gsr_ctx *ctx, const void *kernel, const char *name);
int heads_map(gsr_ctx *ctx, CUtensorMap *map, const gsr_heads &t, int dtype, int64_t batch, int64_t tokens,
              int64_t heads, int dim, int rows);

}  // namespace gsr
