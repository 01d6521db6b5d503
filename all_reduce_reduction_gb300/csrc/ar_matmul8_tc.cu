// The E4M3 product on the tensor cores (tcgen05), operands by TMA.
//
// A scale belongs to 128 elements along k, so the tensor core can sum one such
// block only: 128 x N x 128 products go to an accumulator in tensor memory,
// and the epilogue warps read it back, multiply it with sa * sb and add it to
// binary32 sums in their registers, while the tensor core fills the next
// accumulator.
//
// Two forms.  k_matmul8_rows puts rows of a on the accumulator's lanes, 256 for a
// pair of CTAs, and 256 rows of b on its columns: a thread's row scale is then
// one register.  k_matmul8_few is for few rows per group: 128 rows of b on the
// lanes, 16 to 64 rows of a on the columns, several CTAs of a cluster along k;
// it streams the weights once with all SMs even when there is one row.
//
// Every wait is bounded: past kWaitNs it writes AR_ERR_TIMEOUT to the caller's
// status word and the CTA's roles all leave.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>

#include "ar_cluster.cuh"
#include "ar_matmul8.cuh"

namespace ar {
namespace {

constexpr uint64_t kWaitNs = 2000000000ull;

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" :: "r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;"
                 :: "r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" :: "r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
// Bounded wait for the phase of this parity; false if this wait ran out or
// another role of the CTA gave up.  Called after a first try.
__device__ __noinline__ bool mbar_wait_slow(uint32_t bar, uint32_t parity, volatile int *abort,
                                            int *status) {
    uint64_t deadline = 0;
    for (uint32_t tries = 1;; ++tries) {
        if (mbar_test(bar, parity))
            return true;
        if (*abort)
            return false;
        const uint64_t now = globaltimer_ns();
        if (deadline == 0)
            deadline = now + kWaitNs;
        if (now > deadline) {
            if (status)
                record_error(status, AR_ERR_TIMEOUT);
            *abort = 1;
            return false;
        }
    }
}
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int *abort,
                                          int *status) {
    return mbar_test(bar, parity) || mbar_wait_slow(bar, parity, abort, status);
}

// The same by a whole warp, all lanes with one answer.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *abort,
                                          int *status) {
    if (__all_sync(0xFFFFFFFFu, mbar_test(bar, parity)))
        return true;
    return __all_sync(0xFFFFFFFFu, mbar_wait_slow(bar, parity, abort, status));
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok));
    return ok != 0;
}

// After an abort only: bounded waits until what is in flight has ended, so that
// nothing touches the CTA's memory after it has left.  `issued` loads over
// `stages` stages; products through the barrier `drain`, which nothing else uses.
__device__ __forceinline__ void mbar_drain(uint32_t bar, uint32_t parity) {
    const uint64_t deadline = globaltimer_ns() + kWaitNs;
    while (!mbar_test(bar, parity) && globaltimer_ns() < deadline) {
    }
}
__device__ __forceinline__ void drain_loads(uint32_t full, uint32_t issued, uint32_t stages) {
    for (uint32_t k = issued < stages ? 0 : issued - stages; k < issued; ++k)
        mbar_drain(full + 8 * (k % stages), (k / stages) & 1);
}

// The same where the loads are counted by a barrier of the other CTA, which this one
// cannot wait on: far longer than any load takes.
__device__ __forceinline__ void linger() {
    const uint64_t deadline = globaltimer_ns() + 1000000ull;
    while (globaltimer_ns() < deadline) {
    }
}

// Tile of a tensor map into shared memory; x is a byte offset along k, a
// multiple of 128.
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap *map, int x, int y,
                                       uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];"
        :: "r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
}
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z,
                                       uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];"
        :: "r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}

// The same for a CTA of a pair, the bytes counted by a barrier of either CTA.
__device__ __forceinline__ void tma_pair_2d(uint32_t dst, const CUtensorMap *map, int x, int y,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];"
        :: "r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
}
__device__ __forceinline__ void tma_pair_3d(uint32_t dst, const CUtensorMap *map, int x, int y,
                                            int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];"
        :: "r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}

// Arrival at a barrier of either CTA.  It hands over tensor memory that has been
// read, which tcgen05.fence orders; nothing in ordinary memory goes with it, so
// it needs no wider release (at cluster scope that doubled the kernel's time).
__device__ __forceinline__ void mbar_arrive_peer(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" :: "r"(bar) : "memory");
}

// ---- tcgen05 -------------------------------------------------------------------

// PAIR: the two CTAs of a cluster work on one accumulator tile (cta_group::2);
// one warp of each allocates and frees.
template <int COLS, bool PAIR> __device__ __forceinline__ void tmem_alloc(uint32_t *slot) {
    if (PAIR) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                     :: "r"(smem_addr(slot)), "n"(COLS) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     :: "r"(smem_addr(slot)), "n"(COLS) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
}
template <int COLS, bool PAIR> __device__ __forceinline__ void tmem_free(uint32_t addr) {
    if (PAIR)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;"
                     :: "r"(addr), "n"(COLS));
    else
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;"
                     :: "r"(addr), "n"(COLS));
}
__device__ __forceinline__ void fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                 :: "r"(bar) : "memory");
}
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
        :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add) : "memory");
}
// The pair's forms: both CTAs hold their half of each operand at the same place
// of their shared memory, one thread of the first CTA issues, and a commit
// arrives at the barrier of this place in both.
__device__ __forceinline__ void mma_pair_commit(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
        "[%0], %1;" :: "r"(bar), "h"((uint16_t)3) : "memory");
}
__device__ __forceinline__ void mma_pair_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                              bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
        :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add) : "memory");
}
// Operand tile of rows of 128 bytes, 128-byte swizzle, K-major: eight rows
// (1024 bytes) between the groups of the stride offset.
__device__ __forceinline__ uint64_t operand(uint32_t addr) {
    return (uint64_t)((addr >> 4) & 0x3FFFu) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// Instruction descriptor: E4M3 x E4M3 to binary32, M x N.
__host__ __device__ constexpr uint32_t mma_shape(int m, int n) {
    return 1u << 4 | (uint32_t)(n >> 3) << 17 | (uint32_t)(m >> 4) << 24;
}
// 16 columns of the warp's 32 lanes.  Load and wait are one statement: passing
// the registers through a separate wait cost a move each, as many instructions
// as the multiply-adds.
__device__ __forceinline__ void tmem_load(uint32_t addr, float v[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
          "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]),
          "=f"(v[14]), "=f"(v[15])
        : "r"(addr) : "memory");
}

// ---- many rows ----------------------------------------------------------------

constexpr int kRowsM = 256, kRowsN = 256, kRowsStages = 6;
constexpr int kRowsHalf = 128;                    // rows of a, and of b, of one CTA of the pair
constexpr int kRowsEpilogueWarps = 8;
constexpr int kRowsRun = 32;                      // columns an epilogue warp stores at a time
constexpr int kRowsAccs = 4, kRowsAccCols = 128;  // accumulators, and columns of one
constexpr int kRowsThreads = 32 * (kRowsEpilogueWarps + 3);
constexpr int kRowsScales = 8;                    // blocks along k whose scales a slot holds
constexpr int kRowsOperand = kRowsHalf * 128;
constexpr int kRowsStage = 2 * kRowsOperand;
// row tiles walked side by side before the next columns: the weights of a
// column tile are read by that many CTAs at about the same time
constexpr int kRowsBand = 8;

struct RowsShared {
    uint4 stage[kRowsEpilogueWarps][128];         // an epilogue warp's way to d
    uint64_t full[kRowsStages], empty[kRowsStages], acc_full[kRowsAccs],
        acc_empty[kRowsAccs], drain;
    uint64_t scale_full[2], scale_empty[2];
    // the row scales of kRowsScales blocks, and those of the tile's two weight blocks
    float sa[2][kRowsScales][kRowsHalf];
    alignas(8) float sb[2][kRowsScales][2];
    uint32_t tmem;
    int abort;
    uint32_t tiles;                               // row tiles of all groups
    uint32_t first[AR_MOE_MAX_EXPERTS];           // row tiles before the group
};
constexpr size_t kRowsSmem = 1024 + (size_t)kRowsStages * kRowsStage + sizeof(RowsShared);

struct RowsTile {
    int group;
    uint32_t row, rows, n0;
};

// Tile `index`: bands of kRowsBand row tiles, in a band column tile by column
// tile, so that CTAs at work at the same time share rows of a and of b in L2.
__device__ __forceinline__ RowsTile rows_tile(const MatmulArgs &a, const RowsShared &sh,
                                              uint32_t ntiles, uint64_t index) {
    const uint64_t per = (uint64_t)kRowsBand * ntiles;
    const uint32_t band = (uint32_t)(index / per);
    const uint32_t in = (uint32_t)(index - band * per);
    const uint32_t rt0 = band * kRowsBand;
    const uint32_t width = sh.tiles - rt0 < kRowsBand ? sh.tiles - rt0 : kRowsBand;
    const uint32_t rt = rt0 + in % width;
    RowsTile t;
    t.n0 = in / width * kRowsN;
    int lo = 0, hi = a.E - 1;                     // last group that starts at or before rt
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (sh.first[mid] <= rt)
            lo = mid;
        else
            hi = mid - 1;
    }
    t.group = lo;
    uint32_t begin, end;
    group_range(a, lo, begin, end);
    t.row = begin + (rt - sh.first[lo]) * kRowsM;
    t.rows = end - t.row < kRowsM ? end - t.row : kRowsM;
    return t;
}

// A warp's 32 rows x 32 columns of sums to d: rows from m0 and columns from n0
// on, as far as `rows` and N.  64 bytes of every row at a time go through the
// warp's 2 KB of shared memory (16-byte words in an order that keeps both sides
// free of bank conflicts), so that a store instruction writes whole sectors of
// eight rows.
template <int OUT>
__device__ __forceinline__ void store_rows(const MatmulArgs &a, uint4 *stage, uint64_t m0,
                                           uint32_t rows, uint32_t n0,
                                           const float acc[kRowsRun]) {
    constexpr int kSize = Elem<OUT>::kSize, kWord = 16 / kSize, kCols = 64 / kSize;
    const uint32_t lane = threadIdx.x & 31;
    auto word = [&](uint32_t row, uint32_t q) -> uint4 & {
        return stage[row * 4 + (q ^ (row >> 1 & 3))];
    };
#pragma unroll
    for (int c = 0; c < kRowsRun; c += kCols) {
        if (n0 + c >= a.N)
            break;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int e = c + q * kWord + i * (kWord / 4);
                w[i] = kSize == 4 ? __float_as_uint(acc[e])
                                  : narrow2<OUT>(acc[e], acc[e + (kSize == 2)]);
            }
            word(lane, q) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        __syncwarp();
        if (a.dwide && n0 + c + kCols <= a.N) {
#pragma unroll
            for (uint32_t i = 0; i < 4; ++i) {
                const uint32_t row = i * 8 + lane / 4, q = lane % 4;
                if (row < rows)
                    reinterpret_cast<uint4 *>(a.d + (m0 + row) * a.ldd +
                                              (uint64_t)(n0 + c) * kSize)[q] = word(row, q);
            }
        } else {
            for (uint32_t i = lane; i < rows * kCols; i += 32) {
                const uint32_t row = i / kCols, col = i % kCols;
                if (n0 + c + col < a.N)
                    st_elem<OUT>(a.d + (m0 + row) * a.ldd, n0 + c + col,
                                 ld_elem<OUT>(&word(row, col / kWord), col % kWord));
            }
        }
        __syncwarp();
    }
}

// Persistent: a pair of CTAs takes a tile of 256 x 256, then the next of every
// gridDim.x / 2.  CTA `rank` holds rows 128 * rank, ... of the tile's rows of a
// and of its rows of b; the tensor cores of both SMs read both halves of b, and
// the sums of a CTA's rows of a are in its own tensor memory.  One CTA's tile of
// 128 x 256 needs 48 KB a block to be written to and read from shared memory,
// more than its 128 bytes a clock allow beside the products; the pair's 32 KB
// fit better.
//
// A block is multiplied in two halves of 128 columns with an accumulator each,
// two blocks' worth in all, so that the products of a half run while the three
// before it are read back.  Warps 0-7: epilogue (lanes 32 * (warp % 4), half
// warp / 4); warp 8: TMA; warp 9: MMA, in the first CTA; warp 10: scales.  The
// scales of a tile's rows are a column of sa, one sector a row: read by every
// epilogue warp for every block they kept the L1 pipe, which also feeds the
// tensor core, half busy.  Warp 10 reads each once, eight blocks at a time, and
// lays them out by block in shared memory.
//
// Bound by the epilogue's chain per warp and block (wait, read back, multiply-
// add, arrive: about 870 clocks) over the products' 640.  8192^3: 415 to 457 us
// by box, 2.4 to 2.6 PFLOP/s; 16384 rows over 64 experts of 2048 x 8192: 340 to 357.
__global__ void __launch_bounds__(kRowsThreads, 1)
k_matmul8_rows(const __grid_constant__ MatmulArgs a, const __grid_constant__ CUtensorMap map_a,
               const __grid_constant__ CUtensorMap map_b) {
    extern __shared__ uint8_t raw[];
    uint8_t *stages = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
    RowsShared &sh = *reinterpret_cast<RowsShared *>(stages + kRowsStages * kRowsStage);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = blockIdx.x & 1, pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    volatile int *abort = &sh.abort;
    const uint32_t full = smem_addr(sh.full), empty = smem_addr(sh.empty);
    const uint32_t acc_full = smem_addr(sh.acc_full), acc_empty = smem_addr(sh.acc_empty);
    const uint32_t scale_full = smem_addr(sh.scale_full), scale_empty = smem_addr(sh.scale_empty);

    if (threadIdx.x == 0) {
        for (int s = 0; s < kRowsStages; ++s) {
            mbar_init(full + 8 * s, 1);
            mbar_init(empty + 8 * s, 1);
        }
        for (int b = 0; b < kRowsAccs; ++b) {
            mbar_init(acc_full + 8 * b, 1);
            mbar_init(acc_empty + 8 * b, kRowsEpilogueWarps);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(scale_full + 8 * b, 1);
            mbar_init(scale_empty + 8 * b, kRowsEpilogueWarps);
        }
        mbar_init(smem_addr(&sh.drain), 1);
        sh.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kRowsEpilogueWarps + 1)
        tmem_alloc<512, true>(&sh.tmem);
    kernel_prologue();
    if (warp == 0) {
        uint32_t base = 0;
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            uint32_t lo = 0, hi = 0;
            if (e0 + lane < a.E)
                group_range(a, e0 + lane, lo, hi);
            const uint32_t n = (hi - lo + kRowsM - 1) / kRowsM;
            uint32_t scan = n;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, scan, d);
                scan += lane >= d ? v : 0u;
            }
            if (e0 + lane < a.E)
                sh.first[e0 + lane] = base + scan - n;
            base = __shfl_sync(0xFFFFFFFFu, base + scan, 31);
        }
        if (lane == 0)
            sh.tiles = base;
    }
    fence_before();
    cluster_sync();                               // both CTAs' barriers are ready
    fence_after();
    const uint32_t tmem = sh.tmem;
    const uint32_t ntiles = (a.N + kRowsN - 1) / kRowsN;
    const uint64_t total = (uint64_t)sh.tiles * ntiles;

    uint32_t used = 0;                            // stages filled or drained by this role
    if (warp == kRowsEpilogueWarps) {
        if (lane == 0) {
            for (uint64_t i = pair; i < total && !*abort; i += pairs) {
                const RowsTile t = rows_tile(a, sh, ntiles, i);
                for (int kb = 0; kb < a.kb; ++kb, ++used) {
                    const uint32_t s = used % kRowsStages, turn = used / kRowsStages;
                    if (turn > 0 && !mbar_wait(empty + 8 * s, (turn - 1) & 1, abort, a.status))
                        break;
                    const uint32_t at = smem_addr(stages) + s * kRowsStage;
                    const uint32_t bar = map_to_rank(full + 8 * s, 0);
                    // a tile of at most 128 rows leaves the second CTA's rows
                    // of a alone: their sums are not stored
                    const bool both = t.rows > kRowsHalf;
                    if (rank == 0)
                        mbar_expect(full + 8 * s, (both ? 4 : 3) * kRowsOperand);
                    if (rank == 0 || both)
                        tma_pair_2d(at, &map_a, kb * 128, (int)(t.row + rank * kRowsHalf), bar);
                    tma_pair_3d(at + kRowsOperand, &map_b, kb * 128,
                                (int)(t.n0 + rank * kRowsHalf), t.group, bar);
                }
            }
            // the last stages' arrivals come from the first CTA: this one stays
            // until they are in
            for (uint32_t k = used < kRowsStages ? 0 : used - kRowsStages; k < used && !*abort; ++k)
                (void)mbar_wait(empty + 8 * (k % kRowsStages), (k / kRowsStages) & 1, abort,
                                a.status);
        }
        __syncwarp();
    } else if (warp == kRowsEpilogueWarps + 1 && rank == 0) {
        // The whole warp walks the blocks and one lane issues: in a branch of
        // one lane the descriptors would not stay in uniform registers, and
        // the issue alone took longer than the products.
        const uint64_t desc_a = operand(smem_addr(stages));
        const uint64_t desc_b = operand(smem_addr(stages) + kRowsOperand);
        const bool one = elect_one();
        bool ok = true;
        for (uint64_t i = pair; i < total && ok; i += pairs) {
            for (int kb = 0; kb < a.kb; ++kb, ++used) {
                const uint32_t s = used % kRowsStages;
                if (!warp_wait(full + 8 * s, (used / kRowsStages) & 1, abort, a.status)) {
                    ok = false;
                    break;
                }
                // the block's two halves: rows 64 * half, ... of either CTA's b
#pragma unroll
                for (uint32_t half = 0; half < 2; ++half) {
                    const uint32_t b = (2 * used + half) % kRowsAccs, turn = used / 2;
                    ok = turn == 0 || warp_wait(acc_empty + 8 * b, (turn - 1) & 1, abort, a.status);
                    if (!ok)
                        break;
                    fence_after();
                    const uint64_t da = desc_a + s * (kRowsStage >> 4);
                    const uint64_t db = desc_b + s * (kRowsStage >> 4) + half * (64 * 128 >> 4);
                    if (one) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_pair_e4m3(tmem + b * kRowsAccCols, da + 2 * k, db + 2 * k,
                                          mma_shape(kRowsM, kRowsAccCols), k > 0);
                        if (half == 1)
                            mma_pair_commit(empty + 8 * s);
                        mma_pair_commit(acc_full + 8 * b);
                    }
                    __syncwarp();
                }
                if (!ok)
                    break;
            }
        }
    } else if (warp == kRowsEpilogueWarps + 1) {
        __syncwarp();                             // the first CTA issues for both
    } else if (warp == kRowsEpilogueWarps + 2) {
        uint32_t slots = 0;
        bool ok = true;
        for (uint64_t i = pair; i < total && ok; i += pairs) {
            const RowsTile t = rows_tile(a, sh, ntiles, i);
            for (int kb0 = 0; kb0 < a.kb; kb0 += kRowsScales, ++slots) {
                // rows and columns past the tile's end take a valid scale and
                // are not stored
                float v[kRowsHalf / 32][kRowsScales], w = 0.0f;
#pragma unroll
                for (int j = 0; j < kRowsHalf / 32; ++j) {
                    const uint32_t r = rank * kRowsHalf + j * 32 + lane;
                    const float *sa = a.sa + (uint64_t)(r < t.rows ? t.row + r : t.row) * a.sa_row +
                                      kb0;
                    if (a.sa_wide) {
#pragma unroll
                        for (int k = 0; k < kRowsScales; k += 4) {
                            float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                            if (kb0 + k < a.kb)
                                f = *reinterpret_cast<const float4 *>(sa + k);
                            v[j][k] = f.x;
                            v[j][k + 1] = f.y;
                            v[j][k + 2] = f.z;
                            v[j][k + 3] = f.w;
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < kRowsScales; ++k)
                            v[j][k] = kb0 + k < a.kb ? sa[k] : 0.0f;
                    }
                }
                const int k = lane & (kRowsScales - 1), side = lane / kRowsScales;
                const uint32_t nb = t.n0 / 128 + side;
                if (side < 2 && kb0 + k < a.kb)
                    w = a.sb[t.group * a.sb_group + (uint64_t)(nb * 128 < a.N ? nb : 0) * a.kb +
                             kb0 + k];
                const uint32_t slot = slots & 1, round = slots >> 1;
                ok = round == 0 || warp_wait(scale_empty + 8 * slot, (round - 1) & 1, abort,
                                             a.status);
                if (!ok)
                    break;
#pragma unroll
                for (int j = 0; j < kRowsHalf / 32; ++j)
#pragma unroll
                    for (int b = 0; b < kRowsScales; ++b)
                        sh.sa[slot][b][j * 32 + lane] = v[j][b];
                if (side < 2)
                    sh.sb[slot][k][side] = w;
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(scale_full + 8 * slot);
            }
        }
        __syncwarp();
    } else {
        // A warp takes one half of every block.  Columns 0-63 of a half are rows
        // 64 * half, ... of the first CTA's b, columns 64-127 of the second's.
        const int quarter = warp & 3, half = warp >> 2;
        const uint32_t empty_bar = map_to_rank(acc_empty, 0);
        const uint32_t lanes = tmem + ((uint32_t)quarter * 32 << 16);
        const uint32_t in = quarter * 32 + lane;
        uint32_t blocks = 0, slots = 0;
        bool ok = true;
        for (uint64_t i = pair; i < total && ok; i += pairs) {
            const RowsTile t = rows_tile(a, sh, ntiles, i);
            float acc[4][kRowsRun];
#pragma unroll
            for (int c = 0; c < kRowsRun; ++c)
                acc[0][c] = acc[1][c] = acc[2][c] = acc[3][c] = 0.0f;
            for (int kb = 0; kb < a.kb; ++kb, ++blocks) {
                const uint32_t slot = slots & 1, k = kb & (kRowsScales - 1);
                const uint32_t b = (2 * blocks + half) % kRowsAccs;
                if (k == 0)
                    ok = warp_wait(scale_full + 8 * slot, (slots >> 1) & 1, abort, a.status);
                const float sa = sh.sa[slot][k][in];
                const float2 sb = *reinterpret_cast<const float2 *>(sh.sb[slot][k]);
                ok = ok && warp_wait(acc_full + 8 * b, (blocks / 2) & 1, abort, a.status);
                if (!ok)
                    break;
                fence_after();
                const float scale[2] = {sa * sb.x, sa * sb.y};
#pragma unroll
                for (int c = 0; c < kRowsAccCols; c += 16) {
                    float v[16];
                    tmem_load(lanes + b * kRowsAccCols + c, v);
                    if (c + 16 == kRowsAccCols) {
                        fence_before();
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive_peer(empty_bar + 8 * b);
                    }
#pragma unroll
                    for (int j = 0; j < 16; j += 2)
                        fma2(&acc[c / kRowsRun][c % kRowsRun + j], scale[c / 64], scale[c / 64],
                             v[j], v[j + 1]);
                }
                if (k == kRowsScales - 1 || kb + 1 == a.kb) {
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(scale_empty + 8 * slot);
                    ++slots;
                }
            }
            const uint32_t first = rank * kRowsHalf + quarter * 32;
            if (ok && first < t.rows) {
                const uint32_t rows = t.rows - first < 32 ? t.rows - first : 32;
                uint4 *stage = sh.stage[warp];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint32_t n = t.n0 + (c / 2) * 128 + half * 64 + (c % 2) * kRowsRun;
                    if (a.out == AR_BF16)
                        store_rows<AR_BF16>(a, stage, t.row + first, rows, n, acc[c]);
                    else if (a.out == AR_FP16)
                        store_rows<AR_FP16>(a, stage, t.row + first, rows, n, acc[c]);
                    else
                        store_rows<AR_FP32>(a, stage, t.row + first, rows, n, acc[c]);
                }
            }
            __syncwarp();
        }
        __syncwarp();
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (*abort) {
        if (threadIdx.x == kRowsEpilogueWarps * 32) {
            if (rank == 0)
                drain_loads(full, used, kRowsStages);
            else
                linger();
        }
        if (warp == kRowsEpilogueWarps + 1 && rank == 0 && elect_one()) {
            mma_pair_commit(smem_addr(&sh.drain));
            mbar_drain(smem_addr(&sh.drain), 0);
        }
        __syncthreads();
    }
    cluster_sync();                               // nothing of the pair is in flight
    if (warp == kRowsEpilogueWarps + 1)
        tmem_free<512, true>(tmem);
}

// ---- few rows -------------------------------------------------------------------

constexpr int kFewEpilogueWarps = 4;
constexpr int kFewThreads = 32 * (kFewEpilogueWarps + 3);
constexpr int kMaxParts = 8;                      // CTAs of a cluster
constexpr int kFewScales = 8;                     // blocks along k whose scales a slot holds
constexpr int kFewWeights = 128 * 128;            // bytes of a stage's weights

// NT: rows of a per tile.  Two CTAs per SM share its shared and tensor memory.
template <int NT> struct Few {
    static constexpr int kStage = kFewWeights + NT * 128;
    static constexpr int kStages = NT <= 32 ? 5 : 4;
    static constexpr int kAccs = 4;
    static constexpr int kCols = NT * kAccs;
    static_assert(kCols <= 256, "two CTAs' accumulators share 512 columns");
    static_assert(kStages * kStage >= NT * 512, "the joined sums reuse the stages");
};
template <int NT> struct FewShared {
    uint64_t full[Few<NT>::kStages], empty[Few<NT>::kStages];
    uint64_t acc_full[Few<NT>::kAccs], acc_empty[Few<NT>::kAccs], drain;
    uint64_t scale_full[2], scale_empty[2];
    alignas(16) float scale[2][kFewScales][NT];   // sa * sb by block and row
    uint32_t tmem;
    int abort;
};
template <int NT> constexpr size_t few_smem() {
    return 1024 + (size_t)Few<NT>::kStages * Few<NT>::kStage + sizeof(FewShared<NT>);
}

// blockIdx.x: CTA of the cluster (its share of the blocks along k);
// blockIdx.y: tile of 128 weight rows; blockIdx.z: row tile, counted over the
// groups.  Warps 0-3: epilogue, lane + 32 * warp is the weight row; warp 4:
// TMA; warp 5: MMA; warp 6: scales, sa * sb for eight blocks at a time.  Bound by
// the stream of the weights: 4096 rows over 64 experts of 2048 x 8192 187 to 200 us
// (5.6 to 6.0 TB/s); one row of 8192 x 8192 14.0 us, of which about 5 are launch, first loads
// and join.
template <int NT>
__global__ void __launch_bounds__(kFewThreads, 2)
k_matmul8_few(const __grid_constant__ MatmulArgs a, const __grid_constant__ CUtensorMap map_a,
              const __grid_constant__ CUtensorMap map_b) {
    using F = Few<NT>;
    extern __shared__ uint8_t raw[];
    uint8_t *stages = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
    FewShared<NT> &sh = *reinterpret_cast<FewShared<NT> *>(stages + F::kStages * F::kStage);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int *abort = &sh.abort;
    const uint32_t full = smem_addr(sh.full), empty = smem_addr(sh.empty);
    const uint32_t acc_full = smem_addr(sh.acc_full), acc_empty = smem_addr(sh.acc_empty);
    const uint32_t scale_full = smem_addr(sh.scale_full), scale_empty = smem_addr(sh.scale_empty);

    // what needs no memory of earlier kernels comes before the wait for them
    if (threadIdx.x == 0) {
        for (int s = 0; s < F::kStages; ++s) {
            mbar_init(full + 8 * s, 1);
            mbar_init(empty + 8 * s, 1);
        }
        for (int b = 0; b < F::kAccs; ++b) {
            mbar_init(acc_full + 8 * b, 1);
            mbar_init(acc_empty + 8 * b, kFewEpilogueWarps);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(scale_full + 8 * b, 1);
            mbar_init(scale_empty + 8 * b, kFewEpilogueWarps);
        }
        mbar_init(smem_addr(&sh.drain), 1);
        sh.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 5)
        tmem_alloc<F::kCols, false>(&sh.tmem);
    kernel_prologue();
    int group = 0;
    uint32_t row = 0, rows = 0;
    // the same answer in the whole cluster
    const bool tile = find_rows(a, NT, blockIdx.z, group, row, rows);
    fence_before();
    __syncthreads();
    fence_after();
    if (!tile) {
        if (warp == 5)
            tmem_free<F::kCols, false>(sh.tmem);
        return;
    }
    const uint32_t tmem = sh.tmem;
    const int parts = gridDim.x, part = blockIdx.x;
    const int kb0 = (int)((int64_t)a.kb * part / parts);
    const int kb1 = (int)((int64_t)a.kb * (part + 1) / parts);
    const uint32_t n0 = blockIdx.y * 128;
    const uint32_t n = n0 + threadIdx.x;          // epilogue: this thread's weight row
    float acc[NT];
    uint32_t used = 0;                            // stages filled or drained by this role

    if (warp == 4) {
        if (lane == 0) {
            for (int kb = kb0; kb < kb1; ++kb, ++used) {
                const uint32_t s = used % F::kStages, turn = used / F::kStages;
                if (turn > 0 && !mbar_wait(empty + 8 * s, (turn - 1) & 1, abort, a.status))
                    break;
                const uint32_t at = smem_addr(stages) + s * F::kStage;
                mbar_expect(full + 8 * s, F::kStage);
                tma_3d(at, &map_b, kb * 128, (int)n0, group, full + 8 * s);
                tma_2d(at + kFewWeights, &map_a, kb * 128, (int)row, full + 8 * s);
            }
        }
        __syncwarp();
    } else if (warp == 5) {
        const uint64_t desc_b = operand(smem_addr(stages));
        const uint64_t desc_a = operand(smem_addr(stages) + kFewWeights);
        const bool one = elect_one();
        for (int kb = kb0; kb < kb1; ++kb, ++used) {
            const uint32_t s = used % F::kStages, b = used % F::kAccs, round = used / F::kAccs;
            if (round > 0 && !warp_wait(acc_empty + 8 * b, (round - 1) & 1, abort, a.status))
                break;
            if (!warp_wait(full + 8 * s, (used / F::kStages) & 1, abort, a.status))
                break;
            fence_after();
            if (one) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mma_e4m3(tmem + b * NT, desc_b + s * (F::kStage >> 4) + 2 * k,
                             desc_a + s * (F::kStage >> 4) + 2 * k, mma_shape(128, NT), k > 0);
                mma_commit(empty + 8 * s);
                mma_commit(acc_full + 8 * b);
            }
            __syncwarp();
        }
    } else if (warp == 6) {
        constexpr int kPer = (NT + 31) / 32;
        const float *sb = a.sb + group * a.sb_group + (uint64_t)(n0 / 128) * a.kb;
        uint32_t slots = 0;
        for (int kb = kb0; kb < kb1; kb += kFewScales, ++slots) {
            // rows past the tile's end take a valid scale and are not stored
            float v[kPer][kFewScales];
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const uint32_t r = lane + 32 * j;
                const float *sa = a.sa + (uint64_t)(r < rows ? row + r : row) * a.sa_row + kb;
                if (a.sa_wide && kb % 4 == 0) {
                    // rows of scales are whole 16-byte words up to the last
#pragma unroll
                    for (int k = 0; k < kFewScales; k += 4) {
                        float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        if (kb + k < kb1)
                            f = *reinterpret_cast<const float4 *>(sa + k);
                        v[j][k] = f.x;
                        v[j][k + 1] = f.y;
                        v[j][k + 2] = f.z;
                        v[j][k + 3] = f.w;
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < kFewScales; ++k)
                        v[j][k] = kb + k < kb1 ? sa[k] : 0.0f;
                }
#pragma unroll
                for (int k = 0; k < kFewScales; ++k)
                    v[j][k] *= kb + k < kb1 ? sb[kb + k] : 0.0f;
            }
            const uint32_t slot = slots & 1, round = slots >> 1;
            if (round > 0 && !warp_wait(scale_empty + 8 * slot, (round - 1) & 1, abort, a.status))
                break;
#pragma unroll
            for (int j = 0; j < kPer; ++j)
#pragma unroll
                for (int k = 0; k < kFewScales; ++k)
                    if (lane + 32 * j < NT)
                        sh.scale[slot][k][lane + 32 * j] = v[j][k];
            __syncwarp();
            if (lane == 0)
                mbar_arrive(scale_full + 8 * slot);
        }
        __syncwarp();
    } else {
        const uint32_t lanes = tmem + ((uint32_t)warp * 32 << 16);
#pragma unroll
        for (int c = 0; c < NT; ++c)
            acc[c] = 0.0f;
        uint32_t slots = 0;
        for (int kb = kb0; kb < kb1; ++kb, ++used) {
            const uint32_t b = used % F::kAccs, slot = slots & 1, k = used % kFewScales;
            if (k == 0 && !warp_wait(scale_full + 8 * slot, (slots >> 1) & 1, abort, a.status))
                break;
            if (!warp_wait(acc_full + 8 * b, (used / F::kAccs) & 1, abort, a.status))
                break;
            fence_after();
            const float *scale = sh.scale[slot][k];
#pragma unroll
            for (int c = 0; c < NT; c += 16) {
                float v[16];
                tmem_load(lanes + b * NT + c, v);
                if (c + 16 == NT) {
                    fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(acc_empty + 8 * b);
                }
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(scale + c + j);
                    fma2(&acc[c + j], f.x, f.y, v[j], v[j + 1]);
                    fma2(&acc[c + j + 2], f.z, f.w, v[j + 2], v[j + 3]);
                }
            }
            if (k == kFewScales - 1 || kb + 1 == kb1) {
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(scale_empty + 8 * slot);
                ++slots;
            }
        }
        __syncwarp();
    }
    // every load has landed and every product is done: the stages are free
    fence_before();
    __syncthreads();
    fence_after();
    if (*abort) {
        if (threadIdx.x == 4 * 32)
            drain_loads(full, used, F::kStages);
        if (warp == 5 && elect_one()) {
            mma_commit(smem_addr(&sh.drain));
            mbar_drain(smem_addr(&sh.drain), 0);
        }
        __syncthreads();
    }
    if (warp == 5)
        tmem_free<F::kCols, false>(tmem);
    if (parts == 1) {
        if (warp < kFewEpilogueWarps && n < a.N)
#pragma unroll
            for (int c = 0; c < NT; ++c)
                if (c < (int)rows)
                    store_out(a.d + (uint64_t)(row + c) * a.ldd, n, acc[c], a.out);
        return;
    }
    // join the parts: CTA p of the cluster sums its share of the rows over all
    // CTAs, in their order along k
    float *sums = reinterpret_cast<float *>(stages);      // [NT][128]
    if (warp < kFewEpilogueWarps)
#pragma unroll
        for (int c = 0; c < NT; ++c)
            sums[c * 128 + threadIdx.x] = acc[c];
    cluster_sync();
    // (the loads of kAt rows from every CTA are in flight together: one after
    // the other they cost 0.5 us each, 14 us for 1000 x 1000 x 1000)
    constexpr int kAt = 4;
    if (warp < kFewEpilogueWarps)
        for (uint32_t c0 = part; c0 < rows; c0 += parts * kAt) {
            float v[kMaxParts][kAt];
#pragma unroll
            for (int p = 0; p < kMaxParts; ++p)
#pragma unroll
                for (int j = 0; j < kAt; ++j) {
                    const uint32_t c = c0 + j * parts;
                    v[p][j] = p < parts && c < rows
                                  ? ld_peer_f32(sums + c * 128 + threadIdx.x, p)
                                  : 0.0f;
                }
#pragma unroll
            for (int j = 0; j < kAt; ++j) {
                const uint32_t c = c0 + j * parts;
                float sum = v[0][j];
#pragma unroll
                for (int p = 1; p < kMaxParts; ++p)
                    sum += v[p][j];
                if (c < rows && n < a.N)
                    store_out(a.d + (uint64_t)(row + c) * a.ldd, n, sum, a.out);
            }
        }
    cluster_sync();
}

// ---- host ---------------------------------------------------------------------

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static std::atomic<void *> found{nullptr};
    void *p = found.load(std::memory_order_acquire);
    if (!p) {
        cudaDriverEntryPointQueryResult how;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &how) != cudaSuccess ||
            how != cudaDriverEntryPointSuccess) {
            (void)cudaGetLastError();
            return nullptr;
        }
        found.store(p, std::memory_order_release);
    }
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
}

// Tiles of 128 bytes x `rows`; bytes past k and rows past the end read as zero.
bool encode(CUtensorMap *map, const void *base, uint64_t k, uint64_t rows, uint64_t stride,
            uint64_t groups, uint32_t box_rows) {
    const cuuint64_t dims[3] = {k, rows, groups};
    const cuuint64_t strides[2] = {stride, stride * rows};
    const cuuint32_t box[3] = {128, box_rows, 1}, ones[3] = {1, 1, 1};
    return encoder()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, groups ? 3 : 2,
                     const_cast<void *>(base), dims, strides, box, ones,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NT>
cudaError_t launch_few(const MatmulArgs &a, int parts, cudaStream_t s) {
    CUtensorMap ma, mb;
    if (!encode(&ma, a.a, a.K, a.M, a.lda, 0, NT) ||
        !encode(&mb, a.b, a.K, a.N, a.ldb, a.E, 128))
        return cudaErrorInvalidValue;
    const cudaError_t e = opt_in_smem<k_matmul8_few<NT>>(few_smem<NT>());
    if (e != cudaSuccess)
        return e;
    // row tiles: every group adds at most one that is not full
    const uint32_t groups = (uint32_t)a.E < a.M ? (uint32_t)a.E : a.M;
    const uint32_t tiles = a.offsets ? a.M / NT + groups : (a.M + NT - 1) / NT;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(parts, (a.N + 127) / 128, tiles);
    cfg.blockDim = kFewThreads;
    cfg.dynamicSmemBytes = few_smem<NT>();
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = parts;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k_matmul8_few<NT>, a, ma, mb);
}

cudaError_t launch_rows(const MatmulArgs &a, int sms, cudaStream_t s) {
    CUtensorMap ma, mb;
    if (!encode(&ma, a.a, a.K, a.M, a.lda, 0, kRowsHalf) ||
        !encode(&mb, a.b, a.K, a.N, a.ldb, a.E, kRowsHalf))
        return cudaErrorInvalidValue;
    const cudaError_t e = opt_in_smem<k_matmul8_rows>(kRowsSmem);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = sms / 2 * 2;
    cfg.blockDim = kRowsThreads;
    cfg.dynamicSmemBytes = kRowsSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k_matmul8_rows, a, ma, mb);
}

}  // namespace

bool matmul8_tc_ready() { return encoder() != nullptr; }

cudaError_t launch_matmul8_tc(const MatmulArgs &a, cudaStream_t s) {
    const int sms = sm_count();
    if (sms < 1)
        return cudaErrorUnknown;
    const uint64_t groups = (uint64_t)a.E < a.M ? a.E : a.M;
    // tiles of n rows: every group adds at most one that is not full
    auto tiles = [&](uint64_t n) { return a.offsets ? a.M / n + groups : (a.M + n - 1) / n; };
    auto waves = [](uint64_t n, uint64_t at_once) { return (n + at_once - 1) / at_once; };

    const uint64_t columns = (a.N + 127) / 128;
    // Estimates in hundredths of a us from measured launches.  The few form, two
    // CTAs an SM: a wave of CTAs costs `wave` and `block` for each of its blocks
    // along k; cutting k over the CTAs of a cluster shortens that and adds `join`,
    // as long as the clusters fill at most 7/8 of a wave (a full one of fours ran in
    // two: 300 x 500 x 700 8.3 us).  The rows form: 2.9 us and 0.45 a block for
    // every wave of pairs.
    // Either side as measured (us), few and rows: K = N = 8192 at M = 64, 128,
    // 256, 512: 16.8, 22.9, 34.9, 66.8 and 31.9, 32.8, 33.1, 35.1; 64 experts of
    // 2048 x 8192 at M = 1024, 4096, 8192, 16384: 159, 187, 282, 478 and 218, 228,
    // 265, 364; 2000 x 3000 x 128: 13.3 and 11.2; 300 x 500 x 700: 4.1 and 13.7.
    // Parts, one row of 8192 x 8192: 20.5, 15.7, 14.1 and 17.2 in 1, 2, 4 and 8.
    struct { int nt, wave, block, join; } const kForms[] = {
        {16, 200, 40, 150}, {32, 280, 42, 200}, {64, 380, 45, 250}};
    uint64_t best = waves(tiles(kRowsM) * ((a.N + kRowsN - 1) / kRowsN), sms / 2) *
                    (290 + 45 * (uint64_t)a.kb);
    int nt = 0, parts = 1;
    for (const auto &f : kForms) {
        // the grid's y and z dimensions end at 65535
        if (columns > 65535 || tiles(f.nt) > 65535)
            continue;
        const uint64_t ctas = tiles(f.nt) * columns, room = 2 * (uint64_t)sms;
        for (int p = 1; p == 1 || (p <= kMaxParts && p <= a.kb && ctas * p * 8 <= room * 7);
             p *= 2) {
            const uint64_t cost = waves(ctas * p, room) * (f.wave + waves(a.kb, p) * f.block) +
                                  (p > 1 ? f.join : 0);
            if (cost < best) {
                best = cost;
                nt = f.nt;
                parts = p;
            }
        }
    }
    switch (nt) {
    case 0: return launch_rows(a, sms, s);
    case 16: return launch_few<16>(a, parts, s);
    case 32: return launch_few<32>(a, parts, s);
    default: return launch_few<64>(a, parts, s);
    }
}

}  // namespace ar
