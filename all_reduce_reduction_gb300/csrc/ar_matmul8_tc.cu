// The E4M3 product on the tensor cores (tcgen05), operands by TMA.
//
// A scale belongs to 128 elements along k, so the tensor core can sum one such
// block only: 128 x N x 128 products go to an accumulator in tensor memory,
// and the epilogue warps read it back, multiply it with sa * sb and add it to
// binary32 sums in their registers, while the tensor core fills the next
// accumulator.
//
// Two forms.  k_matmul8_rows puts 128 rows of a on the accumulator's lanes and
// 256 rows of b on its columns: a thread's row scale is then one register.
// k_matmul8_few is for few rows per group: 128 rows of b on the lanes, 16 to
// 128 rows of a on the columns, several CTAs of a cluster along k; it streams
// the weights once with all SMs even when there is one row.
//
// Every wait is bounded: past kWaitNs it writes AR_ERR_TIMEOUT to the caller's
// status word and the CTA's roles all leave.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>

#include "ar_matmul8.cuh"

namespace ar {
namespace {

constexpr uint64_t kWaitNs = 2000000000ull;

__device__ __forceinline__ uint32_t smem_addr(const void *p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}
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
// another role of the CTA gave up.
__device__ __noinline__ bool mbar_wait_slow(uint32_t bar, uint32_t parity, volatile int *abort,
                                            int *status) {
    const uint64_t deadline = globaltimer_ns() + kWaitNs;
    for (;;) {
        if (mbar_test(bar, parity))
            return true;
        if (*abort)
            return false;
        if (globaltimer_ns() > deadline) {
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

// ---- tcgen05 -------------------------------------------------------------------

template <int COLS> __device__ __forceinline__ void tmem_alloc(uint32_t *slot) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 :: "r"(smem_addr(slot)), "n"(COLS) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
template <int COLS> __device__ __forceinline__ void tmem_free(uint32_t addr) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(addr), "n"(COLS));
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
// One block along k: 128 bytes, 32 per instruction.
__device__ __forceinline__ void mma_block(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc) {
    const uint64_t da = operand(a), db = operand(b);
#pragma unroll
    for (int k = 0; k < 4; ++k)
        mma_e4m3(d, da + 2 * k, db + 2 * k, idesc, k > 0);
}

// 16 columns of the warp's 32 lanes; the values are there after tmem_wait.
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t v[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
          "=r"(v[14]), "=r"(v[15])
        : "r"(addr));
}
// The registers pass through the wait, so that nothing reads them before it.
__device__ __forceinline__ void tmem_wait(uint32_t v[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]),
                   "+r"(v[6]), "+r"(v[7]), "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]),
                   "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
                 :: "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&p);
}
__device__ __forceinline__ uint32_t pack_fp16(float a, float b) {
    const __half2 p = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&p);
}

// ---- many rows ----------------------------------------------------------------

constexpr int kRowsM = 128, kRowsN = 256, kRowsStages = 4;
constexpr int kRowsEpilogueWarps = 8;
constexpr int kRowsThreads = 32 * (kRowsEpilogueWarps + 2);
constexpr int kRowsABytes = kRowsM * 128, kRowsBBytes = kRowsN * 128;
constexpr int kRowsStage = kRowsABytes + kRowsBBytes;
// row tiles walked side by side before the next columns: the weights of a
// column tile are read by that many CTAs at about the same time
constexpr int kRowsBand = 16;

struct RowsShared {
    uint64_t full[kRowsStages], empty[kRowsStages], acc_full[2], acc_empty[2], drain;
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

__device__ __forceinline__ void group_range(const MatmulArgs &a, int e, uint32_t &lo,
                                            uint32_t &hi) {
    if (!a.offsets) {
        lo = 0;
        hi = a.M;
        return;
    }
    const int32_t x = a.offsets[e], y = a.offsets[e + 1];
    lo = x < 0 ? 0u : (uint32_t)x < a.M ? (uint32_t)x : a.M;
    hi = y < 0 ? 0u : (uint32_t)y < a.M ? (uint32_t)y : a.M;
    hi = hi < lo ? lo : hi;
}

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

// 128 sums of one row to d, columns n to n + 127 as far as N.
__device__ __forceinline__ void store_row(const MatmulArgs &a, uint64_t m, uint32_t n,
                                          const float acc[128]) {
    uint8_t *row = a.d + m * a.ldd;
    if (a.out == AR_FP32) {
        float4 *to = reinterpret_cast<float4 *>(row + (uint64_t)n * 4);
#pragma unroll
        for (int c = 0; c < 128; c += 4) {
            if (a.dwide && n + c + 4 <= a.N)
                to[c / 4] = make_float4(acc[c], acc[c + 1], acc[c + 2], acc[c + 3]);
            else
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (n + c + j < a.N)
                        store_out(row, n + c + j, acc[c + j], AR_FP32);
        }
    } else {
        uint4 *to = reinterpret_cast<uint4 *>(row + (uint64_t)n * 2);
        const bool bf16 = a.out == AR_BF16;
#pragma unroll
        for (int c = 0; c < 128; c += 8) {
            if (a.dwide && n + c + 8 <= a.N) {
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    w[j] = bf16 ? pack_bf16(acc[c + 2 * j], acc[c + 2 * j + 1])
                                : pack_fp16(acc[c + 2 * j], acc[c + 2 * j + 1]);
                to[c / 8] = make_uint4(w[0], w[1], w[2], w[3]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (n + c + j < a.N)
                        store_out(row, n + c + j, acc[c + j], a.out);
            }
        }
    }
}

// Persistent: one CTA per SM takes tiles blockIdx.x, + gridDim.x, ...
// Warps 0-7: epilogue (lanes 32 * (warp % 4), columns 128 * (warp / 4));
// warp 8: TMA; warp 9: MMA.
__global__ void __launch_bounds__(kRowsThreads, 1)
k_matmul8_rows(const __grid_constant__ MatmulArgs a, const __grid_constant__ CUtensorMap map_a,
               const __grid_constant__ CUtensorMap map_b) {
    extern __shared__ uint8_t raw[];
    uint8_t *stages = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
    RowsShared &sh = *reinterpret_cast<RowsShared *>(stages + kRowsStages * kRowsStage);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int *abort = &sh.abort;
    const uint32_t full = smem_addr(sh.full), empty = smem_addr(sh.empty);
    const uint32_t acc_full = smem_addr(sh.acc_full), acc_empty = smem_addr(sh.acc_empty);

    if (threadIdx.x == 0) {
        for (int s = 0; s < kRowsStages; ++s) {
            mbar_init(full + 8 * s, 1);
            mbar_init(empty + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(acc_full + 8 * b, 1);
            mbar_init(acc_empty + 8 * b, kRowsEpilogueWarps);
        }
        mbar_init(smem_addr(&sh.drain), 1);
        sh.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 9)
        tmem_alloc<512>(&sh.tmem);
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
    __syncthreads();
    fence_after();
    const uint32_t tmem = sh.tmem;
    const uint32_t ntiles = (a.N + kRowsN - 1) / kRowsN;
    const uint64_t total = (uint64_t)sh.tiles * ntiles;

    uint32_t used = 0;                            // stages filled or drained by this role
    if (warp == 8) {
        if (lane == 0) {
            for (uint64_t i = blockIdx.x; i < total && !*abort; i += gridDim.x) {
                const RowsTile t = rows_tile(a, sh, ntiles, i);
                for (int kb = 0; kb < a.kb; ++kb, ++used) {
                    const uint32_t s = used % kRowsStages, turn = used / kRowsStages;
                    if (turn > 0 && !mbar_wait(empty + 8 * s, (turn - 1) & 1, abort, a.status))
                        break;
                    const uint32_t at = smem_addr(stages) + s * kRowsStage;
                    mbar_expect(full + 8 * s, kRowsStage);
                    tma_2d(at, &map_a, kb * 128, (int)t.row, full + 8 * s);
                    tma_3d(at + kRowsABytes, &map_b, kb * 128, (int)t.n0, t.group, full + 8 * s);
                }
            }
        }
        __syncwarp();
    } else if (warp == 9) {
        if (lane == 0) {
            uint32_t blocks = 0;                  // accumulators filled
            for (uint64_t i = blockIdx.x; i < total && !*abort; i += gridDim.x) {
                for (int kb = 0; kb < a.kb; ++kb, ++used, ++blocks) {
                    const uint32_t s = used % kRowsStages, turn = used / kRowsStages;
                    const uint32_t b = blocks & 1, round = blocks >> 1;
                    if (round > 0 &&
                        !mbar_wait(acc_empty + 8 * b, (round - 1) & 1, abort, a.status))
                        break;
                    if (!mbar_wait(full + 8 * s, turn & 1, abort, a.status))
                        break;
                    fence_after();
                    const uint32_t at = smem_addr(stages) + s * kRowsStage;
                    mma_block(tmem + b * kRowsN, at, at + kRowsABytes,
                              mma_shape(kRowsM, kRowsN));
                    mma_commit(empty + 8 * s);
                    mma_commit(acc_full + 8 * b);
                }
            }
        }
        __syncwarp();
    } else {
        const int quarter = warp & 3, side = warp >> 2;
        const uint32_t lanes = tmem + ((uint32_t)quarter * 32 << 16) + side * 128;
        uint32_t blocks = 0;
        bool ok = true;
        for (uint64_t i = blockIdx.x; i < total && ok; i += gridDim.x) {
            const RowsTile t = rows_tile(a, sh, ntiles, i);
            const uint32_t r = quarter * 32 + lane;
            const bool here = r < t.rows;
            const uint32_t n = t.n0 + side * 128;
            // rows and columns past the tile's end read a valid scale and are
            // not stored
            const float *sa = a.sa + (uint64_t)(here ? t.row + r : t.row) * a.sa_row;
            const float *sb = a.sb + t.group * a.sb_group + (uint64_t)(n < a.N ? n / 128 : 0) * a.kb;
            float acc[128];
#pragma unroll
            for (int c = 0; c < 128; ++c)
                acc[c] = 0.0f;
            float next = sa[0] * sb[0];
            for (int kb = 0; kb < a.kb; ++kb, ++blocks) {
                const float scale = next;
                if (kb + 1 < a.kb)
                    next = sa[kb + 1] * sb[kb + 1];
                const uint32_t b = blocks & 1;
                ok = __all_sync(0xFFFFFFFFu,
                                mbar_wait(acc_full + 8 * b, (blocks >> 1) & 1, abort, a.status));
                if (!ok)
                    break;
                fence_after();
                uint32_t v[2][16];
                tmem_load(lanes + b * kRowsN, v[0]);
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    tmem_wait(v[c & 1]);
                    if (c < 7)
                        tmem_load(lanes + b * kRowsN + (c + 1) * 16, v[(c + 1) & 1]);
                    else {
                        fence_before();
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(acc_empty + 8 * b);
                    }
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        acc[c * 16 + j] += scale * __uint_as_float(v[c & 1][j]);
                }
            }
            if (ok && here)
                store_row(a, t.row + r, n, acc);
            __syncwarp();
        }
        __syncwarp();
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (*abort) {
        if (threadIdx.x == 8 * 32)
            drain_loads(full, used, kRowsStages);
        if (threadIdx.x == 9 * 32) {
            mma_commit(smem_addr(&sh.drain));
            mbar_drain(smem_addr(&sh.drain), 0);
        }
        __syncthreads();
    }
    if (warp == 9)
        tmem_free<512>(tmem);
}

// ---- few rows -------------------------------------------------------------------

constexpr int kFewEpilogueWarps = 4;
constexpr int kFewThreads = 32 * (kFewEpilogueWarps + 2);
constexpr int kFewWeights = 128 * 128;            // bytes of a stage's weights

// NT: rows of a per tile.  Two CTAs per SM share its shared and tensor memory.
template <int NT> struct Few {
    static constexpr int kStage = kFewWeights + NT * 128;
    static constexpr int kStages = NT <= 32 ? 5 : NT == 64 ? 4 : 3;
    static constexpr int kAccs = NT <= 32 ? 4 : 2;
    static constexpr int kCols = NT * kAccs < 32 ? 32 : NT * kAccs;
    static_assert(kCols <= 256, "two CTAs' accumulators share 512 columns");
    static_assert(kStages * kStage >= NT * 512, "the joined sums reuse the stages");
};
template <int NT> struct FewShared {
    uint64_t full[Few<NT>::kStages], empty[Few<NT>::kStages];
    uint64_t acc_full[Few<NT>::kAccs], acc_empty[Few<NT>::kAccs], drain;
    uint32_t tmem;
    int abort;
    alignas(16) float scale[kFewEpilogueWarps][2][NT];
};
template <int NT> constexpr size_t few_smem() {
    return 1024 + (size_t)Few<NT>::kStages * Few<NT>::kStage + sizeof(FewShared<NT>);
}

__device__ __forceinline__ float ld_peer_f32(uint32_t local, uint32_t rank) {
    uint32_t remote;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(remote) : "memory");
    return v;
}

// blockIdx.x: CTA of the cluster (its share of the blocks along k);
// blockIdx.y: tile of 128 weight rows; blockIdx.z: row tile, counted over the
// groups.  Warps 0-3: epilogue, lane + 32 * warp is the weight row; warp 4:
// TMA; warp 5: MMA.
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

    kernel_prologue();
    int group = 0;
    uint32_t row = 0, rows = 0;
    // the same answer in the whole cluster, before any barrier
    if (!find_rows(a, NT, blockIdx.z, group, row, rows))
        return;
    if (threadIdx.x == 0) {
        for (int s = 0; s < F::kStages; ++s) {
            mbar_init(full + 8 * s, 1);
            mbar_init(empty + 8 * s, 1);
        }
        for (int b = 0; b < F::kAccs; ++b) {
            mbar_init(acc_full + 8 * b, 1);
            mbar_init(acc_empty + 8 * b, kFewEpilogueWarps);
        }
        mbar_init(smem_addr(&sh.drain), 1);
        sh.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 5)
        tmem_alloc<F::kCols>(&sh.tmem);
    fence_before();
    __syncthreads();
    fence_after();
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
        if (lane == 0) {
            for (int kb = kb0; kb < kb1; ++kb, ++used) {
                const uint32_t s = used % F::kStages, turn = used / F::kStages;
                const uint32_t b = used % F::kAccs, round = used / F::kAccs;
                if (round > 0 && !mbar_wait(acc_empty + 8 * b, (round - 1) & 1, abort, a.status))
                    break;
                if (!mbar_wait(full + 8 * s, turn & 1, abort, a.status))
                    break;
                fence_after();
                const uint32_t at = smem_addr(stages) + s * F::kStage;
                mma_block(tmem + b * NT, at, at + kFewWeights, mma_shape(128, NT));
                mma_commit(empty + 8 * s);
                mma_commit(acc_full + 8 * b);
            }
        }
        __syncwarp();
    } else {
        const uint32_t lanes = tmem + ((uint32_t)warp * 32 << 16);
        const float *sb = a.sb + group * a.sb_group + (uint64_t)(n0 / 128) * a.kb;
        constexpr int kPer = (NT + 31) / 32;
        // lane l brings the scales of rows l, l + 32, ... one block ahead
        const float *sa[kPer];
        float next[kPer];
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const uint32_t r = lane + 32 * j;
            sa[j] = a.sa + (uint64_t)(r < rows ? row + r : row) * a.sa_row;
            next[j] = kb0 < kb1 ? sa[j][kb0] * sb[kb0] : 0.0f;
        }
#pragma unroll
        for (int c = 0; c < NT; ++c)
            acc[c] = 0.0f;
        for (int kb = kb0; kb < kb1; ++kb, ++used) {
            float *scale = sh.scale[warp][used & 1];
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                if (lane + 32 * j < NT)
                    scale[lane + 32 * j] = next[j];
            __syncwarp();
            if (kb + 1 < kb1)
#pragma unroll
                for (int j = 0; j < kPer; ++j)
                    next[j] = sa[j][kb + 1] * sb[kb + 1];
            const uint32_t b = used % F::kAccs;
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(acc_full + 8 * b, (used / F::kAccs) & 1, abort,
                                                   a.status)))
                break;
            fence_after();
            uint32_t v[2][16];
            tmem_load(lanes + b * NT, v[0]);
#pragma unroll
            for (int c = 0; c < NT / 16; ++c) {
                tmem_wait(v[c & 1]);
                if (c + 1 < NT / 16)
                    tmem_load(lanes + b * NT + (c + 1) * 16, v[(c + 1) & 1]);
                else {
                    fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(acc_empty + 8 * b);
                }
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(scale + c * 16 + j);
                    acc[c * 16 + j] += f.x * __uint_as_float(v[c & 1][j]);
                    acc[c * 16 + j + 1] += f.y * __uint_as_float(v[c & 1][j + 1]);
                    acc[c * 16 + j + 2] += f.z * __uint_as_float(v[c & 1][j + 2]);
                    acc[c * 16 + j + 3] += f.w * __uint_as_float(v[c & 1][j + 3]);
                }
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
        if (threadIdx.x == 5 * 32) {
            mma_commit(smem_addr(&sh.drain));
            mbar_drain(smem_addr(&sh.drain), 0);
        }
        __syncthreads();
    }
    if (warp == 5)
        tmem_free<F::kCols>(tmem);
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
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (warp < kFewEpilogueWarps)
        for (uint32_t c = part; c < rows; c += parts) {
            float v = 0.0f;
            for (int p = 0; p < parts; ++p)
                v += ld_peer_f32(smem_addr(sums + c * 128 + threadIdx.x), p);
            if (n < a.N)
                store_out(a.d + (uint64_t)(row + c) * a.ldd, n, v, a.out);
        }
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
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

// SMs of the current device (asked once per device).
int sm_count() {
    static std::atomic<int> known[64];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0)
        return 0;
    if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0)
        return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    if (dev < 64)
        known[dev].store(n, std::memory_order_relaxed);
    return n;
}

template <int NT>
cudaError_t launch_few(const MatmulArgs &a, int parts, cudaStream_t s) {
    CUtensorMap ma, mb;
    if (!encode(&ma, a.a, a.K, a.M, a.lda, 0, NT) ||
        !encode(&mb, a.b, a.K, a.N, a.ldb, a.E, 128))
        return cudaErrorInvalidValue;
    const cudaError_t e = cudaFuncSetAttribute(
        k_matmul8_few<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)few_smem<NT>());
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
    if (!encode(&ma, a.a, a.K, a.M, a.lda, 0, kRowsM) ||
        !encode(&mb, a.b, a.K, a.N, a.ldb, a.E, kRowsN))
        return cudaErrorInvalidValue;
    const cudaError_t e = cudaFuncSetAttribute(
        k_matmul8_rows, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRowsSmem);
    if (e != cudaSuccess)
        return e;
    return launch_kernel(k_matmul8_rows, sms, kRowsThreads, kRowsSmem, s, true, a, ma, mb);
}

}  // namespace

bool matmul8_tc_ready() { return encoder() != nullptr; }

cudaError_t launch_matmul8_tc(const MatmulArgs &a, cudaStream_t s) {
    const int sms = sm_count();
    if (sms < 1)
        return cudaErrorUnknown;
    const uint64_t groups = (uint64_t)a.E < a.M ? a.E : a.M;
    const uint64_t per = (a.M + groups - 1) / groups;              // rows per group, on average
    const uint64_t tiles = (a.offsets ? a.M / kRowsM + groups : (a.M + kRowsM - 1) / kRowsM) *
                           ((a.N + kRowsN - 1) / kRowsN);
    const uint64_t columns = (a.N + 127) / 128;
    // the grid's y and z dimensions of the form for few rows end at 65535
    if (tiles >= (uint64_t)sms || columns > 65535 || a.M / 16 + groups > 65535)
        return launch_rows(a, sms, s);
    // as many CTAs along k as keep the SMs at two CTAs each
    const int nt = per <= 16 ? 16 : per <= 32 ? 32 : per <= 64 ? 64 : 128;
    const uint64_t ctas = (a.offsets ? a.M / nt + groups : (a.M + nt - 1) / nt) * columns;
    int parts = 1;
    while (parts < 8 && ctas * parts * 2 <= 2 * (uint64_t)sms && parts * 2 <= a.kb)
        parts *= 2;
    switch (nt) {
    case 16: return launch_few<16>(a, parts, s);
    case 32: return launch_few<32>(a, parts, s);
    case 64: return launch_few<64>(a, parts, s);
    default: return launch_few<128>(a, parts, s);
    }
}

}  // namespace ar
