// Product of E4M3 rows with E4M3 weights, with a scale for each block of 128:
//
//   d[m][n] = round( sum_kb sa[m][kb] * sb[e][n / 128][kb] *
//                    sum_{k in kb} a[m][k] * b[e][n][k] )
//
// for one matrix, or for E of them, the rows of a grouped by matrix through
// offsets that only the device knows.
#include <cuda_fp8.h>

#include "ar_matmul8.cuh"

namespace ar {

// ---- general form ------------------------------------------------------------
// Any alignment.  64 x 64 of d per CTA, 4 x 4 a thread, the operands of 32
// steps along k in shared memory as binary32.  Bound by the shared-memory
// reads of the multiply-adds: 4096 x 4096 x 4095 4949 us (27.8 TFLOP/s; 69 us with
// padded rows, by the tensor cores); 1 x 8192 x 8191 1026 us (10.6).
constexpr int kAnyTile = 64, kAnyStep = 32;

__global__ void __launch_bounds__(256) k_matmul8_any(const __grid_constant__ MatmulArgs a) {
    __shared__ alignas(16) float as[kAnyStep][kAnyTile + 4];
    __shared__ alignas(16) float bs[kAnyStep][kAnyTile + 4];
    // the products' loop reads four at a time
    static_assert(__alignof__(as) >= sizeof(float4) && __alignof__(bs) >= sizeof(float4),
                  "operands in shared memory start on 16-byte boundaries");
    static_assert((kAnyTile + 4) % 4 == 0, "and so does every step of them");
    kernel_prologue();
    int e;
    uint32_t row, rows;
    const uint32_t ntiles = (a.N + kAnyTile - 1) / kAnyTile;
    if (!find_rows(a, kAnyTile, blockIdx.x / ntiles, e, row, rows))
        return;
    const uint32_t n0 = blockIdx.x % ntiles * kAnyTile;
    const uint8_t *b = a.b + (uint64_t)e * a.N * a.ldb;
    const float *sb = a.sb + (uint64_t)e * a.sb_group;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    for (int kb = 0; kb < a.kb; ++kb) {
        float part[4][4] = {};
        for (uint32_t k0 = kb * 128u; k0 < kb * 128u + 128u && k0 < a.K; k0 += kAnyStep) {
            __syncthreads();
            for (int i = threadIdx.x; i < kAnyTile * kAnyStep; i += 256) {
                const uint32_t r = i / kAnyStep, k = i % kAnyStep;
                __nv_fp8_e4m3 x, y;
                x.__x = y.__x = 0;
                if (k0 + k < a.K) {
                    if (r < rows)
                        x.__x = a.a[(uint64_t)(row + r) * a.lda + k0 + k];
                    if (n0 + r < a.N)
                        y.__x = b[(uint64_t)(n0 + r) * a.ldb + k0 + k];
                }
                as[k][r] = (float)x;
                bs[k][r] = (float)y;
            }
            __syncthreads();
#pragma unroll 8
            for (int k = 0; k < kAnyStep; ++k) {
                const float4 x = *reinterpret_cast<const float4 *>(&as[k][ty * 4]);
                const float4 y = *reinterpret_cast<const float4 *>(&bs[k][tx * 4]);
                const float xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        part[i][j] += xs[i] * ys[j];
            }
        }
        // a thread's four columns lie in one block of 128 (the tile starts at
        // a multiple of 64)
        const uint32_t n = n0 + tx * 4;
        const float w = n < a.N ? sb[(uint64_t)(n / 128) * a.kb + kb] : 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t r = ty * 4 + i;
            const float s = r < rows ? a.sa[(uint64_t)(row + r) * a.sa_row + kb] * w : 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[i][j] += s * part[i][j];
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t r = ty * 4 + i, n = n0 + tx * 4 + j;
            if (r < rows && n < a.N)
                store_out(a.d + (uint64_t)(row + r) * a.ldd, n, acc[i][j], a.out);
        }
}

static cudaError_t launch_any(const MatmulArgs &a, cudaStream_t s, bool *too_large) {
    const uint64_t tiles = (uint64_t)a.M / kAnyTile + (a.offsets ? a.E : 1);
    const uint64_t grid = tiles * ((a.N + kAnyTile - 1) / kAnyTile);
    *too_large = grid >= (1ull << 31);
    if (*too_large)
        return cudaSuccess;
    return launch_kernel(k_matmul8_any, (int)grid, 256, 0, s, true, a);
}

}  // namespace ar

using namespace ar;

extern "C" {

int ar_matmul8(const void *a, size_t lda, const float *sa, const void *b, size_t ldb,
               const float *sb, const int32_t *offsets, int E, void *d, size_t ldd, size_t M,
               size_t N, size_t K, int out_dtype, int *status, cudaStream_t stream) {
    if (!float_dtype(out_dtype) || N < 1 || K < 1 || E < 1 || (!offsets && E != 1) ||
        (uintptr_t)status % 4 != 0)
        return AR_ERR_INVALID;
    const size_t most = ((size_t)1 << 31) - 256;
    if (M >= most || N >= most || K >= most || E > AR_MOE_MAX_EXPERTS)
        return AR_ERR_UNSUPPORTED;
    if (M == 0)
        return AR_OK;
    if (!a || !sa || !b || !sb || !d)
        return AR_ERR_INVALID;
    const size_t nb = (N - 1) / AR_SCALE_BLOCK + 1, kb = (K - 1) / AR_SCALE_BLOCK + 1;
    const Matrix ma = matrix(a, lda, M, K, 1), mb = matrix(b, ldb, (size_t)E * N, K, 1);
    const Matrix md = matrix(d, ldd, M, N, elem_size(out_dtype));
    const Matrix ms = matrix(sa, 0, M, kb, 4), mt = matrix(sb, 0, (size_t)E * nb, kb, 4);
    const Matrix mo = matrix(offsets, 0, 1, (size_t)E + 1, 4), mu = matrix(status, 0, 1, 1, 4);
    if (!ma.ok || !mb.ok || !md.ok || !ms.ok || !mt.ok || !mo.ok || meet(md, ma) || meet(md, mb) ||
        meet(md, ms) || meet(md, mt) || meet(md, mo) || meet(md, mu))
        return AR_ERR_INVALID;
    MatmulArgs g;
    g.a = static_cast<const uint8_t *>(a);
    g.b = static_cast<const uint8_t *>(b);
    g.sa = sa;
    g.sb = sb;
    g.offsets = offsets;
    g.d = static_cast<uint8_t *>(d);
    g.sa_row = kb;
    g.sb_group = nb * kb;
    g.lda = ma.stride;
    g.ldb = mb.stride;
    g.ldd = md.stride;
    g.M = (uint32_t)M;
    g.N = (uint32_t)N;
    g.K = (uint32_t)K;
    g.E = E;
    g.kb = (int)kb;
    g.out = out_dtype;
    g.sa_wide = wide(ms);
    g.dwide = wide(md);
    g.status = status;
    if (wide(ma) && wide(mb)) {
        if (!matmul8_tc_ready())
            return AR_ERR_CUDA;
        return launched(launch_matmul8_tc(g, stream));
    }
    bool too_large = false;
    const int rc = launched(launch_any(g, stream, &too_large));
    return too_large ? AR_ERR_UNSUPPORTED : rc;
}

}  // extern "C"
