// What the kernels of the E4M3 product share: its arguments, the walk over the
// groups' row tiles, and the launchers.
#pragma once

#include "ar_rows.cuh"

namespace ar {

struct MatmulArgs {
    const uint8_t *a, *b;
    const float *sa, *sb;
    const int32_t *offsets;       // NULL: one group, all rows
    uint8_t *d;
    uint64_t sa_row, sb_group;    // scales between rows of a, between matrices of b
    uint64_t lda, ldb, ldd;       // bytes between rows
    uint32_t M, N, K;
    int E;
    int kb;                       // blocks along k
    int out;                      // enum ar_dtype
    int sa_wide;                  // rows of sa start on 16-byte boundaries
    int dwide;                    // rows of d start on 16-byte boundaries
    int *status;
};

// The rows [lo, hi) of group e.
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

// Row tile `index` of all groups' tiles of TM rows: its group, first row and
// rows.  Called by a whole warp; false if there are fewer tiles.
__device__ __forceinline__ bool find_rows(const MatmulArgs &a, uint32_t tm, uint32_t index,
                                          int &group, uint32_t &row, uint32_t &rows) {
    if (!a.offsets) {
        const uint64_t r = (uint64_t)index * tm;
        if (r >= a.M)
            return false;
        group = 0;
        row = (uint32_t)r;
        rows = a.M - row < tm ? a.M - row : tm;
        return true;
    }
    const int lane = threadIdx.x & 31;
    uint32_t base = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
        const int e = e0 + lane;
        uint32_t lo = 0, hi = 0;
        if (e < a.E)
            group_range(a, e, lo, hi);
        const uint32_t tiles = (hi - lo + tm - 1) / tm;
        uint32_t scan = tiles;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, scan, d);
            scan += lane >= d ? v : 0u;
        }
        const uint32_t hit = __ballot_sync(0xFFFFFFFFu, base + scan > index);
        if (hit) {
            const int l = __ffs(hit) - 1;
            const uint32_t first = __shfl_sync(0xFFFFFFFFu, base + scan - tiles, l);
            const uint32_t start = __shfl_sync(0xFFFFFFFFu, lo, l);
            const uint32_t end = __shfl_sync(0xFFFFFFFFu, hi, l);
            group = e0 + l;
            row = start + (index - first) * tm;
            rows = end - row < tm ? end - row : tm;
            return true;
        }
        base = __shfl_sync(0xFFFFFFFFu, base + scan, 31);
    }
    return false;
}

__device__ __forceinline__ void store_out(uint8_t *row, uint32_t n, float v, int out) {
    if (out == AR_BF16)
        reinterpret_cast<uint16_t *>(row)[n] = (uint16_t)narrow1<AR_BF16>(v);
    else if (out == AR_FP16)
        reinterpret_cast<uint16_t *>(row)[n] = (uint16_t)narrow1<AR_FP16>(v);
    else
        reinterpret_cast<float *>(row)[n] = v;
}

// ar_matmul8_tc.cu.  Both need 16-byte aligned a and b with row strides that
// are multiples of 16 bytes.
bool matmul8_tc_ready();          // the tensor-map encoder was found
cudaError_t launch_matmul8_tc(const MatmulArgs &a, cudaStream_t s);

}  // namespace ar
