// Root-mean-square norm with the residual's addition, and its gradient.
//
//   v = x + res,  r = 1 / sqrt(mean(v^2) + eps),  y = v * r * gamma
//   dx = r * (gamma*dy - n * mean(gamma*dy*n)) + dsum,  dgamma = sum_t dy * n,
//   n = s * r
//
// Both are bound by memory: a row is read once, kept in registers across the
// row's reduction, and written once; the units beyond what the registers hold
// (rows past 2048 units: 16384 elements of a two-byte type) are read a second
// time.  8192 x 8192 bf16 with a residual to 8 bits: 74.5 us (6.3 TB/s); the
// gradient 96 us (5.6 TB/s; issue and the barriers between rows are the rest).
#include "ar_rows.cuh"

namespace ar {

struct NormArgs {
    const uint8_t *x, *res;
    const void *gamma;
    uint8_t *sum, *y;
    float *scale, *rstd;
    uint64_t sx, sres, ssum, sy;      // bytes between rows
    uint64_t T;
    uint32_t H;
    float eps;
};

// Two binary32 values to two E4M3 codes, `a` in the low byte; nearest even,
// saturating, NaN to the NaN code.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
    uint16_t q;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(q) : "f"(b), "f"(a));
    return q;
}

// A block's largest magnitude counts as at least this, so that neither the
// scale nor its reciprocal leaves the range of normal numbers.
constexpr float kLeastBlock = 0x1p-96f;
constexpr float kTopE4M3 = 448.0f;

// Whether a thread for each unit no longer fits the SMs at once.
static bool many_units(uint64_t rows, uint32_t units) {
    return rows > (uint64_t)sm_count() * 1024 / units;
}

// The unit's share of y in 8 bits, and its block's scale.  Called by whole warps.
// Both quotients are products with a rounded reciprocal: correctly rounded
// divisions cost an instruction sequence for every element (8192 x 8192 bf16: 94 us
// against 75) and change only codes whose value lies on the middle between two.
template <int DT, bool WIDE>
__device__ __forceinline__ void store_e4m3(uint8_t *row, float *scales, uint32_t u, uint32_t H,
                                           const float *v) {
    using L = Rows<DT, WIDE>;
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < L::E; ++i)
        m = fmaxf(m, fabsf(v[i]));
#pragma unroll
    for (int d = L::kBlockLanes / 2; d > 0; d >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
    const float scale = fmaxf(m, kLeastBlock) * (1.0f / kTopE4M3);
    const float inv = __frcp_rn(scale);
    if (L::at(u, 0) >= H)
        return;
    if (u % L::kBlockLanes == 0)
        scales[u / L::kBlockLanes] = scale;
    uint32_t q[(L::E + 3) / 4];
#pragma unroll
    for (int i = 0; i < L::E; i += 4) {
        float t[4] = {v[i], v[i + 1], v[i + 2], v[i + 3]};
        mul2(t, inv, inv);
        mul2(t + 2, inv, inv);
        q[i / 4] = e4m3x2(t[0], t[1]) | e4m3x2(t[2], t[3]) << 16;
    }
    if (L::whole(u, H)) {
        if (L::E == 8)
            reinterpret_cast<uint2 *>(row)[u] = make_uint2(q[0], q[L::E / 4 - 1]);
        else
            reinterpret_cast<uint32_t *>(row)[u] = q[0];
        return;
    }
#pragma unroll
    for (int i = 0; i < L::E; ++i)
        if (L::at(u, i) < H)
            row[L::at(u, i)] = (uint8_t)(q[i / 4] >> (8 * (i & 3)));
}

// One CTA, or one warp, per row.  UNITS units of a thread stay in registers.
// Every loop over units has the same trip count in a whole warp (the bound is a
// multiple of 32), which the shuffles of store_e4m3 need.
template <int DT, bool WIDE, bool E4M3, RowSplit SPLIT, int UNITS, int THREADS, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS) k_rmsnorm(const __grid_constant__ NormArgs a) {
    using L = Rows<DT, WIDE>;
    __shared__ float part[32];
    kernel_prologue();
    static_assert(SPLIT != kGroups, "a row has one warp or all of them");
    const RowGroup<SPLIT> group(0);
    const uint32_t H = a.H, units = L::warp_units(H);
    for (uint64_t t = (uint64_t)blockIdx.x * group.groups() + group.g(); t < a.T;
         t += (uint64_t)gridDim.x * group.groups()) {
        const uint8_t *x = a.x + t * a.sx;
        const uint8_t *res = a.res ? a.res + t * a.sres : nullptr;
        uint8_t *sum = a.sum ? a.sum + t * a.ssum : nullptr;
        uint8_t *y = a.y + t * a.sy;
        float *scale = E4M3 ? a.scale + t * ((H + AR_SCALE_BLOCK - 1) / AR_SCALE_BLOCK) : nullptr;

        auto total = [&](uint4 px, uint4 pr, float *b) {     // x + res
            L::widen(px, b);
            if (res) {
                float w[L::E];
                L::widen(pr, w);
#pragma unroll
                for (int i = 0; i < L::E; i += 2)
                    add2(b + i, w[i], w[i + 1]);
            }
        };
        const uint32_t past = group.thread() + UNITS * group.threads();
        float v[UNITS][L::E];
        float squares[2] = {0.0f, 0.0f};
        {
            uint4 px[UNITS], pr[UNITS];
#pragma unroll
            for (int j = 0; j < UNITS; ++j) {
                const uint32_t u = group.thread() + j * group.threads();
                px[j] = pr[j] = make_uint4(0u, 0u, 0u, 0u);
                if (u < units) {
                    px[j] = L::load(x, u, H);
                    if (res)
                        pr[j] = L::load(res, u, H);
                }
            }
#pragma unroll
            for (int j = 0; j < UNITS; ++j) {
                total(px[j], pr[j], v[j]);
#pragma unroll
                for (int i = 0; i < L::E; i += 2)
                    fma2(squares, v[j][i], v[j][i + 1], v[j][i], v[j][i + 1]);
            }
        }
        for (uint32_t u = past; u < units; u += group.threads()) {
            float b[L::E];
            total(L::load(x, u, H), res ? L::load(res, u, H) : make_uint4(0u, 0u, 0u, 0u), b);
#pragma unroll
            for (int i = 0; i < L::E; i += 2)
                fma2(squares, b[i], b[i + 1], b[i], b[i + 1]);
        }
        const float ss = group.sum(squares[0] + squares[1], part);
        const float r = __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(ss, (float)H) + a.eps));
        if (a.rstd && group.thread() == 0)
            a.rstd[t] = r;

        auto finish = [&](uint32_t u, float *b) {
            if (sum)
                L::store(sum, u, H, b);
#pragma unroll
            for (int i = 0; i < L::E; i += 2)
                mul2(b + i, r, r);
            if (a.gamma) {
                float g[L::E];
                L::widen(L::template load<true>(a.gamma, u, H), g);
#pragma unroll
                for (int i = 0; i < L::E; i += 2)
                    mul2(b + i, g[i], g[i + 1]);
            }
            if (E4M3)
                store_e4m3<DT, WIDE>(y, scale, u, H, b);
            else
                L::store(y, u, H, b);
        };
        // the units past the registers: read again, before sum or y overwrites them
        for (uint32_t u = past; u < units; u += group.threads()) {
            float b[L::E];
            total(L::load(x, u, H), res ? L::load(res, u, H) : make_uint4(0u, 0u, 0u, 0u), b);
            finish(u, b);
        }
#pragma unroll
        for (int j = 0; j < UNITS; ++j) {
            const uint32_t u = group.thread() + j * group.threads();
            if (u < units)
                finish(u, v[j]);
        }
        if (SPLIT == kOneRow)
            __syncthreads();                         // `part` is free for the next row
    }
}

template <int DT, bool WIDE, bool E4M3>
static cudaError_t norm_units(const NormArgs &a, cudaStream_t s) {
    const uint32_t units = Rows<DT, WIDE>::warp_units(a.H);
    auto grid = [&](uint64_t rows) {
        const uint64_t g = (a.T + rows - 1) / rows;
        return (int)(g < (1u << 30) ? g : (1u << 30));
    };
    auto threads = [&](uint32_t per, uint32_t most) {
        const uint32_t n = ((units + per - 1) / per + 31) / 32 * 32;
        return (int)(n < most ? n : most);
    };
    // Many units: four a thread, so that an SM holds several CTAs and one row's
    // loads run while another's reduction waits (8192 x 8192 bf16 to 8 bits: 75 us;
    // with one unit a thread 107 to 154; 333 x 4099: 5.0 and 6.1).  Few units: a
    // thread for each, for latency (1000 x 1024: 3.9 us; four a thread 5.6).  Short
    // rows go eight to a CTA, one a warp (65536 x 512: 60 us; one a CTA 68; 4000 x
    // 100: 3.7 and 5.2; but 32768 x 1024: 46 and 41).
    const bool many = many_units(a.T, units);
    if (units <= 64 && a.T > 1024)
        return launch_kernel(k_rmsnorm<DT, WIDE, E4M3, kWarpRow, 4, 256, 4>, grid(8), 256, 0, s,
                             true, a);
    if (many && units <= 1024)
        return launch_kernel(k_rmsnorm<DT, WIDE, E4M3, kOneRow, 4, 256, 4>, grid(1),
                             threads(4, 256), 0, s, true, a);
    if (many)
        return launch_kernel(k_rmsnorm<DT, WIDE, E4M3, kOneRow, 4, 512, 2>, grid(1),
                             threads(4, 512), 0, s, true, a);
    return launch_kernel(k_rmsnorm<DT, WIDE, E4M3, kOneRow, 2, 1024, 1>, grid(1),
                         threads(units <= 1024 ? 1 : 2, 1024), 0, s, true, a);
}

template <int DT>
static cudaError_t norm_dt(const NormArgs &a, bool w, bool e4m3, cudaStream_t s) {
    if (e4m3)
        return w ? norm_units<DT, true, true>(a, s) : norm_units<DT, false, true>(a, s);
    return w ? norm_units<DT, true, false>(a, s) : norm_units<DT, false, false>(a, s);
}

// ---- gradient ----------------------------------------------------------------

struct NormGradArgs {
    const uint8_t *dy, *dsum, *s;
    const void *gamma;
    const float *rstd;
    uint8_t *dx;
    float *work;                      // gridDim.x rows of H partial sums, or NULL
    float *dgamma;
    uint64_t sdy, sdsum, ss, sdx;     // bytes between rows
    uint64_t T;
    uint32_t H;
    int row_warps;                    // warps that share a row
};

// Copy of 16 bytes (or fewer: the rest reads as zero) to shared memory, done
// in the background.
__device__ __forceinline__ void copy_async(uint4 *to, const void *from, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                 :: "r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int LEFT> __device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" :: "n"(LEFT) : "memory");
}

// One element block of the gradient.  With c = r^2 * sum(d * s) / H:
//   d = gamma * dy,  dgamma += dy * (s * r),  dx = r * (d - c * s) + dsum
// (c has the size of r and c * s that of d; r^3 would leave binary32 for rows
// whose own gradient does not).
// Pass 1: d from dy and gamma; the products' sum and dgamma's share.
template <int DT, bool WIDE>
__device__ __forceinline__ float grad_open(const NormGradArgs &a, uint32_t u, uint4 ps, uint4 pd,
                                           float r, float *d, float *dg) {
    using L = Rows<DT, WIDE>;
    float s[L::E], n[L::E], dot[2] = {0.0f, 0.0f};
    L::widen(ps, s);
    L::widen(pd, d);
#pragma unroll
    for (int i = 0; i < L::E; i += 2) {
        n[i] = s[i];
        n[i + 1] = s[i + 1];
        mul2(n + i, r, r);
        fma2(dg + i, d[i], d[i + 1], n[i], n[i + 1]);
    }
    if (a.gamma) {
        float g[L::E];
        L::widen(L::template load<true>(a.gamma, u, a.H), g);
#pragma unroll
        for (int i = 0; i < L::E; i += 2)
            mul2(d + i, g[i], g[i + 1]);
    }
#pragma unroll
    for (int i = 0; i < L::E; i += 2)
        fma2(dot, d[i], d[i + 1], s[i], s[i + 1]);
    return dot[0] + dot[1];
}
// Pass 2.
template <int DT, bool WIDE>
__device__ __forceinline__ void grad_close(const NormGradArgs &a, uint32_t u, uint4 ps, float *d,
                                           uint4 pu, float r, float c, uint8_t *dx) {
    using L = Rows<DT, WIDE>;
    float s[L::E];
    L::widen(ps, s);
#pragma unroll
    for (int i = 0; i < L::E; i += 2) {
        fma2(d + i, -c, -c, s[i], s[i + 1]);
        mul2(d + i, r, r);
    }
    if (a.dsum) {
        float w[L::E];
        L::widen(pu, w);
#pragma unroll
        for (int i = 0; i < L::E; i += 2)
            add2(d + i, w[i], w[i + 1]);
    }
    L::store(dx, u, a.H, d);
}

// A CTA takes a row, or one per group of a.row_warps warps, at a time, then the
// next of every gridDim.x such sets.  Each thread owns the columns of its units
// and keeps their share of dgamma in registers over all of its rows; the groups'
// shares are joined in order at the end.  RING: the next row's s, dy and dsum come to
// shared memory by background copies while this row is at work; a thread copies
// and reads its own units only, so the copies need no barrier.  Without it (rows
// that are not 16-byte aligned, or longer than UNITS units a thread) rows are
// loaded in their turn, and the units past the registers are read twice, their
// dgamma kept in the CTA's row of `work` (one group then).
template <int DT, bool WIDE, RowSplit SPLIT, int UNITS, int THREADS, int CTAS, bool RING>
__global__ void __launch_bounds__(THREADS, CTAS)
k_rmsnorm_grad(const __grid_constant__ NormGradArgs a) {
    using L = Rows<DT, WIDE>;
    extern __shared__ uint4 ring[];               // [2][3][UNITS][THREADS], or the join's sums
    __shared__ float part[2][32];
    kernel_prologue();
    const RowGroup<SPLIT> group(a.row_warps);
    const uint32_t H = a.H;
    float *work = a.work ? a.work + (uint64_t)blockIdx.x * H : nullptr;
    float dg[UNITS][L::E];
#pragma unroll
    for (int j = 0; j < UNITS; ++j)
#pragma unroll
        for (int i = 0; i < L::E; ++i)
            dg[j][i] = 0.0f;
    auto slot = [&](int turn, int array, int j) -> uint4 & {
        return ring[((turn * 3 + array) * UNITS + j) * THREADS + threadIdx.x];
    };
    auto fetch = [&](uint64_t t, int turn) {      // the ring's copies of row t
        if (t < a.T && group.g() < group.groups()) {
            const uint8_t *s = a.s + t * a.ss, *dy = a.dy + t * a.sdy;
            const uint8_t *dsum = a.dsum ? a.dsum + t * a.sdsum : nullptr;
#pragma unroll
            for (int j = 0; j < UNITS; ++j) {
                const uint32_t u = group.thread() + j * group.threads();
                const uint32_t left = u * L::E < H ? (H - u * L::E) * L::kSize : 0u;
                const uint32_t n = left < 16u ? left : 16u;
                const uint64_t at = n ? (uint64_t)u * 16 : 0;
                copy_async(&slot(turn, 0, j), s + at, n);
                copy_async(&slot(turn, 1, j), dy + at, n);
                if (dsum)
                    copy_async(&slot(turn, 2, j), dsum + at, n);
            }
        }
        copies_commit();
    };
    int turn = 0;
    const uint64_t step = (uint64_t)gridDim.x * group.groups();
    if (RING)
        fetch((uint64_t)blockIdx.x * group.groups() + group.g(), 0);
    for (uint64_t t0 = (uint64_t)blockIdx.x * group.groups(); t0 < a.T; t0 += step, turn ^= 1) {
        const bool on = group.g() < group.groups() && t0 + group.g() < a.T;
        const uint64_t t = on ? t0 + group.g() : t0;
        const uint32_t units = on ? L::warp_units(H) : 0u;
        const uint8_t *dy = a.dy + t * a.sdy, *s = a.s + t * a.ss;
        const uint8_t *dsum = a.dsum ? a.dsum + t * a.sdsum : nullptr;
        uint8_t *dx = a.dx + t * a.sdx;
        const float r = a.rstd[t];
        const uint4 none = make_uint4(0u, 0u, 0u, 0u);
        const uint32_t past = group.thread() + UNITS * group.threads();
        float dot = 0.0f;
        uint4 ps[UNITS], pd[UNITS], pu[UNITS];
        float d[UNITS][L::E];
        if (RING) {
            fetch(t0 + step + group.g(), turn ^ 1);
            copies_wait<1>();
#pragma unroll
            for (int j = 0; j < UNITS; ++j) {
                ps[j] = slot(turn, 0, j);
                pd[j] = slot(turn, 1, j);
            }
        } else {
#pragma unroll
            for (int j = 0; j < UNITS; ++j) {
                const uint32_t u = group.thread() + j * group.threads();
                ps[j] = pd[j] = pu[j] = none;
                if (u < units) {
                    ps[j] = L::load(s, u, H);
                    pd[j] = L::load(dy, u, H);
                    if (dsum)
                        pu[j] = L::load(dsum, u, H);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < UNITS; ++j) {
            const uint32_t u = group.thread() + j * group.threads();
            if (u < units)
                dot += grad_open<DT, WIDE>(a, u, ps[j], pd[j], r, d[j], dg[j]);
        }
        if (!RING)
            for (uint32_t u = past; u < units; u += group.threads()) {
                float e[L::E], w[L::E];
#pragma unroll
                for (int i = 0; i < L::E; ++i)
                    w[i] = work && L::at(u, i) < H && t != blockIdx.x ? work[L::at(u, i)] : 0.0f;
                dot += grad_open<DT, WIDE>(a, u, L::load(s, u, H), L::load(dy, u, H), r, e, w);
#pragma unroll
                for (int i = 0; i < L::E; ++i)
                    if (work && L::at(u, i) < H)
                        work[L::at(u, i)] = w[i];
            }
        const float c = __fdiv_rn(group.sum(dot, part[turn]) * r * r, (float)H);
#pragma unroll
        for (int j = 0; j < UNITS; ++j) {
            const uint32_t u = group.thread() + j * group.threads();
            if (u < units)
                grad_close<DT, WIDE>(a, u, ps[j], d[j], RING ? slot(turn, 2, j) : pu[j], r, c, dx);
        }
        if (!RING)
            for (uint32_t u = past; u < units; u += group.threads()) {
                float e[L::E], w[L::E];
                const uint4 s4 = L::load(s, u, H);
                grad_open<DT, WIDE>(a, u, s4, L::load(dy, u, H), r, e, w);
                grad_close<DT, WIDE>(a, u, s4, e, dsum ? L::load(dsum, u, H) : none, r, c, dx);
            }
    }
    if (!work)
        return;
    if (SPLIT == kOneRow) {
        const bool vectors = (uintptr_t)work % 16 == 0;
#pragma unroll
        for (int j = 0; j < UNITS; ++j) {
            const uint32_t u = group.thread() + j * group.threads();
            if (L::whole(u, H) && vectors) {
#pragma unroll
                for (int i = 0; i < L::E; i += 4)
                    *reinterpret_cast<float4 *>(work + L::at(u, i)) =
                        make_float4(dg[j][i], dg[j][i + 1], dg[j][i + 2], dg[j][i + 3]);
                continue;
            }
#pragma unroll
            for (int i = 0; i < L::E; ++i)
                if (L::at(u, i) < H && u < L::warp_units(H))
                    work[L::at(u, i)] = dg[j][i];
        }
        return;
    }
    float *sums = reinterpret_cast<float *>(ring);        // [groups][H]
    __syncthreads();                                      // the ring is done with
    if (group.g() < group.groups())
#pragma unroll
        for (int j = 0; j < UNITS; ++j) {
            const uint32_t u = group.thread() + j * group.threads();
#pragma unroll
            for (int i = 0; i < L::E; ++i)
                if (L::at(u, i) < H && u < L::warp_units(H))
                    sums[(uint32_t)group.g() * H + L::at(u, i)] = dg[j][i];
        }
    __syncthreads();
    for (uint32_t h = threadIdx.x; h < H; h += blockDim.x) {
        float v = sums[h];
        for (int g = 1; g < group.groups(); ++g)
            v += sums[(uint32_t)g * H + h];
        work[h] = v;
    }
}

// dgamma[h] = sum of the G partial rows, a fixed tree: 32 columns a CTA, thread
// row y adds the rows y, y + TY, ... and the TY sums of a column are then joined.
template <int TY>
__global__ void __launch_bounds__(32 * TY)
k_join_rows(const float *work, float *out, uint64_t H, int G) {
    __shared__ float part[TY][33];
    kernel_prologue();
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const uint64_t h = (uint64_t)blockIdx.x * 32 + x;
    float v = 0.0f;
    if (h < H)
#pragma unroll 4
        for (int g = y; g < G; g += TY)
            v += work[(uint64_t)g * H + h];
    part[y][x] = v;
    __syncthreads();
    // warp y joins columns y, y + TY, ...
    for (int c = y; c < 32; c += TY) {
        v = warp_sum(x < TY ? part[x][c] : 0.0f);
        const uint64_t col = (uint64_t)blockIdx.x * 32 + c;
        if (x == 0 && col < H)
            out[col] = v;
    }
}

static cudaError_t join_rows(const float *work, float *out, uint64_t H, int G, cudaStream_t s) {
    const dim3 grid((unsigned)((H + 31) / 32));
    return G > 32 ? launch_kernel(k_join_rows<32>, grid, 1024, 0, s, true, work, out, H, G)
                  : launch_kernel(k_join_rows<8>, grid, 256, 0, s, true, work, out, H, G);
}

// Launches the gradient's form with these numbers and at most `most` CTAs;
// *partial: rows of `work` it fills.
template <int DT, bool WIDE, RowSplit SPLIT, int UNITS, int THREADS, int CTAS, bool RING>
static cudaError_t norm_grad_form(NormGradArgs a, int most, cudaStream_t s, int *partial) {
    using L = Rows<DT, WIDE>;
    constexpr auto kernel = k_rmsnorm_grad<DT, WIDE, SPLIT, UNITS, THREADS, CTAS, RING>;
    // the ring's six arrays; the join needs no more than THREADS * UNITS * E floats
    constexpr size_t join = SPLIT == kGroups ? (size_t)UNITS * THREADS * L::E * sizeof(float) : 0;
    constexpr size_t smem = RING ? (size_t)6 * UNITS * THREADS * sizeof(uint4) : join;
    static_assert(smem >= join, "room for the join");
    const cudaError_t e = opt_in_smem<kernel>(smem);
    if (e != cudaSuccess)
        return e;
    const uint32_t units = L::warp_units(a.H);
    a.row_warps = (int)((units / 32 + UNITS - 1) / UNITS);
    const int groups = SPLIT == kGroups ? THREADS / 32 / a.row_warps : 1;
    const uint64_t sets = (a.T + groups - 1) / groups;
    *partial = (int)(sets < (uint64_t)most ? sets : most);
    if (*partial == 1 && a.work)
        a.work = a.dgamma;
    const int few = units < THREADS ? (int)units : THREADS;
    return launch_kernel(kernel, *partial, SPLIT == kGroups ? THREADS : few, smem, s, true, a);
}

template <int DT, bool WIDE>
static cudaError_t norm_grad_units(const NormGradArgs &a, cudaStream_t s, int *partial) {
    const uint32_t units = Rows<DT, WIDE>::warp_units(a.H);
    // Few units: a CTA per row, no ring, for latency (one row of 8192 bf16: 3.8 us;
    // with the ring 6.3; 300 x 4096: 7.1 and 10.9).
    // Units of eight elements need twice the registers, so two of them a thread.
    constexpr int kUnits = Rows<DT, WIDE>::E / 4, kThreads = 1024 / kUnits;
    const bool few = !many_units(a.T, units);
    if (few && units <= 1024)
        return norm_grad_form<DT, WIDE, kOneRow, kUnits, kThreads, 1, false>(a, AR_NORM_GRAD_ROWS,
                                                                              s, partial);
    if (few && units <= 2048)
        return norm_grad_form<DT, WIDE, kOneRow, 2 * kUnits, kThreads, 1, false>(
            a, AR_NORM_GRAD_ROWS, s, partial);
    // One or two CTAs an SM, each with a row of partial sums.
    const int sms = sm_count(), most = 2 * sms < AR_NORM_GRAD_ROWS ? 2 * sms : AR_NORM_GRAD_ROWS;
    if (sms < 1)
        return cudaErrorUnknown;
    // With the ring, two CTAs an SM (8192 x 8192 bf16: 96 us; one CTA 120, without
    // the ring 124).  Rows that fill half a CTA or less go side by side
    // (32768 x 1024: 57 us; one a CTA 195).
    if constexpr (WIDE) {
        if (units <= 512)
            return norm_grad_form<DT, WIDE, kGroups, 2, 512, 2, true>(a, most, s, partial);
        if (units <= 1024)
            return norm_grad_form<DT, WIDE, kOneRow, 2, 512, 2, true>(a, most, s, partial);
    } else {
        if (units <= 512)
            return norm_grad_form<DT, WIDE, kGroups, 4, 256, 2, false>(a, most, s, partial);
        if (units <= 1024)
            return norm_grad_form<DT, WIDE, kOneRow, 4, 256, 2, false>(a, most, s, partial);
    }
    return norm_grad_form<DT, WIDE, kOneRow, 4, 512, 1, false>(a, most / 2, s, partial);
}

template <int DT>
static cudaError_t norm_grad_dt(const NormGradArgs &a, bool w, cudaStream_t s, int *partial) {
    return w ? norm_grad_units<DT, true>(a, s, partial) : norm_grad_units<DT, false>(a, s, partial);
}

}  // namespace ar

using namespace ar;

extern "C" {

int ar_rmsnorm(const void *x, size_t ldx, const void *res, size_t ldres, const void *gamma,
               float eps, void *sum, size_t ldsum, void *y, size_t ldy, float *scale,
               float *rstd, size_t T, size_t H, int dtype, int out_dtype, cudaStream_t stream) {
    const bool e4m3 = out_dtype == AR_E4M3;
    if (!float_dtype(dtype) || !(e4m3 || out_dtype == dtype) || H < 1 || !(eps >= 0.0f) ||
        e4m3 != (scale != nullptr))
        return AR_ERR_INVALID;
    if (H >= (size_t)1 << 31)
        return AR_ERR_UNSUPPORTED;
    if (T == 0)
        return AR_OK;
    if (!x || !y)
        return AR_ERR_INVALID;
    const size_t esz = elem_size(dtype), nb = (H - 1) / AR_SCALE_BLOCK + 1;
    const Matrix mx = matrix(x, ldx, T, H, esz), mr = matrix(res, ldres, T, H, esz);
    const Matrix mg = matrix(gamma, 0, 1, H, esz);
    const Matrix ms = matrix(sum, ldsum, T, H, esz), my = matrix(y, ldy, T, H, e4m3 ? 1 : esz);
    const Matrix mc = matrix(scale, 0, T, nb, 4), mt = matrix(rstd, 0, T, 1, 4);
    if (!mx.ok || !mr.ok || !mg.ok || !ms.ok || !my.ok || !mc.ok || !mt.ok)
        return AR_ERR_INVALID;
    if (clash(ms, mx) || clash(ms, mr) || meet(ms, mg) || meet(ms, my) || meet(my, mg) ||
        (e4m3 ? meet(my, mx) || meet(my, mr) : clash(my, mx) || clash(my, mr)))
        return AR_ERR_INVALID;
    const Matrix *all[] = {&mx, &mr, &mg, &ms, &my};
    for (const Matrix *m : all)
        if (meet(mc, *m) || meet(mt, *m))
            return AR_ERR_INVALID;
    if (meet(mc, mt))
        return AR_ERR_INVALID;
    NormArgs a;
    a.x = static_cast<const uint8_t *>(x);
    a.res = static_cast<const uint8_t *>(res);
    a.gamma = gamma;
    a.sum = static_cast<uint8_t *>(sum);
    a.y = static_cast<uint8_t *>(y);
    a.scale = scale;
    a.rstd = rstd;
    a.sx = mx.stride;
    a.sres = mr.stride;
    a.ssum = ms.stride;
    a.sy = my.stride;
    a.T = T;
    a.H = (uint32_t)H;
    a.eps = eps;
    const bool w = wide(mx) && (!res || wide(mr)) && mg.p % 16 == 0 && (!sum || wide(ms)) &&
                   wide(my, e4m3 ? 16 / esz : 16);
    switch (dtype) {
    case AR_BF16: return launched(norm_dt<AR_BF16>(a, w, e4m3, stream));
    case AR_FP16: return launched(norm_dt<AR_FP16>(a, w, e4m3, stream));
    default: return launched(norm_dt<AR_FP32>(a, w, e4m3, stream));
    }
}

int ar_rmsnorm_grad(const void *dy, size_t lddy, const void *dsum, size_t lddsum, const void *s,
                    size_t lds, const void *gamma, const float *rstd, void *dx, size_t lddx,
                    float *dgamma, float *work, size_t work_bytes, size_t T, size_t H, int dtype,
                    cudaStream_t stream) {
    if (!float_dtype(dtype) || H < 1 || (uintptr_t)dgamma % 4 != 0)
        return AR_ERR_INVALID;
    if (H >= (size_t)1 << 31)
        return AR_ERR_UNSUPPORTED;
    if (T == 0) {
        if (!dgamma)
            return AR_OK;
        return launched(join_rows(nullptr, dgamma, H, 0, stream));
    }
    if (!dy || !s || !rstd || !dx || (dgamma != nullptr) != (work != nullptr))
        return AR_ERR_INVALID;
    const size_t esz = elem_size(dtype);
    const size_t rows = T < AR_NORM_GRAD_ROWS ? T : AR_NORM_GRAD_ROWS;
    const Matrix my = matrix(dy, lddy, T, H, esz), mu = matrix(dsum, lddsum, T, H, esz);
    const Matrix ms = matrix(s, lds, T, H, esz), mx = matrix(dx, lddx, T, H, esz);
    const Matrix mg = matrix(gamma, 0, 1, H, esz), mt = matrix(rstd, 0, T, 1, 4);
    const Matrix md = matrix(dgamma, 0, 1, H, 4), mw = matrix(work, 0, rows, H, 4);
    if (!my.ok || !mu.ok || !ms.ok || !mx.ok || !mg.ok || !mt.ok || !md.ok || !mw.ok ||
        mw.p % 16 != 0 || (work && work_bytes < mw.bytes))
        return AR_ERR_INVALID;
    if (clash(mx, my) || clash(mx, mu) || clash(mx, ms) || meet(mx, mg) || meet(mx, mt) ||
        meet(mx, md) || meet(mx, mw) || meet(md, mw))
        return AR_ERR_INVALID;
    const Matrix *in[] = {&my, &mu, &ms, &mg, &mt};
    for (const Matrix *m : in)
        if (meet(md, *m) || meet(mw, *m))
            return AR_ERR_INVALID;
    NormGradArgs a;
    a.dy = static_cast<const uint8_t *>(dy);
    a.dsum = static_cast<const uint8_t *>(dsum);
    a.s = static_cast<const uint8_t *>(s);
    a.gamma = gamma;
    a.rstd = rstd;
    a.dx = static_cast<uint8_t *>(dx);
    a.work = work;
    a.dgamma = dgamma;
    a.sdy = my.stride;
    a.sdsum = mu.stride;
    a.ss = ms.stride;
    a.sdx = mx.stride;
    a.T = T;
    a.H = (uint32_t)H;
    const bool w = wide(my) && (!dsum || wide(mu)) && wide(ms) && wide(mx) && mg.p % 16 == 0;
    cudaError_t e;
    int partial = 0;
    switch (dtype) {
    case AR_BF16: e = norm_grad_dt<AR_BF16>(a, w, stream, &partial); break;
    case AR_FP16: e = norm_grad_dt<AR_FP16>(a, w, stream, &partial); break;
    default: e = norm_grad_dt<AR_FP32>(a, w, stream, &partial); break;
    }
    // one partial row is the gradient itself
    if (e == cudaSuccess && dgamma && partial > 1)
        e = join_rows(work, dgamma, H, partial, stream);
    return launched(e);
}

}  // extern "C"
