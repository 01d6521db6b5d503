// Tokens sorted by expert and back, with weights applied, and the gradients.
//
//   route:    row(t, k) = offsets[id] + number of earlier pairs with the same id
//   dispatch: rows[row(t, k)] = x[t]
//   return:   out[t] = round(fold_k w[t, k] * rows[row(t, k)])
//   gradient: drows[row(t, k)] = round(w[t, k] * dout[t]),
//             dw[t, k] = sum_h dout[t][h] * rows[row(t, k)][h]
//
// The row movers go by token, not by row: a token's row is read once and
// written K times (dispatch, gradient), or K rows are read and one is written
// (return), so each byte crosses memory once whatever the order.
#include "ar_cluster.cuh"
#include "ar_rows.cuh"

namespace ar {

// ---- the order ---------------------------------------------------------------

struct RouteArgs {
    const void *ids;
    int32_t *offsets, *row_of, *src;
    uint32_t n;               // pairs
    int E;
    int wide_ids;             // 8-byte ids
};

constexpr int kRouteCtas = 8;          // CTAs of the one cluster for larger inputs
constexpr int kRouteWarps = 32;
constexpr int kRouteHeld = 8;          // ids a lane keeps in registers

// The expert of pair p, or E for one that is not here.
__device__ __forceinline__ int expert_of(const RouteArgs &a, uint32_t p) {
    const int64_t id = a.wide_ids ? reinterpret_cast<const int64_t *>(a.ids)[p]
                                  : (int64_t) reinterpret_cast<const int32_t *>(a.ids)[p];
    return id >= 0 && id < a.E ? (int)id : a.E;
}

// Stable counting sort in one launch: one CTA, or one cluster of kRouteCtas.
// The pairs are cut into one run per warp, in order.  Each warp counts its
// run's experts (lanes with the same expert are found by a match, the lowest
// one adds their number, so the counts need no atomics and their order is
// fixed); the counts are scanned over a CTA's warps, over the cluster's CTAs
// and over the experts; then each pair's row is the sum of its place in the run,
// kept from the count, and those.  Bound by latency (the input is some hundred
// KB): 128 pairs 3.6 us a call with the launch; 32768 pairs 9.1 call after
// call, 7 before a dispatch; 65536 14.6; 262144, past the ids that are held, 64.
__global__ void __launch_bounds__(1024) k_moe_route(const __grid_constant__ RouteArgs a) {
    extern __shared__ uint32_t route_smem[];
    const int E1 = a.E + 1;                           // expert E: not here
    uint32_t *total = route_smem;                     // [E1]: this CTA's counts
    uint32_t *first = total + E1;                     // [E1]: rows before the expert
    uint32_t *count = first + E1;                     // [warps][E1]
    __shared__ uint32_t part[32];
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t ctas = cluster_size(), rank = cluster_rank();
    kernel_prologue();

    for (int i = threadIdx.x; i < warps * E1; i += blockDim.x)
        count[i] = 0u;
    __syncthreads();
    const uint32_t runs = ctas * warps;
    const uint32_t len = ((a.n + runs - 1) / runs + 31) / 32 * 32;
    const uint64_t lo64 = (uint64_t)(rank * warps + warp) * len;
    const uint32_t lo = lo64 < a.n ? (uint32_t)lo64 : a.n;
    const uint32_t hi = a.n - lo < len ? a.n : lo + len;
    uint32_t *mine = count + warp * E1;
    // the run's first ids are read at once and kept for the second walk
    int held[kRouteHeld];
#pragma unroll
    for (int i = 0; i < kRouteHeld; ++i) {
        const uint32_t p = lo + 32 * i + lane;
        held[i] = p < hi && p >= lo ? expert_of(a, p) : -1;
    }
    // adds 32 pairs to the warp's counts; a pair's place within the warp's run
    auto count_32 = [&](int e) {
        const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
        const uint32_t before = e >= 0 ? mine[e] : 0u;
        __syncwarp();
        if (e >= 0 && lane == __ffs(same) - 1)
            mine[e] = before + __popc(same);
        __syncwarp();
        return before + __popc(same & ((1u << lane) - 1u));
    };
    uint32_t place[kRouteHeld];
#pragma unroll
    for (int i = 0; i < kRouteHeld; ++i)
        if (lo + 32 * i < hi)
            place[i] = count_32(held[i]);
    for (uint32_t p0 = lo + 32 * kRouteHeld; p0 < hi; p0 += 32)
        (void)count_32(p0 + lane < hi ? expert_of(a, p0 + lane) : -1);
    __syncthreads();
    // over the CTA's warps: count[w][e] becomes the number before warp w
    for (int e = threadIdx.x; e < E1; e += blockDim.x) {
        uint32_t sum = 0u;
        for (int w = 0; w < warps; ++w) {
            const uint32_t c = count[w * E1 + e];
            count[w * E1 + e] = sum;
            sum += c;
        }
        total[e] = sum;
    }
    cluster_sync();
    // over the CTAs, then over the experts
    uint32_t carry = 0u;
    for (int e0 = 0; e0 < E1; e0 += blockDim.x) {
        const int e = e0 + threadIdx.x;
        uint32_t before = 0u, all = 0u;
        if (e < E1) {
            uint32_t v[kRouteCtas];               // at most kRouteCtas peers
#pragma unroll
            for (uint32_t c = 0; c < kRouteCtas; ++c)
                v[c] = c < ctas ? ld_peer_u32(total + e, c) : 0u;
#pragma unroll
            for (uint32_t c = 0; c < kRouteCtas; ++c) {
                before += c < rank ? v[c] : 0u;
                all += v[c];
            }
        }
        uint32_t scan = all;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, scan, d);
            scan += lane >= d ? v : 0u;
        }
        if (lane == 31)
            part[warp] = scan;
        __syncthreads();
        uint32_t w = lane < warps ? part[lane] : 0u;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, w, d);
            w += lane >= d ? v : 0u;
        }
        const uint32_t lower = __shfl_sync(0xFFFFFFFFu, w, warp > 0 ? warp - 1 : 0);
        const uint32_t start = carry + (warp > 0 ? lower : 0u) + scan - all;
        carry += __shfl_sync(0xFFFFFFFFu, w, 31);
        if (e < E1) {
            first[e] = start + before;
            if (rank == 0)
                a.offsets[e] = (int32_t)start;
        }
        __syncthreads();
    }
    cluster_sync();                                   // every peer has read `total`
    auto put = [&](uint32_t p, int e, uint32_t row) {
        if (e < 0)
            return;
        a.row_of[p] = e < a.E ? (int32_t)row : -1;
        if (a.src)
            a.src[row] = e < a.E ? (int32_t)p : -1;
    };
#pragma unroll
    for (int i = 0; i < kRouteHeld; ++i)
        if (lo + 32 * i < hi && held[i] >= 0)
            put(lo + 32 * i + lane, held[i], first[held[i]] + mine[held[i]] + place[i]);
    if (lo + 32 * kRouteHeld < hi) {
        // the counts go on from the pairs that were held
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kRouteHeld; ++i)
            (void)count_32(held[i]);
        for (uint32_t p0 = lo + 32 * kRouteHeld; p0 < hi; p0 += 32) {
            const int e = p0 + lane < hi ? expert_of(a, p0 + lane) : -1;
            const uint32_t at = count_32(e);
            put(p0 + lane, e, e >= 0 ? first[e] + at : 0u);
        }
    }
}

static cudaError_t launch_route(const RouteArgs &a, cudaStream_t s) {
    // a warp's run is 32 pairs at least; one CTA up to 1024 pairs; eight warps at
    // least, which also clear and scan the experts' counts
    const uint32_t groups = (a.n + 31) / 32;
    const int warps = groups < 8 ? 8 : groups < (uint32_t)kRouteWarps ? (int)groups : kRouteWarps;
    const int ctas = groups > (uint32_t)kRouteWarps ? kRouteCtas : 1;
    const size_t smem = (size_t)(warps + 2) * (a.E + 1) * sizeof(uint32_t);
    // the opt-in holds for every size used: 34 rows of at most 1025 words
    const cudaError_t e = opt_in_smem<k_moe_route>((kRouteWarps + 2) * (AR_MOE_MAX_EXPERTS + 1) *
                                                   sizeof(uint32_t));
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = ctas;
    cfg.blockDim = warps * 32;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k_moe_route, a);
}

// ---- rows to their experts -----------------------------------------------------

struct MoveArgs {
    const uint8_t *x;
    const float *xscale;
    const int32_t *row_of;
    uint8_t *rows;
    float *rscale;
    uint64_t sx, srows;       // bytes between rows
    uint64_t nrows, T;
    uint64_t bytes;           // of a row
    uint64_t per_token;       // threads per token
    uint32_t units;           // 16-byte words of a row
    int K, nb;                // nb: scales per row
};

// 16 bytes from an address that is a multiple of 4 only plus `shift` bits.
__device__ __forceinline__ uint4 load_shifted(const uint32_t *p, uint32_t shift) {
    const uint32_t a = p[0], b = p[1], c = p[2], d = p[3], e = p[4];
    return make_uint4(__funnelshift_r(a, b, shift), __funnelshift_r(b, c, shift),
                      __funnelshift_r(c, d, shift), __funnelshift_r(d, e, shift));
}

// The threads are counted over the tokens: a.units words, then the bytes past
// them, then the scales of a token, one a thread, each stored to the token's K
// rows.  ALIGNED: every row starts on a 16-byte boundary.  Otherwise a thread
// has a 16-byte word of the destination, assembled from the five aligned words
// of 4 bytes that hold its source; the words that are not whole, or whose
// source words reach past the row, go byte by byte.  Bound by memory: 4096 tokens
// x 8 rows of 8192 bf16 in 93 us (6.5 TB/s).
template <bool ALIGNED>
__global__ void __launch_bounds__(256) k_moe_dispatch(const __grid_constant__ MoveArgs a) {
    kernel_prologue();
    const uint64_t all = a.T * a.per_token;
    for (uint64_t id = (uint64_t)blockIdx.x * 256 + threadIdx.x; id < all;
         id += (uint64_t)gridDim.x * 256) {
        const uint64_t t = id / a.per_token;
        const uint32_t u = (uint32_t)(id - t * a.per_token);
        const uint8_t *x = a.x + t * a.sx;
        const int32_t *row_of = a.row_of + t * a.K;
        const uint32_t tail = ALIGNED ? (uint32_t)(a.bytes - (uint64_t)a.units * 16) : 0u;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (u >= a.units + tail)
            v.x = __float_as_uint(a.xscale[t * a.nb + (u - a.units - tail)]);
        else if (ALIGNED && u < a.units)
            v = ld_v4_stream(reinterpret_cast<const uint4 *>(x) + u);
        else if (ALIGNED)
            v.x = x[(uint64_t)a.units * 16 + (u - a.units)];
        for (int k0 = 0; k0 < a.K; k0 += 8) {
            // the eight rows first: a store between two of these loads would
            // hold the second back
            int32_t r[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                r[k] = k0 + k < a.K ? row_of[k0 + k] : -1;
                if ((uint64_t)(uint32_t)r[k] >= a.nrows)
                    r[k] = -1;
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (r[k] < 0)
                    continue;
                uint8_t *row = a.rows + (uint64_t)r[k] * a.srows;
                if (u >= a.units + tail) {
                    a.rscale[(uint64_t)r[k] * a.nb + (u - a.units - tail)] = __uint_as_float(v.x);
                } else if (ALIGNED && u < a.units) {
                    st_v4(reinterpret_cast<uint4 *>(row) + u, v);
                } else if (ALIGNED) {
                    row[(uint64_t)a.units * 16 + (u - a.units)] = (uint8_t)v.x;
                } else {
                    // bytes [lo, hi) of the row: this word of the destination
                    const int64_t lo = (int64_t)u * 16 - (int64_t)((uintptr_t)row & 15u);
                    const int64_t hi = lo + 16, end = (int64_t)a.bytes;
                    const uint32_t low = (uint32_t)((uintptr_t)(x + lo) & 3u);
                    if (lo - low >= 0 && lo - low + 20 <= end) {
                        const uint32_t *words = reinterpret_cast<const uint32_t *>(x + lo - low);
                        st_v4(row + lo, load_shifted(words, 8 * low));
                    } else {
                        for (int64_t i = lo < 0 ? 0 : lo; i < hi && i < end; ++i)
                            row[i] = x[i];
                    }
                }
            }
        }
    }
}

static cudaError_t launch_dispatch(MoveArgs a, bool aligned, cudaStream_t s) {
    // not aligned: a row of n bytes touches at most n / 16 + 2 words
    a.units = (uint32_t)(a.bytes / 16 + (aligned ? 0 : 2));
    a.per_token = a.units + (aligned ? a.bytes % 16 : 0) + (uint64_t)a.nb;
    const uint64_t ctas = (a.T * a.per_token + 255) / 256;
    const int grid = (int)(ctas < (1u << 30) ? ctas : (1u << 30));
    return aligned ? launch_kernel(k_moe_dispatch<true>, grid, 256, 0, s, true, a)
                   : launch_kernel(k_moe_dispatch<false>, grid, 256, 0, s, true, a);
}

// ---- rows back at their tokens ---------------------------------------------------

struct ReturnArgs {
    const uint8_t *rows;
    const int32_t *row_of;
    const float *w;
    uint8_t *out;
    uint64_t srows, sout;     // bytes between rows
    uint64_t nrows, T;
    uint32_t H;
    int K;
};

// The eight choices from k0 on of a token: their rows (-1: none) and weights.
struct Choices {
    int32_t r[8];
    float w[8];
    __device__ __forceinline__ void read(const int32_t *row_of, const float *w_of, uint64_t t,
                                         int K, int k0, uint64_t nrows) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            r[j] = k0 + j < K ? row_of[t * K + k0 + j] : -1;
            w[j] = w_of && k0 + j < K ? w_of[t * K + k0 + j] : 1.0f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (r[j] < 0 || (uint64_t)r[j] >= nrows)
                r[j] = -1;
    }
};

// A job is 256 units of a token, one a thread; FLAT (rows of fewer units): 256
// units counted over the tokens.  The CTAs stay and take job after job.  Eight
// rows' loads are in flight at a time, and the next job's rows and weights are
// read meanwhile, so that its loads need not wait for them.  Bound by memory: 4096
// tokens x 8 rows of 8192 bf16 in 98 us (6.1 TB/s); with a CTA per job that reads
// its own choices first 115.
template <int DT, bool WIDE, bool FLAT>
__global__ void __launch_bounds__(256, 3) k_moe_return(const __grid_constant__ ReturnArgs a) {
    using L = Rows<DT, WIDE>;
    kernel_prologue();
    const uint32_t units = L::units(a.H), parts = (units + 255) / 256;
    const uint64_t jobs = FLAT ? (a.T * units + 255) / 256 : a.T * parts;
    // token and unit of this thread in a job; a token past the last: none
    auto token = [&](uint64_t job) {
        return FLAT ? (job * 256 + threadIdx.x) / units : job / parts;
    };
    auto unit = [&](uint64_t job, uint64_t t) {
        return FLAT ? (uint32_t)(job * 256 + threadIdx.x - t * units)
                    : (uint32_t)(job - t * parts) * 256 + threadIdx.x;
    };
    Choices next;
    if (blockIdx.x < jobs && token(blockIdx.x) < a.T)
        next.read(a.row_of, a.w, token(blockIdx.x), a.K, 0, a.nrows);
    for (uint64_t job = blockIdx.x; job < jobs; job += gridDim.x) {
        const uint64_t t = token(job);
        const uint32_t u = unit(job, t);
        if (FLAT && t >= a.T)
            break;                            // the last job's threads past the end
        const bool on = FLAT || u < units;
        float acc[L::E];
#pragma unroll
        for (int i = 0; i < L::E; ++i)
            acc[i] = 0.0f;
        bool any = false;
        for (int k0 = 0; k0 < a.K; k0 += 8) {
            Choices c = next;
            if (k0 > 0)
                c.read(a.row_of, a.w, t, a.K, k0, a.nrows);
            uint4 p[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                p[j] = L::load_if(on && c.r[j] >= 0,
                                  a.rows + (uint64_t)(c.r[j] < 0 ? 0 : c.r[j]) * a.srows, u, a.H);
            if (k0 + 8 >= a.K && job + gridDim.x < jobs && token(job + gridDim.x) < a.T)
                next.read(a.row_of, a.w, token(job + gridDim.x), a.K, 0, a.nrows);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c.r[j] >= 0) {
                    float v[L::E];
                    L::widen(p[j], v);
#pragma unroll
                    for (int i = 0; i < L::E; i += 2) {
                        mul2(v + i, c.w[j], c.w[j]);
                        if (any)
                            add2(acc + i, v[i], v[i + 1]);
                        else {
                            acc[i] = v[i];
                            acc[i + 1] = v[i + 1];
                        }
                    }
                    any = true;
                }
        }
        if (on)
            L::store(a.out + t * a.sout, u, a.H, acc);
    }
}

// ---- gradient of the return ------------------------------------------------------

struct ReturnGradArgs {
    const uint8_t *dout, *rows;
    const int32_t *row_of;
    const float *w;
    uint8_t *drows;
    float *dw;
    uint64_t sdout, srows, sdrows;    // bytes between rows
    uint64_t nrows, T;
    uint32_t H;
    int K;
};

// A token's CTAs are one cluster, each with a run of the token's units.  Eight
// choices at a time: every thread walks its units of dout, writes the weighted
// unit to each choice's row of drows and adds its product with the choice's row;
// the eight sums are then joined over the CTA and, in order, over the cluster.
// Bound by memory: 4096 tokens x 8 rows of 8192 bf16 in 186 us (6.1 TB/s); one
// token in 4 us, by one CTA 7.
template <int DT, bool WIDE>
__global__ void __launch_bounds__(256, 2)
k_moe_return_grad(const __grid_constant__ ReturnGradArgs a) {
    using L = Rows<DT, WIDE>;
    __shared__ float part[8][32], sums[8];
    kernel_prologue();
    const uint32_t ctas = cluster_size(), rank = cluster_rank();
    // whole warps of units per CTA
    const uint32_t run = (L::warp_units(a.H) / 32 + ctas - 1) / ctas * 32;
    const uint32_t first = rank * run;
    const uint32_t units = first + run < L::units(a.H) ? first + run : L::units(a.H);
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (uint64_t t = blockIdx.x / ctas; t < a.T; t += gridDim.x / ctas) {
        const uint8_t *dout = a.dout + t * a.sdout;
        for (int k0 = 0; k0 < a.K; k0 += 8) {
            int32_t r[8];
            float w[8], dot[8][2];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                r[j] = k0 + j < a.K ? a.row_of[t * a.K + k0 + j] : -1;
                if (r[j] >= 0 && (uint64_t)r[j] >= a.nrows)
                    r[j] = -1;
                w[j] = a.w && k0 + j < a.K ? a.w[t * a.K + k0 + j] : 1.0f;
                dot[j][0] = dot[j][1] = 0.0f;
            }
            for (uint32_t u = first + threadIdx.x; u < units; u += blockDim.x) {
                uint4 p[8];
                if (a.dw) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        p[j] = L::load_if(r[j] >= 0,
                                          a.rows + (uint64_t)(r[j] < 0 ? 0 : r[j]) * a.srows, u,
                                          a.H);
                }
                float d[L::E];
                L::widen(L::load(dout, u, a.H), d);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (r[j] < 0)
                        continue;
                    if (a.dw) {
                        float v[L::E];
                        L::widen(p[j], v);
#pragma unroll
                        for (int i = 0; i < L::E; i += 2)
                            fma2(dot[j], d[i], d[i + 1], v[i], v[i + 1]);
                    }
                    if (a.drows) {
                        float g[L::E];
#pragma unroll
                        for (int i = 0; i < L::E; i += 2) {
                            g[i] = d[i];
                            g[i + 1] = d[i + 1];
                            mul2(g + i, w[j], w[j]);
                        }
                        L::store(a.drows + (uint64_t)r[j] * a.sdrows, u, a.H, g);
                    }
                }
            }
            if (a.dw) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float v = warp_sum(dot[j][0] + dot[j][1]);
                    if (lane == 0)
                        part[j][warp] = v;
                }
                __syncthreads();
                // warp w joins choices w, w + warps, ...
                for (int j = warp; j < 8; j += warps) {
                    const float v = warp_sum(lane < warps ? part[j][lane] : 0.0f);
                    if (lane == 0 && ctas > 1)
                        sums[j] = v;
                    else if (lane == 0 && k0 + j < a.K)
                        a.dw[t * a.K + k0 + j] = v;
                }
                if (ctas > 1) {
                    cluster_sync();
                    if (rank == 0 && threadIdx.x < 8 && k0 + (int)threadIdx.x < a.K) {
                        float v = 0.0f;
                        for (uint32_t c = 0; c < ctas; ++c)
                            v += ld_peer_f32(sums + threadIdx.x, c);
                        a.dw[t * a.K + k0 + threadIdx.x] = v;
                    }
                    cluster_sync();
                } else {
                    __syncthreads();
                }
            }
        }
    }
}

template <int DT, bool WIDE>
static cudaError_t return_grad_launch(const ReturnGradArgs &a, cudaStream_t s) {
    const uint32_t units = Rows<DT, WIDE>::warp_units(a.H);
    const int threads = (int)(units < 256 ? units : 256);
    // few tokens: as many CTAs a token as its units or half the SMs allow
    int ctas = 1;
    while (ctas < 8 && units >= 512u * ctas && a.T * ctas * 2 <= (uint64_t)sm_count())
        ctas *= 2;
    const uint64_t grid = a.T * ctas, most = 1u << 30;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = (unsigned)(grid < most ? grid : most);
    cfg.blockDim = threads;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k_moe_return_grad<DT, WIDE>, a);
}

template <int DT, bool WIDE> static cudaError_t return_launch(const ReturnArgs &a, cudaStream_t s) {
    const uint64_t units = Rows<DT, WIDE>::units(a.H), most = 3 * (uint64_t)sm_count();
    if (most < 1)
        return cudaErrorUnknown;
    const bool flat = units < 256;
    const uint64_t jobs = flat ? (a.T * units + 255) / 256 : a.T * ((units + 255) / 256);
    const int grid = (int)(jobs < most ? jobs : most);
    return flat ? launch_kernel(k_moe_return<DT, WIDE, true>, grid, 256, 0, s, true, a)
                : launch_kernel(k_moe_return<DT, WIDE, false>, grid, 256, 0, s, true, a);
}

// Sizes every row mover shares: the status code, AR_OK if they hold.
static int check_moe(size_t T, int K, size_t H) {
    if (K < 1 || K > AR_MOE_MAX_CHOICES || H < 1)
        return AR_ERR_INVALID;
    if (H >= (size_t)1 << 31 || T > (((size_t)1 << 31) - 1) / (size_t)K)
        return AR_ERR_UNSUPPORTED;
    return AR_OK;
}

}  // namespace ar

using namespace ar;

extern "C" {

int ar_moe_route(const void *ids, int ids_bytes, size_t T, int K, int E, int32_t *offsets,
                 int32_t *row_of, int32_t *src, cudaStream_t stream) {
    const int rc = check_moe(T, K, 1);
    if (rc != AR_OK)
        return rc;
    if ((ids_bytes != 4 && ids_bytes != 8) || E < 1 || !offsets || (T > 0 && (!ids || !row_of)))
        return AR_ERR_INVALID;
    if (E > AR_MOE_MAX_EXPERTS)
        return AR_ERR_UNSUPPORTED;
    const size_t n = T * (size_t)K;
    const Matrix mi = matrix(ids, 0, 1, n, ids_bytes), mo = matrix(offsets, 0, 1, E + 1, 4);
    const Matrix mr = matrix(row_of, 0, 1, n, 4), ms = matrix(src, 0, 1, n, 4);
    if (!mi.ok || !mo.ok || !mr.ok || !ms.ok || meet(mi, mo) || meet(mi, mr) || meet(mi, ms) ||
        meet(mo, mr) || meet(mo, ms) || meet(mr, ms))
        return AR_ERR_INVALID;
    RouteArgs a;
    a.ids = ids;
    a.offsets = offsets;
    a.row_of = row_of;
    a.src = src;
    a.n = (uint32_t)n;
    a.E = E;
    a.wide_ids = ids_bytes == 8;
    return launched(launch_route(a, stream));
}

int ar_moe_dispatch(const void *x, size_t ldx, const float *xscale, const int32_t *row_of,
                    void *rows, size_t ldrows, float *rscale, size_t nrows, size_t T, int K,
                    size_t H, int dtype, cudaStream_t stream) {
    const int rc = check_moe(T, K, H);
    if (rc != AR_OK)
        return rc;
    if (!(float_dtype(dtype) || dtype == AR_E4M3) || (xscale != nullptr) != (rscale != nullptr))
        return AR_ERR_INVALID;
    if (T == 0 || nrows == 0)
        return AR_OK;
    if (!x || !row_of || !rows)
        return AR_ERR_INVALID;
    const size_t esz = dtype == AR_E4M3 ? 1 : elem_size(dtype);
    const size_t nb = xscale ? (H - 1) / AR_SCALE_BLOCK + 1 : 0;
    const Matrix mx = matrix(x, ldx, T, H, esz), mr = matrix(rows, ldrows, nrows, H, esz);
    const Matrix mi = matrix(row_of, 0, T, K, 4);
    const Matrix mc = matrix(xscale, 0, T, nb, 4), md = matrix(rscale, 0, nrows, nb, 4);
    if (!mx.ok || !mr.ok || !mi.ok || !mc.ok || !md.ok || meet(mr, mx) || meet(mr, mi) ||
        meet(mr, mc) || meet(mr, md) || meet(md, mx) || meet(md, mi) || meet(md, mc))
        return AR_ERR_INVALID;
    MoveArgs a;
    a.x = static_cast<const uint8_t *>(x);
    a.xscale = xscale;
    a.row_of = row_of;
    a.rows = static_cast<uint8_t *>(rows);
    a.rscale = rscale;
    a.sx = mx.stride;
    a.srows = mr.stride;
    a.nrows = nrows;
    a.T = T;
    a.bytes = H * esz;
    a.K = K;
    a.nb = (int)nb;
    return launched(launch_dispatch(a, wide(mx) && wide(mr), stream));
}

int ar_moe_return(const void *rows, size_t ldrows, size_t nrows, const int32_t *row_of,
                  const float *w, void *out, size_t ldout, size_t T, int K, size_t H, int dtype,
                  cudaStream_t stream) {
    const int rc = check_moe(T, K, H);
    if (rc != AR_OK)
        return rc;
    if (!float_dtype(dtype))
        return AR_ERR_INVALID;
    if (T == 0)
        return AR_OK;
    if ((!rows && nrows > 0) || !row_of || !out)
        return AR_ERR_INVALID;
    const size_t esz = elem_size(dtype);
    const Matrix mr = matrix(rows, ldrows, nrows, H, esz), mo = matrix(out, ldout, T, H, esz);
    const Matrix mi = matrix(row_of, 0, T, K, 4), mw = matrix(w, 0, T, K, 4);
    if (!mr.ok || !mo.ok || !mi.ok || !mw.ok || meet(mo, mr) || meet(mo, mi) || meet(mo, mw))
        return AR_ERR_INVALID;
    ReturnArgs a;
    a.rows = static_cast<const uint8_t *>(rows);
    a.row_of = row_of;
    a.w = w;
    a.out = static_cast<uint8_t *>(out);
    a.srows = mr.stride;
    a.sout = mo.stride;
    a.nrows = nrows;
    a.T = T;
    a.H = (uint32_t)H;
    a.K = K;
    const bool v = wide(mr) && wide(mo);
    switch (dtype) {
    case AR_BF16:
        return launched(v ? return_launch<AR_BF16, true>(a, stream)
                          : return_launch<AR_BF16, false>(a, stream));
    case AR_FP16:
        return launched(v ? return_launch<AR_FP16, true>(a, stream)
                          : return_launch<AR_FP16, false>(a, stream));
    default:
        return launched(v ? return_launch<AR_FP32, true>(a, stream)
                          : return_launch<AR_FP32, false>(a, stream));
    }
}

int ar_moe_return_grad(const void *dout, size_t lddout, const void *rows, size_t ldrows,
                       size_t nrows, const int32_t *row_of, const float *w, void *drows,
                       size_t lddrows, float *dw, size_t T, int K, size_t H, int dtype,
                       cudaStream_t stream) {
    const int rc = check_moe(T, K, H);
    if (rc != AR_OK)
        return rc;
    if (!float_dtype(dtype) || (!drows && !dw))
        return AR_ERR_INVALID;
    if (T == 0)
        return AR_OK;
    if (!dout || !row_of || (dw && !rows && nrows > 0))
        return AR_ERR_INVALID;
    if (!dw)
        rows = nullptr;                       // not read
    const size_t esz = elem_size(dtype);
    const Matrix mo = matrix(dout, lddout, T, H, esz), mr = matrix(rows, ldrows, nrows, H, esz);
    const Matrix md = matrix(drows, lddrows, nrows, H, esz);
    const Matrix mi = matrix(row_of, 0, T, K, 4), mw = matrix(w, 0, T, K, 4);
    const Matrix mg = matrix(dw, 0, T, K, 4);
    if (!mo.ok || !mr.ok || !md.ok || !mi.ok || !mw.ok || !mg.ok || clash(md, mr) || meet(md, mo) ||
        meet(md, mi) || meet(md, mw) || meet(md, mg) || meet(mg, mo) || meet(mg, mr) ||
        meet(mg, mi) || meet(mg, mw))
        return AR_ERR_INVALID;
    ReturnGradArgs a;
    a.dout = static_cast<const uint8_t *>(dout);
    a.rows = static_cast<const uint8_t *>(rows);
    a.row_of = row_of;
    a.w = w;
    a.drows = static_cast<uint8_t *>(drows);
    a.dw = dw;
    a.sdout = mo.stride;
    a.srows = mr.stride;
    a.sdrows = md.stride;
    a.nrows = nrows;
    a.T = T;
    a.H = (uint32_t)H;
    a.K = K;
    const bool v = wide(mo) && (!rows || wide(mr)) && (!drows || wide(md));
    switch (dtype) {
    case AR_BF16:
        return launched(v ? return_grad_launch<AR_BF16, true>(a, stream)
                          : return_grad_launch<AR_BF16, false>(a, stream));
    case AR_FP16:
        return launched(v ? return_grad_launch<AR_FP16, true>(a, stream)
                          : return_grad_launch<AR_FP16, false>(a, stream));
    default:
        return launched(v ? return_grad_launch<AR_FP32, true>(a, stream)
                          : return_grad_launch<AR_FP32, false>(a, stream));
    }
}

}  // extern "C"
