// A mixture-of-experts layer for a few tokens, in two launches:
//
//   h = g / (1 + exp(-g)) * u,  g, u = the two halves of up[e] x[t]
//   out[t] = sum_k w[t, k] down[e] h
//
// Bound by memory: the weights of every expert that a token chose are read once.
// They are the 16-row operand of warp-wide products (E4M3 is exact in binary16), the
// tokens its 8 columns: x and h are scaled by a power of two for each 128 of a row
// so that binary16 holds them, in two parts where one would round.  A block of 128
// along k gets its scales in binary32 when it is summed.
//
// Weights go from global memory straight to the lanes that multiply with them: a
// lane takes 16 bytes of a row, and the order of k inside a block is that of the
// lanes, for the tokens too.
//
// First launch: a CTA takes 16 rows of both halves of one expert, its warps share
// the blocks along k.  Second launch: a CTA takes rows of the output, its warps share
// the blocks along k of all experts; each keeps its own sums of all tokens, which
// are added in order.
#include "ar_mma.cuh"
#include "ar_rows.cuh"

namespace ar {

constexpr int kMoeThreads = 256, kMoeWarps = kMoeThreads / 32;
constexpr int kMoePairs = AR_MOE_LAYER_PAIRS;
constexpr int kColumns = 32;          // most pairs of an expert in one pass over its weights

struct MoeArgs {
    const uint8_t *x;
    const void *ids;
    const float *w;
    const uint8_t *up, *down;
    const float *up_scale, *down_scale;
    uint8_t *out;
    float *h;                         // T * K rows of ldh
    uint64_t sx, sout;                // bytes between rows
    uint64_t ldup, lddown, ldh;
    uint32_t T, K, H, F, E;
    uint32_t hb, fb, ub;              // blocks of 128 along H, F and 2F
    int wide_up, wide_down, wide_x;
    int ids8;
};

// The pairs that are here, and the experts they go to in the order of their first pair.
struct Chosen {
    int16_t expert[kMoePairs];        // of a pair, or -1
    int16_t active[kMoePairs];
    int first[AR_MOE_MAX_EXPERTS];
    int count;                        // of active
    int warp_count[kMoePairs / 32];
};

__device__ __forceinline__ void choose(const MoeArgs &a, Chosen &c) {
    const uint32_t pairs = a.T * a.K;
    for (uint32_t e = threadIdx.x; e < a.E; e += kMoeThreads)
        c.first[e] = kMoePairs;
    __syncthreads();
    for (uint32_t p = threadIdx.x; p < pairs; p += kMoeThreads) {
        const int64_t id = a.ids8 ? static_cast<const int64_t *>(a.ids)[p]
                                  : (int64_t) static_cast<const int32_t *>(a.ids)[p];
        const bool here = id >= 0 && id < (int64_t)a.E;
        c.expert[p] = here ? (int16_t)id : (int16_t)-1;
        if (here)
            atomicMin(&c.first[id], (int)p);
    }
    __syncthreads();
    // the first pair of an expert stands for it
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < kMoePairs / kMoeThreads; ++i) {
        const uint32_t p = threadIdx.x + i * kMoeThreads;
        const bool lead = p < pairs && c.expert[p] >= 0 && c.first[c.expert[p]] == (int)p;
        const uint32_t m = __ballot_sync(0xFFFFFFFFu, lead);
        if (lane == 0)
            c.warp_count[p / 32] = __popc(m);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kMoePairs / kMoeThreads; ++i) {
        const uint32_t p = threadIdx.x + i * kMoeThreads;
        const bool lead = p < pairs && c.expert[p] >= 0 && c.first[c.expert[p]] == (int)p;
        const uint32_t m = __ballot_sync(0xFFFFFFFFu, lead);
        int before = 0;
        for (uint32_t w = 0; w < p / 32; ++w)
            before += c.warp_count[w];
        if (lead)
            c.active[before + __popc(m & ((1u << lane) - 1u))] = c.expert[p];
        if (p == kMoePairs - 1)
            c.count = before + __popc(m);
    }
    __syncthreads();
}

// The pairs of expert e in order, by one warp: `list` receives those from `skip` on,
// at most kColumns; returns how many there are in all.
__device__ __forceinline__ int list_pairs(const MoeArgs &a, const Chosen &c, int e, int skip,
                                          int16_t *list) {
    const uint32_t pairs = a.T * a.K, lane = threadIdx.x & 31;
    int n = 0;
    for (uint32_t p0 = 0; p0 < pairs; p0 += 32) {
        const uint32_t p = p0 + lane;
        const bool mine = p < pairs && c.expert[p] == e;
        const uint32_t m = __ballot_sync(0xFFFFFFFFu, mine);
        const int at = n + __popc(m & ((1u << lane) - 1u)) - skip;
        if (mine && at >= 0 && at < kColumns)
            list[at] = (int16_t)p;
        n += __popc(m);
    }
    __syncwarp();
    return n;
}

// 16 codes of a weight row from k on; zeros past K.
__device__ __forceinline__ uint4 load_codes(const uint8_t *row, uint32_t k, uint32_t K, bool wide,
                                            bool on) {
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    if (on && k < K) {
        if (wide && k + 16 <= K)
            return ld_v4_stream(row + k);
        for (uint32_t i = 0; i < 16 && k + i < K; ++i)
            w[i / 4] |= (uint32_t)row[k + i] << (8 * (i & 3));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// 16 elements of a row of x (type DT) from k on as binary32; zeros past K.
template <int DT>
__device__ __forceinline__ void load_column(const uint8_t *row, uint32_t k, uint32_t K, bool wide,
                                            bool on, float *v) {
    constexpr int E = 16 / Elem<DT>::kSize;
    if (on && wide && k + 16 <= K) {
#pragma unroll
        for (int i = 0; i < 16; i += E)
            Rows<DT, true>::widen(ld_v4_l1(row + (uint64_t)(k + i) * Elem<DT>::kSize), v + i);
        return;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i)
        v[i] = on && k + i < K ? widen1<DT>(ld_elem<DT>(row, k + i)) : 0.0f;
}

// One block of 128 along k: MT tiles of 16 weight rows by NT tiles of 8 columns.
//   weights(mt, half, i): the lane's 16 codes of row lane / 4 (i = 0) or that + 8
//   column(nt, half, v):  the lane's 16 values of column lane / 4
// sum[mt][nt] += scale(mt, i) * product.
template <int MT, int NT, bool LO, typename Weights, typename Column, typename Scale>
__device__ __forceinline__ void block_product(float (*sum)[NT][4], Weights weights, Column column,
                                              Scale scale) {
    const int lane = threadIdx.x & 31;
    uint4 q[MT][2][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int half = 0; half < 2; ++half)
                q[mt][half][i] = weights(mt, half, i);
    float ws[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < 2; ++i)
            ws[mt][i] = scale(mt, i);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        float v[32];
        column(nt, 0, v);
        column(nt, 1, v + 16);
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i)
            top = fmaxf(top, fabsf(v[i]));
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        float s, inverse;
        half_range(top, s, inverse);
        float part[MT][4] = {};
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float *x = v + 16 * half + 4 * k;
                const float y[4] = {x[0] * s, x[1] * s, x[2] * s, x[3] * s};
                const uint32_t b0 = half2_of(y[0], y[1]), b1 = half2_of(y[2], y[3]);
                uint32_t c0 = 0, c1 = 0;
                if (LO) {
                    const float2 f0 = __half22float2(*reinterpret_cast<const __half2 *>(&b0));
                    const float2 f1 = __half22float2(*reinterpret_cast<const __half2 *>(&b1));
                    // an infinity has no second part
                    c0 = half2_of(isinf(f0.x) ? 0.0f : y[0] - f0.x, isinf(f0.y) ? 0.0f : y[1] - f0.y);
                    c1 = half2_of(isinf(f1.x) ? 0.0f : y[2] - f1.x, isinf(f1.y) ? 0.0f : y[3] - f1.y);
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const uint4 g = q[mt][half][0], u = q[mt][half][1];
                    uint32_t m[4];
                    from_e4m3x4(k == 0 ? g.x : k == 1 ? g.y : k == 2 ? g.z : g.w, m[0], m[2]);
                    from_e4m3x4(k == 0 ? u.x : k == 1 ? u.y : k == 2 ? u.z : u.w, m[1], m[3]);
                    mma16<AR_FP16>(part[mt], m, b0, b1);
                    if (LO)
                        mma16<AR_FP16>(part[mt], m, c0, c1);
                }
            }
        // the columns that this lane has sums of
        const float i0 = __shfl_sync(0xFFFFFFFFu, inverse, lane % 4 * 8);
        const float i1 = __shfl_sync(0xFFFFFFFFu, inverse, lane % 4 * 8 + 4);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            sum[mt][nt][0] += part[mt][0] * i0 * ws[mt][0];
            sum[mt][nt][1] += part[mt][1] * i1 * ws[mt][0];
            sum[mt][nt][2] += part[mt][2] * i0 * ws[mt][1];
            sum[mt][nt][3] += part[mt][3] * i1 * ws[mt][1];
        }
    }
}

// ---- first launch -------------------------------------------------------------

constexpr int kUpTiles = 2, kUpRows = 8 * kUpTiles;       // rows of each half

struct UpShared {
    Chosen c;
    int16_t list[kMoeWarps][kColumns];
    float part[kMoeWarps][2][kUpRows][kColumns + 1];
};

// Rows f0.. of both halves of expert e times the listed pairs.
template <int DT, int NT>
__device__ __forceinline__ void up_unit(const MoeArgs &a, UpShared &s, int e, uint32_t f0, int n) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int16_t *list = s.list[warp];
    const uint8_t *w = a.up + (uint64_t)e * 2 * a.F * a.ldup;
    const float *ws = a.up_scale + (uint64_t)e * a.ub * a.hb;
    float sum[kUpTiles][NT][4] = {};
    for (uint32_t kb = warp; kb < a.hb; kb += kMoeWarps) {
        auto weights = [&](int mt, int half, int i) {
            const uint32_t f = f0 + mt * 8 + lane / 4;
            return load_codes(w + (uint64_t)(f + i * a.F) * a.ldup,
                              kb * 128 + half * 64 + lane % 4 * 16, a.H, a.wide_up, f < a.F);
        };
        auto column = [&](int nt, int half, float *v) {
            const int c = nt * 8 + lane / 4;
            const uint32_t t = c < n ? list[c] / a.K : 0u;
            load_column<DT>(a.x + t * a.sx, kb * 128 + half * 64 + lane % 4 * 16, a.H, a.wide_x,
                            c < n, v);
        };
        auto scale = [&](int mt, int i) {
            const uint32_t f = f0 + mt * 8 + lane / 4;
            return f < a.F ? ws[(uint64_t)((f + i * a.F) / 128) * a.hb + kb] : 0.0f;
        };
        block_product<kUpTiles, NT, DT == AR_FP32>(sum, weights, column, scale);
    }
#pragma unroll
    for (int mt = 0; mt < kUpTiles; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                s.part[warp][i / 2][mt * 8 + lane / 4][nt * 8 + lane % 4 * 2 + i % 2] =
                    sum[mt][nt][i];
    __syncthreads();
    for (int i = threadIdx.x; i < kUpRows * n; i += kMoeThreads) {
        const int r = i % kUpRows, c = i / kUpRows;
        float g = 0.0f, u = 0.0f;
#pragma unroll
        for (int k = 0; k < kMoeWarps; ++k) {
            g += s.part[k][0][r][c];
            u += s.part[k][1][r][c];
        }
        if (f0 + r < a.F)
            a.h[(uint64_t)list[c] * a.ldh + f0 + r] = __fdiv_rn(g, 1.0f + expf(-g)) * u;
    }
    __syncthreads();
}

template <int DT>
__global__ void __launch_bounds__(kMoeThreads, 2) k_moe_up(const __grid_constant__ MoeArgs a) {
    extern __shared__ uint4 smem[];
    UpShared &s = *reinterpret_cast<UpShared *>(smem);
    kernel_prologue();
    choose(a, s.c);
    const uint32_t tiles = (a.F + kUpRows - 1) / kUpRows;
    const uint64_t units = (uint64_t)s.c.count * tiles;
    for (uint64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const int e = s.c.active[unit / tiles];
        const uint32_t f0 = (uint32_t)(unit % tiles) * kUpRows;
        for (int skip = 0;; skip += kColumns) {
            const int all = list_pairs(a, s.c, e, skip, s.list[threadIdx.x >> 5]);
            const int n = all - skip < kColumns ? all - skip : kColumns;
            if (n <= 8)
                up_unit<DT, 1>(a, s, e, f0, n);
            else if (n <= 16)
                up_unit<DT, 2>(a, s, e, f0, n);
            else
                up_unit<DT, 4>(a, s, e, f0, n);
            if (all - skip <= kColumns)
                break;
        }
    }
}

// ---- second launch --------------------------------------------------------------

constexpr int kDownTiles = 1, kDownRows = 16 * kDownTiles;

struct DownShared {
    Chosen c;
    int16_t list[kMoeWarps][kColumns];
};
static size_t down_smem(uint32_t T) {
    return sizeof(DownShared) + sizeof(float) * kMoeWarps * kDownRows * T;
}

// Blocks [kb0, kb1) along k of expert e times the listed pairs, added to this warp's
// sums of their tokens.
template <int NT>
__device__ __forceinline__ void down_part(const MoeArgs &a, const int16_t *list, float *sums, int e,
                                          uint32_t r0, uint32_t kb0, uint32_t kb1, int n) {
    const int lane = threadIdx.x & 31;
    const uint8_t *w = a.down + (uint64_t)e * a.H * a.lddown;
    const float *ws = a.down_scale + (uint64_t)e * a.hb * a.fb;
    float sum[kDownTiles][NT][4] = {};
    for (uint32_t kb = kb0; kb < kb1; ++kb) {
        auto weights = [&](int mt, int half, int i) {
            const uint32_t r = r0 + mt * 16 + i * 8 + lane / 4;
            return load_codes(w + (uint64_t)r * a.lddown, kb * 128 + half * 64 + lane % 4 * 16, a.F,
                              a.wide_down, r < a.H);
        };
        auto column = [&](int nt, int half, float *v) {
            const int c = nt * 8 + lane / 4;
            const uint32_t p = c < n ? list[c] : 0u;
            load_column<AR_FP32>(reinterpret_cast<const uint8_t *>(a.h + p * a.ldh),
                                 kb * 128 + half * 64 + lane % 4 * 16, a.F, true, c < n, v);
        };
        auto scale = [&](int mt, int i) {
            const uint32_t r = r0 + mt * 16 + i * 8 + lane / 4;
            return r < a.H ? ws[(uint64_t)(r / 128) * a.fb + kb] : 0.0f;
        };
        block_product<kDownTiles, NT, true>(sum, weights, column, scale);
    }
    // columns of different pairs may be one token's (its choices of one expert): one
    // column at a time
    for (int c = 0; c < n; ++c) {
        const int p = list[c];
        const float g = a.w ? a.w[p] : 1.0f;
        if (lane % 4 == c % 8 / 2) {
            float *token = sums + (uint32_t)p / a.K * kDownRows;
#pragma unroll
            for (int mt = 0; mt < kDownTiles; ++mt)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    if (nt == c / 8)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            token[mt * 16 + i * 8 + lane / 4] +=
                                g * (c & 1 ? sum[mt][nt][2 * i + 1] : sum[mt][nt][2 * i]);
        }
        __syncwarp();
    }
}

template <int DT>
__global__ void __launch_bounds__(kMoeThreads, 2) k_moe_down(const __grid_constant__ MoeArgs a) {
    extern __shared__ uint4 smem[];
    DownShared &s = *reinterpret_cast<DownShared *>(smem);
    float *sums = reinterpret_cast<float *>(&s + 1);      // [warp][token][row]
    kernel_prologue();
    choose(a, s.c);
    const int warp = threadIdx.x >> 5;
    const uint32_t r0 = blockIdx.x * kDownRows, each = a.T * kDownRows;
    float *mine = sums + (uint32_t)warp * each;
    for (uint32_t i = threadIdx.x; i < each * kMoeWarps; i += kMoeThreads)
        sums[i] = 0.0f;
    __syncthreads();
    // this warp's run of (expert, block)
    const uint32_t steps = (uint32_t)s.c.count * a.fb;
    uint32_t at = (uint32_t)((uint64_t)steps * warp / kMoeWarps);
    const uint32_t end = (uint32_t)((uint64_t)steps * (warp + 1) / kMoeWarps);
    while (at < end) {
        const uint32_t i = at / a.fb, kb0 = at - i * a.fb;
        const uint32_t kb1 = end - at < a.fb - kb0 ? kb0 + (end - at) : a.fb;
        const int e = s.c.active[i];
        for (int skip = 0;; skip += kColumns) {
            const int all = list_pairs(a, s.c, e, skip, s.list[warp]);
            const int n = all - skip < kColumns ? all - skip : kColumns;
            if (n <= 8)
                down_part<1>(a, s.list[warp], mine, e, r0, kb0, kb1, n);
            else if (n <= 16)
                down_part<2>(a, s.list[warp], mine, e, r0, kb0, kb1, n);
            else
                down_part<4>(a, s.list[warp], mine, e, r0, kb0, kb1, n);
            if (all - skip <= kColumns)
                break;
        }
        at += kb1 - kb0;
    }
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < each; i += kMoeThreads) {
        const uint32_t t = i / kDownRows, r = i % kDownRows;
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < kMoeWarps; ++k)
            v += sums[k * each + i];
        if (r0 + r < a.H)
            st_elem<DT>(a.out + t * a.sout, r0 + r, narrow1<DT>(v));
    }
}

template <int DT> static cudaError_t moe_dt(const MoeArgs &a, cudaStream_t s) {
    const int sms = sm_count();
    if (sms < 1)
        return cudaErrorUnknown;
    cudaError_t e = opt_in_smem<k_moe_up<DT>>(sizeof(UpShared));
    if (e == cudaSuccess)
        e = opt_in_smem<k_moe_down<DT>>(down_smem(AR_MOE_LAYER_TOKENS));
    if (e != cudaSuccess)
        return e;
    const uint64_t units = (uint64_t)((a.F + kUpRows - 1) / kUpRows) * a.T * a.K;
    const uint64_t most = 2 * (uint64_t)sms;
    e = launch_kernel(k_moe_up<DT>, (unsigned)(units < most ? units : most), kMoeThreads,
                      sizeof(UpShared), s, true, a);
    if (e != cudaSuccess)
        return e;
    return launch_kernel(k_moe_down<DT>, (a.H + kDownRows - 1) / kDownRows, kMoeThreads,
                         down_smem(a.T), s, true, a);
}

}  // namespace ar

using namespace ar;

extern "C" {

int ar_moe_layer(const void *x, size_t ldx, const void *ids, int ids_bytes, const float *w,
                 const void *up, size_t ldup, const float *up_scale, const void *down,
                 size_t lddown, const float *down_scale, void *out, size_t ldout, float *work,
                 size_t work_bytes, size_t T, int K, int E, size_t H, size_t F, int dtype,
                 cudaStream_t stream) {
    if (!float_dtype(dtype) || K < 1 || K > AR_MOE_MAX_CHOICES || E < 1 || H < 1 || F < 1 ||
        (ids_bytes != 4 && ids_bytes != 8))
        return AR_ERR_INVALID;
    const size_t most = (size_t)1 << 24;
    if (E > AR_MOE_MAX_EXPERTS || H >= most || F >= most || T > AR_MOE_LAYER_TOKENS ||
        T * K > AR_MOE_LAYER_PAIRS)
        return AR_ERR_UNSUPPORTED;
    if (T == 0)
        return AR_OK;
    if (!x || !ids || !up || !up_scale || !down || !down_scale || !out || !work)
        return AR_ERR_INVALID;
    const size_t size = elem_size(dtype), pairs = T * K;
    const size_t hb = (H - 1) / AR_SCALE_BLOCK + 1, fb = (F - 1) / AR_SCALE_BLOCK + 1;
    const size_t ub = (2 * F - 1) / AR_SCALE_BLOCK + 1;
    const Matrix mx = matrix(x, ldx, T, H, size), mo = matrix(out, ldout, T, H, size);
    const Matrix mi = matrix(ids, 0, 1, pairs, ids_bytes), mg = matrix(w, 0, 1, pairs, 4);
    const Matrix mu = matrix(up, ldup, (size_t)E * 2 * F, H, 1);
    const Matrix md = matrix(down, lddown, (size_t)E * H, F, 1);
    const Matrix ms = matrix(up_scale, 0, E * ub, hb, 4), mt = matrix(down_scale, 0, E * hb, fb, 4);
    const Matrix mw = matrix(work, 0, pairs, F + 128, 4);
    if (!mx.ok || !mo.ok || !mi.ok || !mg.ok || !mu.ok || !md.ok || !ms.ok || !mt.ok || !mw.ok ||
        mw.p % 16 != 0 || work_bytes < mw.bytes)
        return AR_ERR_INVALID;
    const Matrix *in[] = {&mx, &mi, &mg, &mu, &md, &ms, &mt};
    for (const Matrix *m : in)
        if (meet(mo, *m) || meet(mw, *m))
            return AR_ERR_INVALID;
    if (meet(mo, mw))
        return AR_ERR_INVALID;
    MoeArgs a;
    a.x = static_cast<const uint8_t *>(x);
    a.ids = ids;
    a.w = w;
    a.up = static_cast<const uint8_t *>(up);
    a.down = static_cast<const uint8_t *>(down);
    a.up_scale = up_scale;
    a.down_scale = down_scale;
    a.out = static_cast<uint8_t *>(out);
    a.h = work;
    a.sx = mx.stride;
    a.sout = mo.stride;
    a.ldup = mu.stride;
    a.lddown = md.stride;
    a.ldh = (F + 3) / 4 * 4;
    a.T = (uint32_t)T;
    a.K = (uint32_t)K;
    a.H = (uint32_t)H;
    a.F = (uint32_t)F;
    a.E = (uint32_t)E;
    a.hb = (uint32_t)hb;
    a.fb = (uint32_t)fb;
    a.ub = (uint32_t)ub;
    a.wide_up = wide(mu);
    a.wide_down = wide(md);
    a.wide_x = wide(mx);
    a.ids8 = ids_bytes == 8;
    switch (dtype) {
    case AR_BF16: return launched(moe_dt<AR_BF16>(a, stream));
    case AR_FP16: return launched(moe_dt<AR_FP16>(a, stream));
    default: return launched(moe_dt<AR_FP32>(a, stream));
    }
}

}  // extern "C"
