// Attention of one new token a sequence over its paged cache, split over the
// cache's length and joined.
//
//   s_j = scale <q, k_j>,  out = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m)
//
// Bound by memory: every key and value of the cache is read once, for all query
// heads that share it.  A unit is one sequence's key-value head with up to
// kRows of its query heads; its positions are cut into tiles.  The tiles of all
// units, in order, are dealt to the CTAs in runs of one length, so that a batch
// of any lengths loads every SM alike.  A CTA walks its run with the running
// maximum m and sum l of each row:
//   m' = max(m, max s),  l' = l 2^(m - m') + sum 2^(s - m'),  o' likewise
// (exponents of two: scale carries log2 e).  A unit that lies in one run is
// finished there; the others leave (m, l, o) in the workspace and a second
// launch joins them in order.
#include "ar_cache_attention.cuh"

namespace ar {

// ---- any type and alignment -----------------------------------------------------

// A tile of keys, then of values, in shared memory as binary32; a thread has one
// key and four rows of the scores, then one or two columns of the outputs and half
// of the rows.
constexpr int kRows = 16;             // query heads of a unit
constexpr int kAnyThreads = 256;
constexpr uint32_t kAnyTile = 64;

static size_t any_smem(uint32_t D) {
    return sizeof(float) * ((size_t)kRows * D + kAnyTile * (D | 1) + kRows * (kAnyTile + 1));
}

template <int DT, bool CACHE8>
__global__ void __launch_bounds__(kAnyThreads)
k_attention_any(const __grid_constant__ AttnArgs a) {
    extern __shared__ float smem[];
    __shared__ uint64_t scan[33];
    __shared__ float m_[kRows], l_[kRows], alpha_[kRows];
    __shared__ int2 place[kAnyTile];
    kernel_prologue();
    const uint32_t D = a.g.D, stride = D | 1, tid = threadIdx.x;
    float *qs = smem, *kv = qs + kRows * D, *sc = kv + kAnyTile * stride;
    if (tid == 0)
        WorkSpace(a.work).meta[blockIdx.x] = make_int4(0, 0, -1, 0);
    empty_rows<DT, kAnyTile>(a);
    uint64_t per;
    Cursor<kAnyTile> c = find_run<kAnyTile>(a, scan, &per);
    for (; !c.done(); c.next_unit(a)) {
        const UnitRows u = unit_rows(a, c.unit);
        const uint32_t b = c.b;
        __syncthreads();
        const uint8_t *q = a.q + (uint64_t)b * a.sq + (uint64_t)u.head * D * Elem<DT>::kSize;
        for (uint32_t i = tid; i < kRows * D; i += kAnyThreads)
            qs[i] = i < u.rows * D ? widen1<DT>(ld_elem<DT>(q, i)) : 0.0f;
        if (tid < kRows) {
            m_[tid] = -INFINITY;
            l_[tid] = 0.0f;
        }
        float acc[2][kRows / 2];          // columns tid % 128 (+ 128), rows of one half
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int r = 0; r < kRows / 2; ++r)
                acc[i][r] = 0.0f;
        for (uint32_t t = c.t; t < c.t1; ++t) {
            const uint32_t j0 = c.span.origin + t * kAnyTile;
            __syncthreads();              // the last tile is done with
            if (tid < kAnyTile) {
                const uint32_t j = j0 + tid;
                place[tid] = j < c.span.n ? make_int2(a.g.page_of(b, j), (int)a.g.slot_of(j))
                                          : make_int2(-1, 0);
            }
            __syncthreads();
            auto load = [&](const uint8_t *pool, const float *scales) {
                for (uint32_t i = tid; i < kAnyTile * D; i += kAnyThreads) {
                    const uint32_t r = i / D, d = i - r * D;
                    const int2 p = place[r];
                    float v = 0.0f;
                    if (p.x >= 0) {
                        const uint8_t *page = pool + (uint64_t)p.x * a.g.stride;
                        const uint32_t e = a.g.in_page(u.kv, p.y) + d;
                        if (CACHE8) {
                            uint32_t h;
                            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)page[e]));
                            v = __half2float(__ushort_as_half((unsigned short)h)) *
                                scales[a.g.scale_at(p.x, u.kv, p.y)];
                        } else {
                            v = widen1<DT>(ld_elem<DT>(page, e));
                        }
                    }
                    kv[r * stride + d] = v;
                }
            };
            load(a.g.k, a.g.ks);
            __syncthreads();
            {
                const uint32_t key = tid % kAnyTile, r0 = tid / kAnyTile * 4;
                float s[4] = {};
                if (r0 < u.rows)
                    for (uint32_t d = 0; d < D; ++d) {
                        const float k = kv[key * stride + d];
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            s[r] += qs[(r0 + r) * D + d] * k;
                    }
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    sc[(r0 + r) * (kAnyTile + 1) + key] =
                        place[key].x >= 0 ? s[r] * a.scale2 : -INFINITY;
            }
            __syncthreads();
            load(a.g.v, a.g.vs);
            for (uint32_t r = tid / 32; r < u.rows; r += kAnyThreads / 32) {
                float *row = sc + r * (kAnyTile + 1);
                const uint32_t lane = tid & 31;
                const float x = row[lane], y = row[lane + 32];
                // a NaN score makes its row NaN: the maximum must not drop it
                float top = fmaxf(x, y);
#pragma unroll
                for (int d = 16; d > 0; d >>= 1)
                    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
                const float was = m_[r], now = fmaxf(was, top), base = finite_max(now);
                const float p0 = exp2f(x - base), p1 = exp2f(y - base);
                const float sum = warp_sum(p0 + p1), al = exp2f(was - base);
                row[lane] = p0;
                row[lane + 32] = p1;
                __syncwarp();
                if (lane == 0) {
                    m_[r] = now;
                    l_[r] = l_[r] * al + sum;
                    alpha_[r] = al;
                }
            }
            __syncthreads();
            {
                const uint32_t d0 = tid % 128, r0 = tid / 128 * (kRows / 2);
                const uint32_t keys = c.span.n - j0 < kAnyTile ? c.span.n - j0 : kAnyTile;
                if (r0 < u.rows)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t d = d0 + 128 * i;
                        if (d >= D)
                            break;
#pragma unroll
                        for (int r = 0; r < kRows / 2; ++r)
                            if (r0 + r < u.rows)
                                acc[i][r] *= alpha_[r0 + r];
                        for (uint32_t k = 0; k < keys; ++k) {
                            const float v = kv[k * stride + d];
#pragma unroll
                            for (int r = 0; r < kRows / 2; ++r)
                                acc[i][r] += sc[(r0 + r) * (kAnyTile + 1) + k] * v;
                        }
                    }
            }
        }
        const int part = segment_part(a, c, per);
        const uint32_t r0 = tid / 128 * (kRows / 2);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t d = tid % 128 + 128 * i;
#pragma unroll
            for (int r = 0; r < kRows / 2; ++r) {
                if (d >= D || r0 + r >= u.rows)
                    continue;
                if (part < 0)
                    store_row<DT>(a.out + (uint64_t)b * a.sout, (u.head + r0 + r) * D + d,
                                  output_of(acc[i][r], l_[r0 + r]));
                else
                    WorkSpace(a.work).o[((uint64_t)part * a.unit_rows + r0 + r) * D + d] = acc[i][r];
            }
        }
        if (tid < u.rows) {
            if (part >= 0)
                WorkSpace(a.work).ml[part * a.unit_rows + tid] = make_float2(m_[tid], l_[tid]);
            else if (a.lse)
                a.lse[(uint64_t)b * a.heads + u.head + tid] = lse_of(m_[tid], l_[tid]);
        }
    }
}

// ---- the join ---------------------------------------------------------------------

// CTA (c, r): row r of the unit that begins in CTA c's run and ends in another's.  Its
// warps take a share of the parts each, VEC columns a lane at a time, and their sums
// are added in order.  Bound by latency: most CTAs find nothing to do, the others wait
// three times for memory.
constexpr int kJoinThreads = 128, kJoinWarps = kJoinThreads / 32;

template <int DT, int VEC> __global__ void __launch_bounds__(kJoinThreads)
k_attention_join(const __grid_constant__ AttnArgs a) {
    constexpr int kSteps = AR_CACHE_MAX_DIM / (32 * VEC);
    __shared__ float weight[kMaxCtas], part[kJoinWarps], sums[kJoinWarps - 1][AR_CACHE_MAX_DIM];
    wait_for_input();
    const WorkSpace w(a.work);
    const int c = blockIdx.x, r = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int4 meta = w.meta[c];
    if (meta.z < 0)
        return;
    const UnitRows u = unit_rows(a, (uint32_t)meta.y);
    if (r >= (int)u.rows)
        return;
    const int parts = meta.z - c + 1;
    const uint32_t D = a.g.D;
    auto slot = [&](int i) {
        return (uint32_t)(i == 0 ? 2 * c + 1 : 2 * (c + i)) * a.unit_rows + r;
    };
    float top = -INFINITY;
    for (int i = tid; i < parts; i += kJoinThreads)
        top = fmaxf(top, weight[i] = w.ml[slot(i)].x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
    if (lane == 0)
        part[warp] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kJoinWarps; ++i)
        top = fmaxf(top, part[i]);
    float l = 0.0f;
    for (int i = tid; i < parts; i += kJoinThreads) {
        weight[i] = exp2f(weight[i] - finite_max(top));
        l += w.ml[slot(i)].y * weight[i];
    }
    l = warp_sum(l);
    __syncthreads();
    if (lane == 0)
        part[warp] = l;
    float o[kSteps][VEC];
#pragma unroll
    for (int k = 0; k < kSteps; ++k)
#pragma unroll
        for (int v = 0; v < VEC; ++v)
            o[k][v] = 0.0f;
#pragma unroll 8
    for (int i = warp; i < parts; i += kJoinWarps) {
        const float *row = w.o + (uint64_t)slot(i) * D;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            const uint32_t d = (uint32_t)(k * 32 + lane) * VEC;
            if (d >= D)
                continue;
            if (VEC == 4) {
                const float4 x = *reinterpret_cast<const float4 *>(row + d);
                o[k][0] += x.x * weight[i];
                o[k][1 % VEC] += x.y * weight[i];
                o[k][2 % VEC] += x.z * weight[i];
                o[k][3 % VEC] += x.w * weight[i];
            } else {
                o[k][0] += row[d] * weight[i];
            }
        }
    }
    if (warp > 0)
#pragma unroll
        for (int k = 0; k < kSteps; ++k)
#pragma unroll
            for (int v = 0; v < VEC; ++v)
                sums[warp - 1][(k * 32 + lane) * VEC + v] = o[k][v];
    __syncthreads();
    if (warp > 0)
        return;
    l = part[0];
#pragma unroll
    for (int i = 1; i < kJoinWarps; ++i)
        l += part[i];
    uint8_t *out = a.out + (uint64_t)meta.x * a.sout;
#pragma unroll
    for (int k = 0; k < kSteps; ++k)
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const uint32_t d = (uint32_t)(k * 32 + lane) * VEC + v;
#pragma unroll
            for (int i = 0; i < kJoinWarps - 1; ++i)
                o[k][v] += sums[i][d];
            if (d < D)
                store_row<DT>(out, (u.head + r) * D + d, output_of(o[k][v], l));
        }
    if (lane == 0 && a.lse)
        a.lse[(uint64_t)meta.x * a.heads + u.head + r] = lse_of(top, l);
}

template <int DT, int VEC>
static cudaError_t join_form(const AttnArgs &a, int grid, cudaStream_t s) {
    const dim3 ctas(grid, a.group < a.unit_rows ? a.group : a.unit_rows);
    return launch_kernel(k_attention_join<DT, VEC>, ctas, kJoinThreads, 0, s, true, a);
}
template <int DT> static cudaError_t launch_join(const AttnArgs &a, int grid, cudaStream_t s) {
    return a.g.D % 4 == 0 ? join_form<DT, 4>(a, grid, s) : join_form<DT, 1>(a, grid, s);
}

template <int DT, bool CACHE8> static cudaError_t attention_any(const AttnArgs &a, cudaStream_t s) {
    const size_t smem = any_smem(a.g.D);
    cudaError_t e = opt_in_smem<k_attention_any<DT, CACHE8>>(any_smem(AR_CACHE_MAX_DIM));
    if (e != cudaSuccess)
        return e;
    const int sms = sm_count();
    if (sms < 1)
        return cudaErrorUnknown;
    const int grid = cta_limit(a.unit_rows, 2 * sms);
    e = launch_kernel(k_attention_any<DT, CACHE8>, grid, kAnyThreads, smem, s, true, a);
    return e != cudaSuccess ? e : launch_join<DT>(a, grid, s);
}

template <int DT>
static cudaError_t attention_dt(AttnArgs &a, bool e4m3, bool w, cudaStream_t s) {
    if (DT != AR_FP32 && w) {
        int grid = 0;
        const cudaError_t e = launch_attention_mma(a, DT, e4m3, &grid, s);
        return e != cudaSuccess ? e : launch_join<DT>(a, grid, s);
    }
    return e4m3 ? attention_any<DT, true>(a, s) : attention_any<DT, false>(a, s);
}

}  // namespace ar

using namespace ar;

extern "C" {

int ar_cache_attention(const void *q, size_t ldq, const void *kcache, const void *vcache,
                       size_t ldpage, const float *kscale, const float *vscale, size_t pages,
                       int page, const int32_t *table, size_t ldtable, size_t width,
                       const int32_t *lens, float scale, size_t window, void *out, size_t ldout,
                       float *lse, float *work, size_t work_bytes, size_t B, int heads,
                       int kv_heads, int D, int dtype, int cache_dtype, cudaStream_t stream) {
    AttnArgs a;
    const PagesCheck c = check_pages(kcache, vcache, ldpage, kscale, vscale, pages, page, table,
                                     ldtable, width, lens, B, kv_heads, D, dtype, cache_dtype,
                                     &a.g);
    if (c.rc != AR_OK)
        return c.rc;
    if (heads < 1 || heads % kv_heads != 0)
        return AR_ERR_INVALID;
    if (heads > AR_CACHE_MAX_HEADS)
        return AR_ERR_UNSUPPORTED;
    if (B == 0)
        return AR_OK;
    if (!q || !out || !work)
        return AR_ERR_INVALID;
    const size_t row = (size_t)heads * D, size = elem_size(dtype);
    const Matrix mq = matrix(q, ldq, B, row, size), mo = matrix(out, ldout, B, row, size);
    const Matrix ml = matrix(lse, 0, B, (size_t)heads, 4);
    const Matrix mw = matrix(work, 0, AR_CACHE_WORK_ROWS, (size_t)D + 2, 4);
    if (!mq.ok || !mo.ok || !ml.ok || !mw.ok || mw.p % 16 != 0 || work_bytes < mw.bytes)
        return AR_ERR_INVALID;
    const Matrix *outs[] = {&mo, &ml, &mw};
    for (const Matrix *m : outs)
        if (c.on(*m) || c.indexed(*m) || meet(*m, mq))
            return AR_ERR_INVALID;
    if (meet(mo, ml) || meet(mo, mw) || meet(ml, mw))
        return AR_ERR_INVALID;
    a.q = static_cast<const uint8_t *>(q);
    a.out = static_cast<uint8_t *>(out);
    a.lse = lse;
    a.work = work;
    a.sq = mq.stride;
    a.sout = mo.stride;
    a.scale2 = scale * kLog2E;
    a.B = (uint32_t)B;
    a.heads = (uint32_t)heads;
    a.group = (uint32_t)(heads / kv_heads);
    a.unit_rows = kRows;
    a.head_tiles = (a.group + kRows - 1) / kRows;
    a.runs = 0;
    a.window = window < ((size_t)1 << 31) ? (uint32_t)window : 0u;
    const bool e4m3 = cache_dtype == AR_E4M3;
    const bool w = pages > 0 && (size_t)D * (e4m3 ? 1 : size) % 16 == 0 && wide(c.k) && wide(c.v);
    switch (dtype) {
    case AR_BF16: return launched(attention_dt<AR_BF16>(a, e4m3, w, stream));
    case AR_FP16: return launched(attention_dt<AR_FP16>(a, e4m3, w, stream));
    default: return launched(attention_dt<AR_FP32>(a, e4m3, w, stream));
    }
}

}  // extern "C"
