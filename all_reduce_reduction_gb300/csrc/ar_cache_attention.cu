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

// Keys and values of binary32, or that are not 16-byte vectors.  Eight query heads are a
// unit; a warp has eight positions of every tile of 32 in shared memory as binary32,
// copied some tiles ahead where they are binary32 vectors and loaded by elements
// otherwise.  Scores: a lane has one key and every fourth 16 bytes of it, for all eight
// heads; the four lanes of a key then share the heads out.  Outputs: a lane has 4 columns
// (8 past D = 128) of all heads.  Bound by shared-memory reads and multiply-adds for many
// heads, by the copies' wait for few.
constexpr int kTeams = 4, kAnyThreads = 32 * kTeams;
constexpr uint32_t kAnyKeys = 8, kAnyHeads = 8, kAnyTile = kAnyKeys * kTeams;

template <int DC, bool ASYNC> struct AnyForm {
    static constexpr uint32_t kRow = DC * 4;
    static constexpr uint32_t kMask = 2 * kAnyKeys * kRow, kStage = kMask + 16;
    static constexpr int kStages = ASYNC ? 3 : 1;
    static constexpr uint32_t kRing = kTeams * kStages * kStage;
    static constexpr uint32_t kQ = kAnyHeads * kRow;
    static constexpr uint32_t kWeights = kAnyKeys * kAnyHeads * 4;           // of a warp
    static constexpr uint32_t kJoin = kTeams * 4 * kRow;                     // four heads
    static constexpr uint32_t kSmem = kRing + kQ + kTeams * kWeights + kJoin;
    static constexpr int kCtas = ASYNC ? (DC == 128 ? 2 : 1) : (DC == 128 ? 4 : 2);
    // 16 bytes c of row r; odd rows are exchanged so that two rows' reads share no bank
    static __device__ __forceinline__ uint32_t chunk(uint32_t r, uint32_t c) {
        return r * kRow + ((c ^ ((r & 1) << 2)) << 4);
    }
};

__device__ __forceinline__ void copy16(uint32_t to, const void *from, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                 :: "r"(to), "l"(from), "r"(bytes) : "memory");
}

template <int DT, bool CACHE8, int DC, bool ASYNC>
__global__ void __launch_bounds__(kAnyThreads, AnyForm<DC, ASYNC>::kCtas)
k_attention_any(const __grid_constant__ AttnArgs a) {
    using F = AnyForm<DC, ASYNC>;
    constexpr int J = DC / 128;                   // vectors of a row that a lane has
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t scan[32];
    __shared__ float team_m[kTeams][kAnyHeads], team_l[kTeams][kAnyHeads];
    const uint32_t D = a.g.D, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t vectors = (D + 15) / 16 * 4;   // of a row, whole groups of four
    uint8_t *ring = smem + warp * (F::kStages * F::kStage), *qs = smem + F::kRing;
    float *weights = reinterpret_cast<float *>(qs + F::kQ + warp * F::kWeights);
    float *join = reinterpret_cast<float *>(qs + F::kQ + kTeams * F::kWeights);
    const uint32_t ring_addr = (uint32_t)__cvta_generic_to_shared(ring);
    kernel_prologue();
    if (tid == 0)
        WorkSpace(a.work).meta[blockIdx.x] = make_int4(0, 0, -1, 0);
    empty_rows<DT, kAnyTile>(a);
    uint64_t per;
    Cursor<kAnyTile> c = find_run<kAnyTile>(a, scan, &per);

    // ---- the positions of a step to shared memory
    Cursor<kAnyTile> f = c;
    uint32_t slot = 0;
    int32_t page = -1;
    auto look_up = [&] {                          // lane r: of row r of the next step
        if (f.done())
            return;
        const uint32_t j = f.span.origin + f.t * kAnyTile + warp * kAnyKeys + (lane & 7);
        page = -1;
        if (j < f.span.n && j >= f.span.lo) {
            page = a.g.page_of(f.b, j);
            slot = a.g.slot_of(j);
        }
    };
    auto fetch = [&](uint32_t stage) {
        if (!f.done()) {
            const uint32_t kv = f.unit / a.head_tiles;
            constexpr uint32_t kCell = CACHE8 ? 1 : Elem<DT>::kSize;
            const uint64_t mine = page >= 0 ? (uint64_t)page * a.g.stride +
                                                  (uint64_t)a.g.in_page(kv, slot) * kCell
                                            : ~0ull;
            const uint32_t mask = __ballot_sync(0xFFFFFFFFu, page >= 0) & 255u;
            uint8_t *to = ring + stage * F::kStage;
            if constexpr (ASYNC) {
                const uint32_t at = ring_addr + stage * F::kStage;
#pragma unroll
                for (uint32_t r = 0; r < kAnyKeys; ++r) {
                    const uint64_t row = __shfl_sync(0xFFFFFFFFu, mine, r);
#pragma unroll
                    for (uint32_t j = 0; j < J; ++j) {
                        const uint32_t v = lane + 32 * j;
                        const bool on = row != ~0ull && v * 4 < D;
                        const uint64_t x = on ? row + v * 16 : 0;
                        if (v < vectors) {
                            copy16(at + F::chunk(r, v), a.g.k + x, on ? 16 : 0);
                            copy16(at + kAnyKeys * F::kRow + F::chunk(r, v), a.g.v + x,
                                   on ? 16 : 0);
                        }
                    }
                }
            } else {
                float ks = 1.0f, vs = 1.0f;
                if (CACHE8 && page >= 0) {
                    ks = a.g.ks[a.g.scale_at(page, kv, slot)];
                    vs = a.g.vs[a.g.scale_at(page, kv, slot)];
                }
                // eight rows' loads in flight, of 32 columns each
                for (uint32_t d0 = 0; d0 < 4 * vectors; d0 += 32) {
                    const uint32_t d = d0 + lane;
                    uint32_t k[kAnyKeys], v[kAnyKeys];
#pragma unroll
                    for (uint32_t r = 0; r < kAnyKeys; ++r) {
                        const uint64_t row = __shfl_sync(0xFFFFFFFFu, mine, r);
                        k[r] = v[r] = 0u;
                        if (row != ~0ull && d < D) {
                            if (CACHE8) {
                                k[r] = a.g.k[row + d];
                                v[r] = a.g.v[row + d];
                            } else {
                                k[r] = ld_elem<DT>(a.g.k + row, d);
                                v[r] = ld_elem<DT>(a.g.v + row, d);
                            }
                        }
                    }
#pragma unroll
                    for (uint32_t r = 0; r < kAnyKeys; ++r) {
                        float x, y;
                        if (CACHE8) {
                            uint32_t h, g;
                            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)k[r]));
                            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(g) : "h"((uint16_t)v[r]));
                            x = __half2float(__ushort_as_half((unsigned short)h)) *
                                __shfl_sync(0xFFFFFFFFu, ks, r);
                            y = __half2float(__ushort_as_half((unsigned short)g)) *
                                __shfl_sync(0xFFFFFFFFu, vs, r);
                            // a row that is not there: zeros, whatever its lane's scales
                            x = mask >> r & 1u ? x : 0.0f;
                            y = mask >> r & 1u ? y : 0.0f;
                        } else {
                            x = widen1<DT>(k[r]);
                            y = widen1<DT>(v[r]);
                        }
                        if (d < 4 * vectors) {
                            const uint32_t at = F::chunk(r, d / 4) + d % 4 * 4;
                            *reinterpret_cast<float *>(to + at) = x;
                            *reinterpret_cast<float *>(to + kAnyKeys * F::kRow + at) = y;
                        }
                    }
                }
            }
            if (lane == 0)
                *reinterpret_cast<uint32_t *>(to + F::kMask) = mask;
            f.next(a);
            look_up();
        }
        if (ASYNC)
            asm volatile("cp.async.commit_group;" ::: "memory");
    };
    look_up();
    if (ASYNC)
#pragma unroll
        for (int i = 0; i < F::kStages - 1; ++i)
            fetch(i);
    uint32_t stage = 0;
    const uint32_t key = lane / 4, quarter = lane % 4;

    while (!c.done()) {
        const UnitRows u = unit_rows(a, c.unit);
        const uint8_t *q = a.q + (uint64_t)c.b * a.sq + (uint64_t)u.head * D * Elem<DT>::kSize;
        for (uint32_t i = tid; i < kAnyHeads * DC; i += kAnyThreads) {
            const uint32_t r = i / DC, d = i % DC;
            reinterpret_cast<float *>(qs)[i] =
                r < u.rows && d < D ? widen1<DT>(ld_elem<DT>(q, r * D + d)) : 0.0f;
        }
        __syncthreads();
        // of this lane's heads 2 * quarter + {0, 1}: the running maximum, what scores are
        // compared with and taken relative to, the sum
        float m[2], bound[2], base[2], l[2];
        float o[J][kAnyHeads][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            m[i] = bound[i] = -INFINITY;
            base[i] = l[i] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (uint32_t h = 0; h < kAnyHeads; ++h)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o[j][h][i] = 0.0f;
        for (uint32_t t = c.t; t < c.t1; ++t) {
            if (ASYNC) {
                asm volatile("cp.async.wait_group %0;" :: "n"(F::kStages - 2) : "memory");
                __syncwarp();
                fetch((stage + F::kStages - 1) % F::kStages);
            } else {
                __syncwarp();                     // the step before is done with
                fetch(0);
                __syncwarp();
            }
            const uint8_t *here = ring + stage * F::kStage;
            const uint32_t mask = *reinterpret_cast<const uint32_t *>(here + F::kMask);
            float s[kAnyHeads][2];
#pragma unroll
            for (uint32_t h = 0; h < kAnyHeads; ++h)
                s[h][0] = s[h][1] = 0.0f;
#pragma unroll 2
            for (uint32_t v = quarter; v < vectors; v += 4) {
                const float4 k = *reinterpret_cast<const float4 *>(here + F::chunk(key, v));
#pragma unroll
                for (uint32_t h = 0; h < kAnyHeads; ++h) {
                    const float4 x = *reinterpret_cast<const float4 *>(qs + h * F::kRow + v * 16);
                    fma2(s[h], x.x, x.y, k.x, k.y);
                    fma2(s[h], x.z, x.w, k.z, k.w);
                }
            }
            // the four lanes of a key: half of the heads change hands, then a quarter
            float e[2];
            {
                float x[4], y[2];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float lo = s[j][0] + s[j][1], hi = s[4 + j][0] + s[4 + j][1];
                    x[j] = quarter & 2 ? hi : lo;
                    x[j] += __shfl_xor_sync(0xFFFFFFFFu, quarter & 2 ? lo : hi, 2);
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    y[j] = quarter & 1 ? x[2 + j] : x[j];
                    y[j] += __shfl_xor_sync(0xFFFFFFFFu, quarter & 1 ? x[j] : x[2 + j], 1);
                    e[j] = mask >> key & 1u ? y[j] * a.scale2 : -INFINITY;
                }
            }
            if (__any_sync(0xFFFFFFFFu, e[0] > bound[0] || e[1] > bound[1])) {
                float al[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float now = fmaxf(m[i], e[i]);
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1)
                        now = fmaxf(now, __shfl_xor_sync(0xFFFFFFFFu, now, d));
                    al[i] = exp2f(m[i] - finite_max(now));
                    m[i] = now;
                    bound[i] = now + kSlack;
                    base[i] = finite_max(now);
                    l[i] *= al[i];
                }
#pragma unroll
                for (uint32_t h = 0; h < kAnyHeads; ++h) {
                    const float by = __shfl_sync(0xFFFFFFFFu, al[h & 1], h / 2);
#pragma unroll
                    for (int j = 0; j < J; ++j) {
                        mul2(o[j][h], by, by);
                        mul2(o[j][h] + 2, by, by);
                    }
                }
            }
            const float2 p = make_float2(exp2f(e[0] - base[0]), exp2f(e[1] - base[1]));
            l[0] += p.x;
            l[1] += p.y;
            *reinterpret_cast<float2 *>(weights + key * kAnyHeads + 2 * quarter) = p;
            __syncwarp();
#pragma unroll 2
            for (uint32_t k = 0; k < kAnyKeys; ++k) {
                const float4 x = *reinterpret_cast<const float4 *>(weights + k * kAnyHeads);
                const float4 y = *reinterpret_cast<const float4 *>(weights + k * kAnyHeads + 4);
                const float w[kAnyHeads] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    const uint32_t v = lane + 32 * j;
                    if (v >= vectors)
                        continue;
                    const float4 g = *reinterpret_cast<const float4 *>(
                        here + kAnyKeys * F::kRow + F::chunk(k, v));
#pragma unroll
                    for (uint32_t h = 0; h < kAnyHeads; ++h) {
                        fma2(o[j][h], w[h], w[h], g.x, g.y);
                        fma2(o[j][h] + 2, w[h], w[h], g.z, g.w);
                    }
                }
            }
            stage = ASYNC ? (stage + 1) % F::kStages : 0;
        }
        const Cursor<kAnyTile> done = c;
        c.next_unit(a);

        // the teams' parts, in their order
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int d = 4; d < 32; d <<= 1)
                l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], d);
            if (key == 0) {
                team_m[warp][2 * quarter + i] = m[i];
                team_l[warp][2 * quarter + i] = l[i];
            }
        }
        __syncthreads();
        const int part = segment_part(a, done, per);
        auto total = [&](uint32_t h, float &sum) {        // of head h over the teams
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < kTeams; ++w)
                top = fmaxf(top, team_m[w][h]);
            sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kTeams; ++w)
                sum += team_l[w][h] * exp2f(team_m[w][h] - finite_max(top));
            return top;
        };
#pragma unroll
        for (uint32_t h0 = 0; h0 < kAnyHeads; h0 += 4) {
            if (h0 >= u.rows)
                break;
            if (h0 > 0)
                __syncthreads();
#pragma unroll
            for (uint32_t h = 0; h < 4; ++h) {
                float top = -INFINITY;
#pragma unroll
                for (int w = 0; w < kTeams; ++w)
                    top = fmaxf(top, team_m[w][h0 + h]);
                const float own = exp2f(team_m[warp][h0 + h] - finite_max(top));
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    const float *x = o[j][h0 + h];
                    *reinterpret_cast<float4 *>(join + (warp * 4 + h) * DC + (lane + 32 * j) * 4) =
                        make_float4(x[0] * own, x[1] * own, x[2] * own, x[3] * own);
                }
            }
            __syncthreads();
            for (uint32_t i = tid; i < 4 * DC; i += kAnyThreads) {
                const uint32_t h = h0 + i / DC, d = i % DC;
                if (h >= u.rows || d >= D)
                    continue;
                float v = join[i];
#pragma unroll
                for (int w = 1; w < kTeams; ++w)
                    v += join[w * 4 * DC + i];
                if (part < 0) {
                    float sum;
                    total(h, sum);
                    store_row<DT>(a.out + (uint64_t)done.b * a.sout, (u.head + h) * D + d,
                                  output_of(v, sum));
                } else {
                    WorkSpace(a.work).o[((uint64_t)part * kAnyHeads + h) * D + d] = v;
                }
            }
        }
        if (tid < u.rows) {
            float sum;
            const float top = total(tid, sum);
            if (part >= 0)
                WorkSpace(a.work).ml[part * kAnyHeads + tid] = make_float2(top, sum);
            else if (a.lse)
                a.lse[(uint64_t)done.b * a.heads + u.head + tid] = lse_of(top, sum);
        }
        __syncthreads();                          // before the next unit's q and sums
    }
    if (ASYNC)
        asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// ---- the join ---------------------------------------------------------------------

// CTA (c, r): row r of the unit that begins in CTA c's run and ends in another's.  Its
// warps take a share of the parts each, VEC columns a lane at a time, and their sums
// are added in order.  Bound by latency: most CTAs find nothing to do, the others wait
// three times for memory.
constexpr int kJoinThreads = 128, kJoinWarps = kJoinThreads / 32;

// This lane's columns of a row of D; zeros past it.
template <int STEPS, int VEC>
__device__ __forceinline__ void load_part(float (&x)[STEPS][VEC], const float *row, uint32_t D) {
#pragma unroll
    for (int k = 0; k < STEPS; ++k) {
        const uint32_t d = (uint32_t)(k * 32 + (threadIdx.x & 31)) * VEC;
#pragma unroll
        for (int v = 0; v < VEC; ++v)
            x[k][v] = 0.0f;
        if (d >= D)
            continue;
        if constexpr (VEC == 4) {
            const float4 f = *reinterpret_cast<const float4 *>(row + d);
            x[k][0] = f.x;
            x[k][1] = f.y;
            x[k][2] = f.z;
            x[k][3] = f.w;
        } else {
            x[k][0] = row[d];
        }
    }
}

template <int DT, int VEC> __global__ void __launch_bounds__(kJoinThreads)
k_attention_join(const __grid_constant__ AttnArgs a) {
    constexpr int kSteps = AR_CACHE_MAX_DIM / (32 * VEC);
    __shared__ float weight[kMaxCtas], part[kJoinWarps], sums[kJoinWarps - 1][AR_CACHE_MAX_DIM];
    wait_for_input();
    const WorkSpace w(a.work);
    const int c = blockIdx.x, r = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t D = a.g.D;
    auto slot = [&](int i) {
        return (uint32_t)(i == 0 ? 2 * c + 1 : 2 * (c + i)) * a.unit_rows + r;
    };
    // what this warp adds first, before it is known whether there is that much: the place
    // is one of the workspace's, and most units have two parts
    float ahead[kSteps][VEC] = {};
    float2 ahead_ml = make_float2(0.0f, 0.0f);
    if (warp < 2 && c + warp < (int)gridDim.x)
        load_part(ahead, w.o + (uint64_t)slot(warp) * D, D);
    if (c + tid < (int)gridDim.x)
        ahead_ml = w.ml[slot(tid)];
    const int4 meta = w.meta[c];
    if (meta.z < 0)
        return;
    const UnitRows u = unit_rows(a, (uint32_t)meta.y);
    if (r >= (int)u.rows)
        return;
    const int parts = meta.z - c + 1;
    float top = -INFINITY;
    for (int i = tid; i < parts; i += kJoinThreads)
        top = fmaxf(top, weight[i] = (i == tid ? ahead_ml : w.ml[slot(i)]).x);
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
        l += (i == tid ? ahead_ml : w.ml[slot(i)]).y * weight[i];
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
    auto add = [&](const float (*x)[VEC], float by) {
#pragma unroll
        for (int k = 0; k < kSteps; ++k)
#pragma unroll
            for (int v = 0; v < VEC; ++v)
                o[k][v] += x[k][v] * by;
    };
    if (warp < 2 && warp < parts)
        add(ahead, weight[warp]);
#pragma unroll 4
    for (int i = warp < 2 ? warp + kJoinWarps : warp; i < parts; i += kJoinWarps) {
        float x[kSteps][VEC];
        load_part(x, w.o + (uint64_t)slot(i) * D, D);
        add(x, weight[i]);
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

template <int DT, bool CACHE8, int DC, bool ASYNC>
static cudaError_t any_form(AttnArgs &a, cudaStream_t s) {
    using F = AnyForm<DC, ASYNC>;
    cudaError_t e = opt_in_smem<k_attention_any<DT, CACHE8, DC, ASYNC>>(F::kSmem);
    if (e != cudaSuccess)
        return e;
    const int sms = sm_count();
    if (sms < 1)
        return cudaErrorUnknown;
    a.unit_rows = kAnyHeads;
    a.head_tiles = (a.group + kAnyHeads - 1) / kAnyHeads;
    a.runs = 0;
    a.cluster = 0;
    const int grid = cta_limit(a.unit_rows, F::kCtas * sms);
    e = launch_kernel(k_attention_any<DT, CACHE8, DC, ASYNC>, grid, kAnyThreads, F::kSmem, s, true,
                      a);
    return e != cudaSuccess ? e : launch_join<DT>(a, grid, s);
}

// w: keys and values are whole 16-byte vectors on 16-byte boundaries.
template <int DT> static cudaError_t attention_dt(AttnArgs &a, bool e4m3, bool w, cudaStream_t s) {
    if (w && (DT != AR_FP32 || e4m3)) {
        int grid = 0;
        const cudaError_t e = launch_attention_mma(a, DT, e4m3, &grid, s);
        return e != cudaSuccess || grid == 0 ? e : launch_join<DT>(a, grid, s);
    }
    if constexpr (DT == AR_FP32)
        if (w)
            return a.g.D <= 128 ? any_form<DT, false, 128, true>(a, s)
                                : any_form<DT, false, 256, true>(a, s);
    if (e4m3)
        return a.g.D <= 128 ? any_form<DT, true, 128, false>(a, s)
                            : any_form<DT, true, 256, false>(a, s);
    return a.g.D <= 128 ? any_form<DT, false, 128, false>(a, s)
                        : any_form<DT, false, 256, false>(a, s);
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
    a.unit_rows = a.head_tiles = a.cluster = 0;           // by the form
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
