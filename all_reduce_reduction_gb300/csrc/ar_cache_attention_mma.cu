// Attention over the paged cache on the tensor cores, for keys and values of two
// bytes (in the type of q) or one (E4M3, in binary16).
//
// Up to 16 query heads that share a key-value head are the 16 rows of a warp's
// products: s = q k' and o += p v for 16 positions at a time.  A warp has its own
// positions of every tile, its own ring of them in shared memory, filled by
// background copies a few tiles ahead (across the ends of units), and its own
// running maximum and sums; nothing waits for another warp until a unit ends.
#include "ar_cache_attention.cuh"
#include "ar_mma.cuh"

namespace ar {

constexpr int kMmaWarps = 4, kMmaThreads = 32 * kMmaWarps;
constexpr uint32_t kMmaTile = 16 * kMmaWarps;

// With E4M3 values the weights are 2^14 times what they are, the most of binary16's
// range; log2 of what a value's scale counts as at least.
constexpr float kWeightBits = 14.0f, kWeightUnit = 0x1p-14f, kLeastScale = -96.0f;

__device__ __forceinline__ uint32_t shared_addr(const void *p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void ldmatrix4(uint32_t r[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t r[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// 16 bytes to shared memory in the background; `bytes` of them, the rest zeros.
__device__ __forceinline__ void fetch16(uint32_t to, const void *from, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                 :: "r"(to), "l"(from), "r"(bytes) : "memory");
}
__device__ __forceinline__ void fetch4(uint32_t to, const void *from, uint32_t bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;"
                 :: "r"(to), "l"(from), "r"(bytes) : "memory");
}
__device__ __forceinline__ void fetch_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int LEFT> __device__ __forceinline__ void fetch_wait() {
    asm volatile("cp.async.wait_group %0;" :: "n"(LEFT) : "memory");
}
__device__ __forceinline__ float exp2_approx(float x) {        // within 2^-22
    float y;
    asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
template <int DT> __device__ __forceinline__ uint32_t pack2(float a, float b) {
    return DT == AR_BF16 ? narrow2<AR_BF16>(a, b) : narrow2<AR_FP16>(a, b);
}

template <int DT, bool CACHE8, int DC> struct MmaForm {
    static constexpr int kType = CACHE8 ? (int)AR_FP16 : DT;      // of the products
    static constexpr uint32_t kCell = CACHE8 ? 1 : 2;
    static constexpr uint32_t kRow = DC * kCell;                   // bytes of a row in shared memory
    static constexpr uint32_t kChunks = kRow / 16;
    // a warp's stage: 16 keys, 16 values, their scales, which positions are there
    static constexpr uint32_t kScales = 32 * kRow, kMask = kScales + (CACHE8 ? 128 : 0);
    static constexpr uint32_t kStage = kMask + 16;
    static constexpr int kStages = 3;
    static constexpr uint32_t kRing = kMmaWarps * kStages * kStage;
    static constexpr uint32_t kQ = kRows * DC * 2;
    // columns that the warps join at a time
    static constexpr int kJoin = CACHE8 && DC == 256 ? 16 : 32;
    static constexpr uint32_t kJoinRow = kJoin + 2;
    static constexpr uint32_t kSmem = kRing + kQ + 4 * kMmaWarps * kRows * kJoinRow;
    static constexpr int kCtas = DC == 256 ? (CACHE8 ? 2 : 1) : DC == 128 ? (CACHE8 ? 3 : 2) : 3;

    // chunk c of row r: the rows of a group of eight lie in different banks
    static __device__ __forceinline__ uint32_t chunk(uint32_t r, uint32_t c) {
        return r * kRow + ((kChunks >= 8 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) << 4);
    }
    static __device__ __forceinline__ uint32_t q_chunk(uint32_t r, uint32_t c) {
        return r * (DC * 2) + ((c ^ (r & 7)) << 4);
    }
    // where element d of q lies in its row: in 16 columns, the order in which four
    // codes of a lane enter a product
    static __device__ __forceinline__ uint32_t q_column(uint32_t d) {
        if (!CACHE8)
            return d;
        const uint32_t c = d % 16 / 4, i = d % 4;
        return d / 16 * 16 + (i < 2 ? 2 * c + i : 8 + 2 * c + i - 2);
    }
};

template <int DT, bool CACHE8, int DC>
__global__ void __launch_bounds__(kMmaThreads, MmaForm<DT, CACHE8, DC>::kCtas)
k_attention_mma(const __grid_constant__ AttnArgs a) {
    using M = MmaForm<DT, CACHE8, DC>;
    constexpr bool kKeepQ = DC <= 128;       // q's operands stay in registers
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t scan[33];
    __shared__ float warp_m[kMmaWarps][kRows], warp_l[kMmaWarps][kRows], row_scale[kRows];
    uint8_t *qs = smem + M::kRing;
    float *join = reinterpret_cast<float *>(qs + M::kQ);
    const uint32_t D = a.g.D, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint8_t *ring = smem + warp * (M::kStages * M::kStage);
    const uint32_t ring_addr = shared_addr(ring), q_addr = shared_addr(qs);
    kernel_prologue();
    if (tid == 0)
        WorkSpace(a.work).meta[blockIdx.x] = make_int4(0, 0, -1, 0);
    empty_rows<DT, kMmaTile>(a);
    uint64_t per, start;
    Cursor<kMmaTile> c = find_run<kMmaTile>(a, scan, &per, &start);
    uint64_t index = start;

    // ---- the copies, some tiles ahead
    Cursor<kMmaTile> f = c;
    const uint32_t my_row = warp * 16 + (lane & 15);       // of a tile
    uint32_t slot = 0;
    int32_t page = -1;
    auto look_up = [&] {                                   // of the next tile to fetch
        if (f.done())
            return;
        const uint32_t j = f.span.lo + f.t * kMmaTile + my_row;
        page = -1;
        if (j < f.span.n) {
            page = a.g.page_of(f.b, j);
            slot = j % a.g.page;
        }
    };
    auto fetch = [&](uint32_t stage) {
        if (!f.done()) {
            const uint32_t kv = f.unit / a.head_tiles;
            const uint32_t to = ring_addr + stage * M::kStage;
            const bool on = page >= 0;
            const uint64_t at = on ? (uint64_t)page * a.g.stride +
                                         (uint64_t)a.g.in_page(kv, slot) * M::kCell
                                   : ~0ull;
            const uint32_t mask = __ballot_sync(0xFFFFFFFFu, on) & 0xFFFFu;
#pragma unroll
            for (uint32_t i = 0; i < M::kChunks / 2; ++i) {
                const uint32_t r = (i * 32 + lane) / M::kChunks, ch = (i * 32 + lane) % M::kChunks;
                const uint64_t row = __shfl_sync(0xFFFFFFFFu, at, r);
                const bool whole = row != ~0ull && ch * 16 < D * M::kCell;
                const uint64_t from = whole ? row + ch * 16 : 0;
                fetch16(to + M::chunk(r, ch), a.g.k + from, whole ? 16 : 0);
                fetch16(to + 16 * M::kRow + M::chunk(r, ch), a.g.v + from, whole ? 16 : 0);
            }
            if (CACHE8) {
                const float *scales = lane < 16 ? a.g.ks : a.g.vs;
                fetch4(to + M::kScales + lane * 4, scales + (on ? a.g.scale_at(page, kv, slot) : 0),
                       on ? 4 : 0);
            }
            if (lane == 0)
                *reinterpret_cast<uint32_t *>(ring + stage * M::kStage + M::kMask) = mask;
            f.next(a);
            look_up();
        }
        fetch_commit();
    };
    look_up();
#pragma unroll
    for (int i = 0; i < M::kStages - 1; ++i)
        fetch(i);
    uint32_t stage = 0;

    // operands' places: lane l gives the address of row l % 8 of matrix l / 8
    const uint32_t k_row = lane % 8 + (CACHE8 ? (lane / 8 & 1) : lane / 16) * 8;
    const uint32_t k_chunk = CACHE8 ? lane / 16 : (lane / 8 & 1);
    const uint32_t v_row = lane % 8 + (lane / 8 & 1) * 8, v_chunk = lane / 16;
    const uint32_t q_row = lane % 16, q_part = lane / 16;

    while (!c.done()) {
        const UnitRows u = unit_rows(a, c.unit);
        const uint32_t b = c.b, unit = c.unit, t0 = c.t, tiles = c.tiles;
        // q, a warp to a row: binary16 after scaling by a power of two where the cache is E4M3
        for (uint32_t r = warp; r < kRows; r += kMmaWarps) {
            const uint8_t *q = a.q + (uint64_t)b * a.sq + (uint64_t)(u.head + r) * D * 2;
            float v[DC / 32], top = 0.0f;
#pragma unroll
            for (int i = 0; i < DC / 32; ++i) {
                const uint32_t d = lane + 32 * i;
                v[i] = r < u.rows && d < D ? widen1<DT>(ld_elem<DT>(q, d)) : 0.0f;
                top = fmaxf(top, fabsf(v[i]));
            }
            float up = 1.0f, back = 1.0f;
            if (CACHE8) {
#pragma unroll
                for (int d = 16; d > 0; d >>= 1)
                    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
                half_range(top, up, back);
            }
#pragma unroll
            for (int i = 0; i < DC / 32; ++i) {
                const uint32_t e = M::q_column(lane + 32 * i);
                *reinterpret_cast<uint16_t *>(qs + M::q_chunk(r, e / 8) + e % 8 * 2) =
                    (uint16_t)narrow1<M::kType>(v[i] * up);
            }
            if (lane == 0)
                row_scale[r] = a.scale2 * back;
        }
        __syncthreads();
        uint32_t qf[kKeepQ ? DC / 16 : 1][4];
        if (kKeepQ)
#pragma unroll
            for (int k = 0; k < DC / 16; ++k)
                ldmatrix4(qf[kKeepQ ? k : 0], q_addr + M::q_chunk(q_row, 2 * k + q_part));
        const float scale[2] = {row_scale[lane / 4], row_scale[lane / 4 + 8]};
        float o[DC / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
        for (int n = 0; n < DC / 8; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[n][i] = 0.0f;

        uint32_t t = t0;
        for (;;) {
            fetch_wait<M::kStages - 2>();
            __syncwarp();
            // every lane is done with the stage before this one
            fetch((stage + M::kStages - 1) % M::kStages);
            const uint32_t at = ring_addr + stage * M::kStage;
            const uint8_t *here = ring + stage * M::kStage;
            const uint32_t mask = *reinterpret_cast<const uint32_t *>(here + M::kMask);
            // scores: position 2 * (lane % 4) + {0, 1} (+ 8) of rows lane / 4 (0, 1) and + 8 (2, 3)
            float s[2][4] = {};
            if (CACHE8) {
#pragma unroll
                for (int k = 0; k < DC / 16; k += 2) {
                    if (k * 16 >= (int)D)
                        break;
                    uint32_t w[4], b0, b1;
                    ldmatrix4(w, at + M::chunk(k_row, k + k_chunk));
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint32_t qx[4];
                        if (!kKeepQ)
                            ldmatrix4(qx, q_addr + M::q_chunk(q_row, 2 * (k + i) + q_part));
                        const uint32_t *qa = kKeepQ ? qf[kKeepQ ? k + i : 0] : qx;
                        from_e4m3x4(w[2 * i], b0, b1);
                        mma16<M::kType>(s[0], qa, b0, b1);
                        from_e4m3x4(w[2 * i + 1], b0, b1);
                        mma16<M::kType>(s[1], qa, b0, b1);
                    }
                }
            } else {
#pragma unroll
                for (int k = 0; k < DC / 16; ++k) {
                    if (k * 16 >= (int)D)
                        break;
                    uint32_t w[4], qx[4];
                    ldmatrix4(w, at + M::chunk(k_row, 2 * k + k_chunk));
                    if (!kKeepQ)
                        ldmatrix4(qx, q_addr + M::q_chunk(q_row, 2 * k + q_part));
                    const uint32_t *qa = kKeepQ ? qf[kKeepQ ? k : 0] : qx;
                    mma16<M::kType>(s[0], qa, w[0], w[1]);
                    mma16<M::kType>(s[1], qa, w[2], w[3]);
                }
            }
            // The scale of a value goes into its position's weight, as an exponent (e), and
            // into the running maximum, so that the weights fit binary16.  The maximum counts
            // it as 2^-96 at least: then l, which has the scores alone, stays finite.
            float e[2][4], lead[2][4];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                float2 ks = make_float2(1.0f, 1.0f), vs = make_float2(0.0f, 0.0f);
                if (CACHE8) {
                    const float *scales = reinterpret_cast<const float *>(here + M::kScales) + 8 * n +
                                          lane % 4 * 2;
                    ks = *reinterpret_cast<const float2 *>(scales);
                    const float2 w = *reinterpret_cast<const float2 *>(scales + 16);
                    vs = make_float2(log2f(w.x), log2f(w.y));
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s[n][i] *= CACHE8 ? scale[i / 2] * (i & 1 ? ks.y : ks.x) : scale[i / 2];
                    e[n][i] = CACHE8 ? s[n][i] + (i & 1 ? vs.y : vs.x) : s[n][i];
                    lead[n][i] = CACHE8 ? s[n][i] + fmaxf(i & 1 ? vs.y : vs.x, kLeastScale)
                                        : s[n][i];
                }
            }
            if (mask != 0xFFFFu) {
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (!(mask >> (8 * n + lane % 4 * 2 + (i & 1)) & 1u))
                            s[n][i] = e[n][i] = lead[n][i] = -INFINITY;
            }
            float top[2], base[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                top[h] = fmaxf(fmaxf(lead[0][2 * h], lead[0][2 * h + 1]),
                               fmaxf(lead[1][2 * h], lead[1][2 * h + 1]));
                top[h] = fmaxf(top[h], __shfl_xor_sync(0xFFFFFFFFu, top[h], 1));
                top[h] = fmaxf(top[h], __shfl_xor_sync(0xFFFFFFFFu, top[h], 2));
            }
            if (__any_sync(0xFFFFFFFFu, top[0] > m[0] || top[1] > m[1])) {
                float al[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float now = fmaxf(m[h], top[h]);
                    al[h] = exp2_approx(m[h] - finite_max(now));
                    m[h] = now;
                    l[h] *= al[h];
                }
#pragma unroll
                for (int n = 0; n < DC / 8; ++n) {
                    mul2(o[n], al[0], al[0]);
                    mul2(o[n] + 2, al[1], al[1]);
                }
            }
            base[0] = finite_max(m[0]);
            base[1] = finite_max(m[1]);
            float p[2][4];
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    p[n][i] = exp2_approx(CACHE8 ? e[n][i] - base[i / 2] + kWeightBits
                                                 : e[n][i] - base[i / 2]);
                    l[i / 2] += CACHE8 ? exp2_approx(s[n][i] - base[i / 2]) : p[n][i];
                }
            // in two parts: one would keep 8 (bf16) or 11 bits of a weight
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float *x = p[i / 2] + 2 * (i & 1);
                hi[i] = pack2<M::kType>(x[0], x[1]);
                const float2 w = widen2<M::kType>(hi[i]);
                lo[i] = pack2<M::kType>(x[0] - w.x, x[1] - w.y);
            }
            const uint32_t v_at = at + 16 * M::kRow;
            if (CACHE8) {
#pragma unroll
                for (int n = 0; n < DC / 16; n += 2) {
                    if (n * 16 >= (int)D)
                        break;
                    uint32_t w[4];
                    ldmatrix4_trans(w, v_at + M::chunk(v_row, n + v_chunk));
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        // a word holds two columns of two positions: to two positions of each
                        uint32_t e0, e1, d0, d1;
                        from_e4m3x4(__byte_perm(w[2 * i], 0, 0x3120), e0, d0);
                        from_e4m3x4(__byte_perm(w[2 * i + 1], 0, 0x3120), e1, d1);
                        float *even = o[2 * (n + i)], *odd = o[2 * (n + i) + 1];
                        mma16<M::kType>(even, hi, e0, e1);
                        mma16<M::kType>(odd, hi, d0, d1);
                        mma16<M::kType>(even, lo, e0, e1);
                        mma16<M::kType>(odd, lo, d0, d1);
                    }
                }
            } else {
#pragma unroll
                for (int n = 0; n < DC / 16; ++n) {
                    if (n * 16 >= (int)D)
                        break;
                    uint32_t w[4];
                    ldmatrix4_trans(w, v_at + M::chunk(v_row, 2 * n + v_chunk));
                    mma16<M::kType>(o[2 * n], hi, w[0], w[1]);
                    mma16<M::kType>(o[2 * n + 1], hi, w[2], w[3]);
                    mma16<M::kType>(o[2 * n], lo, w[0], w[1]);
                    mma16<M::kType>(o[2 * n + 1], lo, w[2], w[3]);
                }
            }
            stage = (stage + 1) % M::kStages;
            ++t;
            ++index;
            const bool more = c.left > 1 && t < tiles;
            c.next(a);
            if (!more)
                break;
        }

        // the warps' parts, in their order
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(0xFFFFFFFFu, l[h], 1);
            l[h] += __shfl_xor_sync(0xFFFFFFFFu, l[h], 2);
            if (lane % 4 == 0) {
                warp_m[warp][lane / 4 + 8 * h] = m[h];
                warp_l[warp][lane / 4 + 8 * h] = l[h];
            }
        }
        __syncthreads();
        const int part = segment_part<kMmaTile>(a, b, unit, t0, t, tiles, per, index - t);
        float own[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float all = -INFINITY;
#pragma unroll
            for (int w = 0; w < kMmaWarps; ++w)
                all = fmaxf(all, warp_m[w][lane / 4 + 8 * h]);
            own[h] = exp2_approx(m[h] - finite_max(all)) * (CACHE8 ? kWeightUnit : 1.0f);
        }
        // the row that this thread finishes: four columns (or two) at a time
        const uint32_t row = tid / 8;
        float row_m = -INFINITY, row_l = 0.0f;
#pragma unroll
        for (int w = 0; w < kMmaWarps; ++w)
            row_m = fmaxf(row_m, warp_m[w][row]);
#pragma unroll
        for (int w = 0; w < kMmaWarps; ++w)
            row_l += warp_l[w][row] * exp2_approx(warp_m[w][row] - finite_max(row_m));
#pragma unroll
        for (int d0 = 0; d0 < DC; d0 += M::kJoin) {
            if (d0 >= (int)D)
                break;
            if (d0 > 0)
                __syncthreads();
            float *mine = join + warp * kRows * M::kJoinRow + lane / 4 * M::kJoinRow;
#pragma unroll
            for (int n = 0; n < M::kJoin / 8; ++n) {
                const float *x = o[d0 / 8 + n];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t d = CACHE8 ? n / 2 * 16 + lane % 4 * 4 + (i & 1) * 2 + (n & 1)
                                              : n * 8 + lane % 4 * 2 + (i & 1);
                    mine[i / 2 * 8 * M::kJoinRow + d] = x[i] * own[i / 2];
                }
            }
            __syncthreads();
            constexpr int kEach = M::kJoin / 8;
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const uint32_t at = row * M::kJoinRow + tid % 8 + 8 * i, d = d0 + tid % 8 + 8 * i;
                float v = join[at];
#pragma unroll
                for (int w = 1; w < kMmaWarps; ++w)
                    v += join[w * kRows * M::kJoinRow + at];
                if (row >= u.rows || d >= D)
                    continue;
                if (part < 0)
                    store_row<DT>(a.out + (uint64_t)b * a.sout, (u.head + row) * D + d,
                                  output_of(v, row_l));
                else
                    WorkSpace(a.work).o[((uint64_t)part * kRows + row) * D + d] = v;
            }
        }
        if (tid % 8 == 0 && row < u.rows) {
            if (part >= 0)
                WorkSpace(a.work).ml[part * kRows + row] = make_float2(row_m, row_l);
            else if (a.lse)
                a.lse[(uint64_t)b * a.heads + u.head + row] = lse_of(row_m, row_l);
        }
    }
    fetch_wait<0>();
}

template <int DT, bool CACHE8, int DC>
static cudaError_t mma_form(const AttnArgs &a, int *grid, cudaStream_t s) {
    using M = MmaForm<DT, CACHE8, DC>;
    const cudaError_t e = opt_in_smem<k_attention_mma<DT, CACHE8, DC>>(M::kSmem);
    if (e != cudaSuccess)
        return e;
    const int sms = sm_count();
    if (sms < 1)
        return cudaErrorUnknown;
    *grid = M::kCtas * sms < kMaxCtas ? M::kCtas * sms : kMaxCtas;
    return launch_kernel(k_attention_mma<DT, CACHE8, DC>, *grid, kMmaThreads, M::kSmem, s, true, a);
}

template <int DT, bool CACHE8>
static cudaError_t mma_dim(const AttnArgs &a, int *grid, cudaStream_t s) {
    return a.g.D <= 64    ? mma_form<DT, CACHE8, 64>(a, grid, s)
           : a.g.D <= 128 ? mma_form<DT, CACHE8, 128>(a, grid, s)
                          : mma_form<DT, CACHE8, 256>(a, grid, s);
}

cudaError_t launch_attention_mma(const AttnArgs &a, int dtype, bool e4m3, int *grid,
                                 cudaStream_t s) {
    if (dtype == AR_BF16)
        return e4m3 ? mma_dim<AR_BF16, true>(a, grid, s) : mma_dim<AR_BF16, false>(a, grid, s);
    return e4m3 ? mma_dim<AR_FP16, true>(a, grid, s) : mma_dim<AR_FP16, false>(a, grid, s);
}

}  // namespace ar
