// The kernel of attention over the paged cache on the tensor cores, for keys and values of two
// bytes (in the type of q) or one (E4M3, in binary16; q then too, in two parts where it
// is binary32).
//
// A warp's products have 16 positions by 8 query heads that share a key-value head:
// s' = k q', then o' += v' p', so that keys and values are the operand of 16 rows and
// heads fill the columns.  Four groups of warps have 16 positions of every tile each,
// in their own ring in shared memory, filled by background copies a few tiles ahead
// (across the ends of units); the 1, 2 or 4 warps of a group take 8 heads each of the
// same positions.  A warp has its own running maximum and sums; groups wait for one
// another only where a unit ends.
//
// One sequence of 131072, 64 / 8 heads of 128 bf16: 96 us with the join (5.6 TB/s); 64
// sequences of 256 to 16384 in 8 bits 117 (5.1; bound by issue beside the stream: 484
// instructions for 16 positions); 32 query heads of 256 on one of keys 44 (1.7; the join of
// the teams' outputs).  With the heads as rows of the products 220 and 92 for the last two.
#pragma once

#include "ar_cache_attention.cuh"
#include "ar_cluster.cuh"
#include "ar_mma.cuh"

namespace ar {

constexpr int kTeams = 4;                     // of warps, 16 positions of a tile each
constexpr uint32_t kMmaTile = 16 * kTeams;

// Products in binary16 (caches of binary16 and E4M3): a weight is held as two such numbers,
// which end at 2^-25, so weights are 2^kBits times what they are relative to the maximum
// (2^15 at most, with the slack).  A weight below kSmall would then have fewer than 12 bits
// where the output is bf16, 14 where it is binary16, 16 where it is binary32.  Where a warp
// has one among its 16 positions, what the two numbers leave of weights below 1 is added in
// a product of its own, 2^24 times as large: they end at 2^-49 then.  (Batch in 8 bits as
// above, scores of standard deviation 2.2: 117 us; with 14 bits 120, without any of it 113.)
constexpr float kRestScale = 0x1p24f;

// E4M3 values: a weight times its value's scale is what is held, so the maximum is that of
// score + log2 scale (whole exponents, -96 at least: the sum of the weights alone stays
// finite).  Scales that ar_cache_write gives are 2^-105 at least; where the output is
// binary32, smaller ones count in full too: the sum of the weights alone then has a maximum
// of its own.
constexpr float kLeastScale = -96.0f;

// A scale as f * 2^e with f in [1, 2); e is -inf for 0, f what is not finite.
__device__ __forceinline__ void split_scale(float v, float &e, float &f) {
    const bool tiny = v < 0x1p-100f;
    const uint32_t bits = __float_as_uint(tiny ? v * 0x1p100f : v);
    const int exponent = (int)(bits >> 23);
    e = v == 0.0f ? -INFINITY : (float)(exponent - 127 - (tiny ? 100 : 0));
    f = __uint_as_float((bits & 0x7FFFFFu) | 0x3F800000u);
    if (exponent == 255) {
        e = 0.0f;
        f = v;
    }
}

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
// 16 bytes to shared memory in the background.
__device__ __forceinline__ void fetch16(uint32_t to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(to), "l"(from) : "memory");
}
// `bytes` of them, the rest zeros.
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
// Within 2^-22; results below 2^-126 are 0.
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The transposed 8 x 8 matrix of two-byte elements, a row of it in four lanes.
__device__ __forceinline__ uint32_t transpose8(uint32_t w) {
    uint32_t t;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(t) : "r"(w));
    return t;
}
template <int DT> __device__ __forceinline__ uint32_t pack2(float a, float b) {
    return DT == AR_BF16 ? narrow2<AR_BF16>(a, b) : narrow2<AR_FP16>(a, b);
}
// The same, rounded toward zero.
template <int DT> __device__ __forceinline__ uint32_t pack2_down(float a, float b) {
    uint32_t w;
    if (DT == AR_BF16)
        asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(b), "f"(a));
    else
        asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(b), "f"(a));
    return w;
}
// Two weights in two parts.  E4M3 values are finite, and both parts rounded to the nearest.
// Otherwise an infinity among the values has to remain one times either part: the first is
// rounded down, and the second is more than what is left, by 2^-23 of the weight (bf16) or so
// that it is 2^-24 at least (binary16; a weight that is 0 or less than 2^-24 needs
// positive_parts).
template <int TYPE, bool CACHE8>
__device__ __forceinline__ void split_weights(float a, float b, uint32_t &hi, uint32_t &lo) {
    hi = CACHE8 ? pack2<TYPE>(a, b) : pack2_down<TYPE>(a, b);
    const float2 x = widen2<TYPE>(hi);
    if (CACHE8)
        lo = pack2<TYPE>(a - x.x, b - x.y);
    else if (TYPE == AR_BF16)
        lo = pack2<TYPE>(fmaf(a, 1.0f + 0x1p-23f, -x.x), fmaf(b, 1.0f + 0x1p-23f, -x.y));
    else
        lo = pack2<TYPE>(fmaxf(a - x.x, 0x1p-24f), fmaxf(b - x.y, 0x1p-24f));
}
// Both parts of two weights in binary16: 0 for weights of 0, else 2^-24 at least.
__device__ __forceinline__ void positive_parts(float a, float b, uint32_t &hi, uint32_t &lo) {
    const uint32_t none = (a == 0.0f ? 0xFFFFu : 0u) | (b == 0.0f ? 0xFFFF0000u : 0u);
    hi |= ((hi & 0xFFFFu) == 0u ? 1u : 0u) | ((hi & 0xFFFF0000u) == 0u ? 0x10000u : 0u);
    const float2 x = widen2<AR_FP16>(hi);
    lo = pack2<AR_FP16>(fmaxf(a - x.x, 0x1p-24f), fmaxf(b - x.y, 0x1p-24f));
    hi &= ~none;
    lo &= ~none;
}
// Two binary16 numbers, those that are not finite as 0.
__device__ __forceinline__ uint32_t finite2(uint32_t w) {
    const uint32_t keep = ((w & 0x7C00u) == 0x7C00u ? 0u : 0xFFFFu) |
                          ((w & 0x7C000000u) == 0x7C000000u ? 0u : 0xFFFF0000u);
    return w & keep;
}

template <int DT, bool CACHE8, int DC, int HG> struct MmaForm {
    static constexpr int kType = CACHE8 ? (int)AR_FP16 : DT;      // of the products
    // the maximum's weight is 2^kBits; weights below kSmall have a third part
    static constexpr float kBits = CACHE8 ? 10.0f : DT == AR_FP16 ? 11.0f : 0.0f;
    // (over binary16 the second number is 2^-24 off, not 2^-25)
    static constexpr float kSmall = !CACHE8         ? 0x1p-10f
                                    : DT == AR_FP32 ? 0x1p-9f
                                    : DT == AR_FP16 ? 0x1p-11f
                                                    : 0x1p-13f;
    static constexpr uint32_t kCell = CACHE8 ? 1 : 2;
    static constexpr uint32_t kHeads = 8 * HG;                     // of a unit
    static constexpr int kThreads = 32 * kTeams * HG;
    static constexpr uint32_t kRow = DC * kCell;                   // bytes of a row in shared memory
    static constexpr uint32_t kChunks = kRow / 16;
    static constexpr uint32_t kRowsPer = 32 / kChunks;             // rows that a warp copies at once
    // a warp's stage: 16 keys, 16 values, their scales, which positions are there
    static constexpr uint32_t kScales = 32 * kRow, kMask = kScales + (CACHE8 ? 128 : 0);
    static constexpr uint32_t kStage = kMask + 16;
    static constexpr int kStages = HG == 4 && DC < 256 ? 5 : 3;
    static constexpr uint32_t kRing = kTeams * kStages * kStage;
    static constexpr int kQParts = DT == AR_FP32 ? 2 : 1;
    static constexpr uint32_t kQPart = kHeads * DC * 2, kQ = kQParts * kQPart;
    // columns of the output that the warps join at a time
    static constexpr int kJoin = DC == 256 || (CACHE8 && DC == 128) ? 16 : 32;
    static constexpr uint32_t kJoinRow = kJoin + 2;
    static constexpr uint32_t kSmem = kRing + kQ + 4 * kTeams * kHeads * kJoinRow;
    // CTAs of an SM: what registers and shared memory hold (and, for 32 heads, parts in
    // the workspace)
    static constexpr int kCtas = HG == 4     ? 1
                                 : DC == 256 ? (CACHE8 && HG == 1 ? 2 : 1)
                                 : DC == 128 ? (!CACHE8 ? 2 : HG == 1 ? (kQParts == 1 ? 4 : 3) : 2)
                                             : (CACHE8 && HG == 1 ? 4 : HG == 1 ? 3 : 2);

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

// The CTAs of a cluster have a share of one unit's positions each: (m, l) of its heads and
// o, rows of D, in their shared memory.  CTA `rank` adds its share of the columns over all
// of them, in their order.  all_m, all_l: shared memory for what the others have.
constexpr uint32_t kMaxParts = 8;
template <int DT, int THREADS>
__device__ __forceinline__ void join_cluster(const AttnArgs &a, uint32_t b, const UnitRows &u,
                                             uint32_t parts, uint32_t rank, const float *o,
                                             const float *m, const float *l, uint32_t heads,
                                             float (*all_m)[32], float (*all_l)[32]) {
    cluster_sync();
    for (uint32_t i = threadIdx.x; i < parts * heads; i += THREADS) {
        all_m[i / heads][i % heads] = ld_peer_f32(m + i % heads, i / heads);
        all_l[i / heads][i % heads] = ld_peer_f32(l + i % heads, i / heads);
    }
    __syncthreads();
    auto total = [&](uint32_t row, float *by, float &sum) {   // factors of the parts
        float top = -INFINITY;
        for (uint32_t p = 0; p < parts; ++p)
            top = fmaxf(top, all_m[p][row]);
        sum = 0.0f;
#pragma unroll
        for (uint32_t p = 0; p < kMaxParts; ++p) {
            by[p] = p < parts ? exp2_approx(all_m[p][row] - finite_max(top)) : 0.0f;
            sum += p < parts ? all_l[p][row] * by[p] : 0.0f;
        }
        return top;
    };
    float by[kMaxParts], sum;
    for (uint32_t i = rank * THREADS + threadIdx.x; i < u.rows * a.g.D; i += parts * THREADS) {
        float v[kMaxParts], x = 0.0f;
#pragma unroll
        for (uint32_t p = 0; p < kMaxParts; ++p)
            v[p] = p < parts ? ld_peer_f32(o + i, p) : 0.0f;
        total(i / a.g.D, by, sum);
#pragma unroll
        for (uint32_t p = 0; p < kMaxParts; ++p)
            x += p < parts ? v[p] * by[p] : 0.0f;
        store_row<DT>(a.out + (uint64_t)b * a.sout, u.head * a.g.D + i, output_of(x, sum));
    }
    if (a.lse && rank == 0 && threadIdx.x < u.rows) {
        const float top = total(threadIdx.x, by, sum);
        a.lse[(uint64_t)b * a.heads + u.head + threadIdx.x] = lse_of(top, sum);
    }
    cluster_sync();                   // the others may still read this CTA's
}

// UNITS: a.cluster CTAs have one unit between them, and each nothing else; otherwise a CTA
// has a run of tiles.
template <int DT, bool CACHE8, int DC, int HG, bool UNITS>
__global__ void __launch_bounds__(MmaForm<DT, CACHE8, DC, HG>::kThreads, MmaForm<DT, CACHE8, DC, HG>::kCtas)
k_attention_mma(const __grid_constant__ AttnArgs a) {
    using M = MmaForm<DT, CACHE8, DC, HG>;
    constexpr uint32_t H = M::kHeads;
    constexpr bool kKeepQ = DC <= 128 && M::kQParts == 1;   // q's operands stay in registers
    constexpr bool kApart = CACHE8 && DT == AR_FP32;        // scores have a maximum of their own
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t scan[33];
    __shared__ float group_m[kTeams][H], group_l[kTeams][H], head_scale[H];
    __shared__ float whole_m[H], whole_l[H];               // of this CTA, for its cluster
    uint8_t *qs = smem + M::kRing;
    float *join = reinterpret_cast<float *>(qs + M::kQ);
    const uint32_t D = a.g.D, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t group = warp / HG, part8 = warp % HG;   // positions; heads
    uint8_t *ring = smem + group * (M::kStages * M::kStage);
    const uint32_t ring_addr = shared_addr(ring), q_addr = shared_addr(qs);
    kernel_prologue();
    const uint32_t parts = UNITS ? a.cluster : 0u, rank = parts > 1 ? cluster_rank() : 0u;
    uint64_t per = 1;
    Cursor<kMmaTile> c = {};
    if constexpr (!UNITS) {
        if (tid == 0)
            WorkSpace(a.work).meta[blockIdx.x] = make_int4(0, 0, -1, 0);
        empty_rows<DT, kMmaTile>(a);
        c = find_run<kMmaTile>(a, scan, &per);
    } else {
        c.share(a, blockIdx.x / parts, rank, parts);
    }

    // ---- q of a unit, two elements a word, a warp to a row: loaded a unit ahead
    constexpr int kWarps = kTeams * HG, kQRows = H / kWarps, kQWords = DC / 64;
    constexpr uint32_t kQSize = Elem<DT>::kSize;
    const bool q_words = ((uintptr_t)a.q | a.sq) % 4 == 0;
    uint32_t qw[kQRows][kQWords][kQSize / 2];
    auto load_q_rows = [&] {
        if (!UNITS && c.done())
            return;
        const UnitRows u = unit_rows(a, c.unit);
        const uint8_t *q = a.q + (uint64_t)c.b * a.sq + (uint64_t)u.head * D * kQSize;
#pragma unroll
        for (int k = 0; k < kQRows; ++k)
#pragma unroll
            for (int i = 0; i < kQWords; ++i) {
                const uint32_t r = warp + k * kWarps, d = 2 * lane + 64 * i;
#pragma unroll
                for (uint32_t w = 0; w < kQSize / 2; ++w) {
                    qw[k][i][w] = 0u;
                    if (r < u.rows && d < D) {
                        const uint8_t *x = q + (uint64_t)(r * D + d) * kQSize + 4 * w;
                        if (kQSize == 4 || q_words)
                            qw[k][i][w] = *reinterpret_cast<const uint32_t *>(x);
                        else
                            qw[k][i][w] = ld_elem<AR_BF16>(x, 0) | ld_elem<AR_BF16>(x, 1) << 16;
                    }
                }
            }
    };
    load_q_rows();

    // ---- the copies, some tiles ahead.  Where 16 positions lie in one page (a.runs) the
    // warp looks up one page, otherwise a lane one for each of its rows.
    Cursor<kMmaTile> f = c;
    // The group's warps copy kCopies sets of kRowsPer rows each.
    constexpr uint32_t kSets = 16 / M::kRowsPer, kCopies = (kSets + HG - 1) / HG;
    const uint32_t copy_row = part8 * kCopies * M::kRowsPer + lane / M::kChunks;
    const uint32_t copy_chunk = lane % M::kChunks;
    const uint32_t row_bytes = D * M::kCell;
    const uint32_t copy_from = copy_row * row_bytes + copy_chunk * 16;
    const bool column = copy_chunk * 16 < row_bytes;
    uint32_t slot = 0;
    int32_t page = -1;
    auto look_up = [&] {                                   // of the next tile to fetch
        if (f.done())
            return;
        const uint32_t j = f.span.origin + f.t * kMmaTile + group * 16 + (a.runs ? 0 : lane & 15);
        page = -1;
        if (j < f.span.n) {
            page = a.g.page_of(f.b, j);
            slot = a.g.slot_of(j);
        }
    };
    auto fetch = [&](uint32_t stage) {
        if (!f.done()) {
            const uint32_t kv = f.unit / a.head_tiles;
            const uint32_t to = ring_addr + stage * M::kStage;
            const uint32_t j0 = f.span.origin + f.t * kMmaTile + group * 16;
            // positions [lo, n) of the 16
            const uint32_t from = f.span.lo > j0 ? f.span.lo - j0 : 0u;
            const uint32_t left = f.span.n > j0 ? f.span.n - j0 : 0u;
            uint32_t mask = ((left < 16 ? 1u << left : 0x10000u) - 1u) & (0xFFFFu << from);
            const uint64_t at = page >= 0 ? (uint64_t)page * a.g.stride +
                                                (uint64_t)a.g.in_page(kv, slot) * M::kCell
                                          : 0;
            if (a.runs) {
                mask = page >= 0 ? mask : 0u;
                const uint8_t *k = a.g.k + at + copy_from, *v = a.g.v + at + copy_from;
                if (mask == 0xFFFFu && row_bytes == M::kRow) {
#pragma unroll
                    for (uint32_t i = 0; i < kCopies; ++i) {
                        if (kCopies * HG > kSets && part8 * kCopies + i >= kSets)
                            break;
                        const uint32_t r = i * M::kRowsPer + copy_row;
                        const uint32_t x = i * M::kRowsPer * M::kRow;
                        fetch16(to + M::chunk(r, copy_chunk), k + x);
                        fetch16(to + 16 * M::kRow + M::chunk(r, copy_chunk), v + x);
                    }
                } else {
#pragma unroll
                    for (uint32_t i = 0; i < kCopies; ++i) {
                        if (kCopies * HG > kSets && part8 * kCopies + i >= kSets)
                            break;
                        const uint32_t r = i * M::kRowsPer + copy_row;
                        const bool on = column && (mask >> r & 1u);
                        const uint32_t x = on ? i * M::kRowsPer * row_bytes : 0u;
                        fetch16(to + M::chunk(r, copy_chunk), on ? k + x : a.g.k, on ? 16 : 0);
                        fetch16(to + 16 * M::kRow + M::chunk(r, copy_chunk), on ? v + x : a.g.v,
                                on ? 16 : 0);
                    }
                }
            } else {
                mask &= __ballot_sync(0xFFFFFFFFu, page >= 0) & 0xFFFFu;
#pragma unroll
                for (uint32_t i = 0; i < kCopies; ++i) {
                    if (kCopies * HG > kSets && part8 * kCopies + i >= kSets)
                        break;
                    const uint32_t r = i * M::kRowsPer + copy_row;
                    const uint64_t row = __shfl_sync(0xFFFFFFFFu, at, r);
                    const bool on = column && (mask >> r & 1u);
                    const uint64_t x = on ? row + copy_chunk * 16 : 0;
                    fetch16(to + M::chunk(r, copy_chunk), a.g.k + x, on ? 16 : 0);
                    fetch16(to + 16 * M::kRow + M::chunk(r, copy_chunk), a.g.v + x, on ? 16 : 0);
                }
            }
            if (CACHE8 && part8 == 0) {
                const float *scales = lane < 16 ? a.g.ks : a.g.vs;
                const bool on = mask >> (lane & 15) & 1u;
                const uint64_t x =
                    on ? a.g.scale_at(page, kv, slot) + (a.runs ? lane & 15 : 0u) : 0;
                fetch4(to + M::kScales + lane * 4, scales + x, on ? 4 : 0);
            }
            if (lane == 0 && part8 == 0)
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
    const uint32_t k_row = lane % 16, k_chunk = lane / 16;
    const uint32_t v_row = CACHE8 ? lane % 16 : lane % 8 + lane / 16 * 8;
    const uint32_t v_chunk = CACHE8 ? lane / 16 : lane / 8 & 1;
    const uint32_t q_row = part8 * 8 + lane % 8, q_part = lane / 8;
    // q's operands of steps k, k + 1 of 16 columns: two words for each
    auto load_q = [&](uint32_t (*q)[2], int k, uint32_t part) {
        uint32_t w[4];
        ldmatrix4(w, q_addr + part * M::kQPart + M::q_chunk(q_row, 2 * k + q_part));
        q[0][0] = w[0];
        q[0][1] = w[1];
        q[1][0] = w[2];
        q[1][1] = w[3];
    };
    auto group_sync = [&] {
        if (HG == 1)
            __syncwarp();
        else
            asm volatile("bar.sync %0, %1;" :: "r"(1 + group), "n"(32 * HG) : "memory");
    };

    // (a CTA of a cluster has its share of a unit to end even if it holds no tile)
    for (bool first_turn = true; !c.done() || (UNITS && first_turn); first_turn = false) {
        // q to shared memory: binary16 after scaling by a power of two where the cache is E4M3
#pragma unroll
        for (int k = 0; k < kQRows; ++k) {
            const uint32_t r = warp + k * kWarps;
            float up = 1.0f, back = 1.0f;
            auto pair = [&](int i) {
                if constexpr (kQSize == 4)
                    return make_float2(__uint_as_float(qw[k][i][0]), __uint_as_float(qw[k][i][1]));
                else
                    return widen2<DT>(qw[k][i][0]);
            };
            if (CACHE8) {
                float top = 0.0f;
#pragma unroll
                for (int i = 0; i < kQWords; ++i) {
                    const float2 x = pair(i);
                    top = fmaxf(top, fmaxf(fabsf(x.x), fabsf(x.y)));
                }
#pragma unroll
                for (int d = 16; d > 0; d >>= 1)
                    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
                half_range(top, up, back);
            }
#pragma unroll
            for (int i = 0; i < kQWords; ++i) {
                const uint32_t e = M::q_column(2 * lane + 64 * i);
                uint8_t *at = qs + M::q_chunk(r, e / 8) + e % 8 * 2;
                uint32_t w = qw[k][i][0];
                if (CACHE8) {
                    const float2 x = pair(i);
                    w = half2_of(x.x * up, x.y * up);
                    if (M::kQParts == 2)
                        *reinterpret_cast<uint32_t *>(at + M::kQPart) =
                            rest_of(w, x.x * up, x.y * up);
                }
                *reinterpret_cast<uint32_t *>(at) = w;
            }
            if (lane == 0)
                head_scale[r] = a.scale2 * back;
        }
        __syncthreads();
        uint32_t qf[kKeepQ ? DC / 16 : 2][2];
        if (kKeepQ)
#pragma unroll
            for (int k = 0; k < DC / 16; k += 2)
                load_q(qf + (kKeepQ ? k : 0), k, 0);
        // of a lane's columns: heads first + {0, 1}
        const uint32_t first = part8 * 8 + lane % 4 * 2;
        // m, and what a score is compared with and taken relative to
        float scale[2], m[2], bound[2], base[2], l[2], o[DC / 16][4];
        float score_m[2], score_bound[2], score_base[2];       // kApart: those of l
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            scale[i] = head_scale[first + i];
            m[i] = bound[i] = -INFINITY;
            base[i] = l[i] = score_base[i] = 0.0f;
            score_m[i] = score_bound[i] = -INFINITY;
        }
#pragma unroll
        for (int d = 0; d < DC / 16; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[d][i] = 0.0f;

        for (uint32_t t = c.t; t < c.t1; ++t) {
            fetch_wait<M::kStages - 2>();
            group_sync();
            // the group has this stage's copies, and is done with the stage before it
            fetch((stage + M::kStages - 1) % M::kStages);
            const uint32_t at = ring_addr + stage * M::kStage;
            const uint8_t *here = ring + stage * M::kStage;
            const uint32_t mask = *reinterpret_cast<const uint32_t *>(here + M::kMask);
            // scores: positions lane / 4 (0, 1) and that + 8 (2, 3), in two sums
            float s[4] = {}, s2[4] = {};
#pragma unroll
            for (int k = 0; k < DC / 16; k += 2) {
                if (k * 16 >= (int)D)
                    break;
                uint32_t ka[2][4];
                if (CACHE8) {
                    uint32_t w[4];
                    ldmatrix4(w, at + M::chunk(k_row, k + k_chunk));
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        from_e4m3x4(w[2 * i], ka[i][0], ka[i][2]);
                        from_e4m3x4(w[2 * i + 1], ka[i][1], ka[i][3]);
                    }
                } else {
                    ldmatrix4(ka[0], at + M::chunk(k_row, 2 * k + k_chunk));
                    ldmatrix4(ka[1], at + M::chunk(k_row, 2 * k + 2 + k_chunk));
                }
#pragma unroll
                for (int part = 0; part < M::kQParts; ++part) {
                    if (!kKeepQ)
                        load_q(qf, k, part);
                    const uint32_t(*q)[2] = qf + (kKeepQ ? k : 0);
                    mma16<M::kType>(s, ka[0], q[0][0], q[0][1]);
                    mma16<M::kType>(s2, ka[1], q[1][0], q[1][1]);
                }
            }
            // scales of the two positions; what they add to the maximum's exponent
            float ks[2], vs[2], lead[2];
            if (CACHE8) {
                const float *scales = reinterpret_cast<const float *>(here + M::kScales) + lane / 4;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    ks[j] = scales[8 * j];
                    vs[j] = scales[16 + 8 * j];
                    if (kApart)
                        split_scale(vs[j], lead[j], vs[j]);
                    else
                        lead[j] = fmaxf((float)((int)(__float_as_uint(vs[j]) >> 23) - 127),
                                        kLeastScale);
                }
            }
            bool above = false;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[i] = (s[i] + s2[i]) * (CACHE8 ? scale[i & 1] * ks[i / 2] : scale[i & 1]);
                if (mask != 0xFFFFu && !(mask >> (lane / 4 + i / 2 * 8) & 1u))
                    s[i] = -INFINITY;
                s2[i] = CACHE8 ? s[i] + lead[i / 2] : s[i];
                above |= s2[i] > bound[i & 1];
                if (kApart)
                    above |= s[i] > score_bound[i & 1];
            }
            if (__any_sync(0xFFFFFFFFu, above)) {
                float al[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float now = fmaxf(m[i], fmaxf(s2[i], s2[2 + i]));
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1)
                        now = fmaxf(now, __shfl_xor_sync(0xFFFFFFFFu, now, d));
                    al[i] = exp2_approx(m[i] - finite_max(now));
                    m[i] = now;
                    bound[i] = now + kSlack;
                    base[i] = finite_max(now) - M::kBits;
                    if (kApart) {
                        float top = fmaxf(score_m[i], fmaxf(s[i], s[2 + i]));
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1)
                            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
                        l[i] *= exp2_approx(score_m[i] - finite_max(top));
                        score_m[i] = top;
                        score_bound[i] = top + kSlack;
                        score_base[i] = finite_max(top);
                    } else {
                        l[i] *= al[i];
                    }
                }
#pragma unroll
                for (int d = 0; d < DC / 16; ++d) {
                    mul2(o[d], al[0], al[1]);
                    mul2(o[d] + 2, al[0], al[1]);
                }
            }
            // weights, in two parts: one would keep 8 (bf16) or 11 bits of them.  Transposed,
            // they are the second operand.
            const uint32_t v_at = at + 16 * M::kRow;
            float p[4];
            uint32_t hi[2], lo[2];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (kApart) {
                    l[i & 1] += exp2_approx(s[i] - score_base[i & 1]);
                    p[i] = exp2_approx(s2[i] - base[i & 1]) * vs[i / 2];
                    continue;
                }
                p[i] = exp2_approx(s[i] - base[i & 1]);
                l[i & 1] += p[i];
                if (CACHE8)
                    p[i] *= vs[i / 2];
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                uint32_t a, b;
                split_weights<M::kType, CACHE8>(p[2 * j], p[2 * j + 1], a, b);
                hi[j] = transpose8(a);
                lo[j] = transpose8(b);
            }
            // columns 16 d .. 16 d + 31 of the values, the first operand of two products
            auto load_v = [&](uint32_t (*va)[4], int d) {
                if (CACHE8) {
                    // a word holds two columns of two positions: to two positions of each; the
                    // rows of a product are the even columns, then the odd ones
                    uint32_t w[4];
                    ldmatrix4_trans(w, v_at + M::chunk(v_row, d + v_chunk));
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        from_e4m3x4(__byte_perm(w[2 * i], 0, 0x3120), va[i][0], va[i][1]);
                        from_e4m3x4(__byte_perm(w[2 * i + 1], 0, 0x3120), va[i][2], va[i][3]);
                    }
                } else {
                    ldmatrix4_trans(va[0], v_at + M::chunk(v_row, 2 * d + v_chunk));
                    ldmatrix4_trans(va[1], v_at + M::chunk(v_row, 2 * d + 2 + v_chunk));
                }
            };
            if constexpr (M::kType == AR_FP16) {
                const float least = fminf(fminf(p[0], p[1]), fminf(p[2], p[3]));
                if (__any_sync(0xFFFFFFFFu, least < M::kSmall)) {
                    // (two parts of it over binary16: it takes back what positive_parts added)
                    uint32_t rest[2], last[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        uint32_t a, b;
                        split_weights<M::kType, CACHE8>(p[2 * j], p[2 * j + 1], a, b);
                        if (!CACHE8) {
                            positive_parts(p[2 * j], p[2 * j + 1], a, b);
                            hi[j] = transpose8(a);
                            lo[j] = transpose8(b);
                        }
                        const float2 x = widen2<AR_FP16>(a), y = widen2<AR_FP16>(b);
                        float r[2] = {p[2 * j] - x.x - y.x, p[2 * j + 1] - x.y - y.y};
                        r[0] = p[2 * j] < 1.0f ? r[0] * kRestScale : 0.0f;
                        r[1] = p[2 * j + 1] < 1.0f ? r[1] * kRestScale : 0.0f;
                        const uint32_t w = pack2<AR_FP16>(r[0], r[1]);
                        rest[j] = transpose8(w);
                        if (!CACHE8)
                            last[j] = transpose8(rest_of(w, r[0], r[1]));
                    }
#pragma unroll
                    for (int d = 0; d < DC / 16; d += 2) {
                        if (d * 16 >= (int)D)
                            break;
                        uint32_t va[2][4];
                        load_v(va, d);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            float sum[4] = {};
                            if (!CACHE8)       // the first parts' products have them
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    va[i][k] = finite2(va[i][k]);
                            mma16<AR_FP16>(sum, va[i], rest[0], rest[1]);
                            if (!CACHE8)
                                mma16<AR_FP16>(sum, va[i], last[0], last[1]);
                            fma2(o[d + i], sum[0], sum[1], 1 / kRestScale, 1 / kRestScale);
                            fma2(o[d + i] + 2, sum[2], sum[3], 1 / kRestScale, 1 / kRestScale);
                        }
                    }
                }
            }
#pragma unroll
            for (int d = 0; d < DC / 16; d += 2) {
                if (d * 16 >= (int)D)
                    break;
                uint32_t va[2][4];
                load_v(va, d);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    mma16<M::kType>(o[d + i], va[i], hi[0], hi[1]);
                    mma16<M::kType>(o[d + i], va[i], lo[0], lo[1]);
                }
            }
            stage = (stage + 1) % M::kStages;
        }
        const Cursor<kMmaTile> done = c;
        c.next_unit(a);
        if (!UNITS)
            load_q_rows();

        // the teams' parts, in their order; what they are relative to
        float half_way[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int d = 4; d < 32; d <<= 1)
                l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], d);
            if (M::kBits != 0.0f)
                m[i] = m[i] == -INFINITY ? m[i] : m[i] - M::kBits;
            if (kApart) {
                // o relative to the scores' maximum, as l: by halves, since the factor itself
                // may have lost bits below 2^-126
                half_way[i] = m[i] == -INFINITY ? 0.0f : exp2f(0.5f * (m[i] - score_m[i]));
                m[i] = score_m[i];
            }
            if (lane < 4) {
                group_m[group][first + i] = m[i];
                group_l[group][first + i] = l[i];
            }
        }
        __syncthreads();
        const UnitRows u = unit_rows(a, done.unit);
        const int part = UNITS ? -1 : segment_part(a, done, per);
        float own[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float all = -INFINITY;
#pragma unroll
            for (int w = 0; w < kTeams; ++w)
                all = fmaxf(all, group_m[w][first + i]);
            own[i] = exp2_approx(m[i] - finite_max(all));
        }
        // the head that this thread finishes, with kLanes - 1 others
        constexpr uint32_t kLanes = M::kThreads / H;
        const uint32_t row = tid / kLanes;
        float row_m = -INFINITY, row_l = 0.0f;
#pragma unroll
        for (int w = 0; w < kTeams; ++w)
            row_m = fmaxf(row_m, group_m[w][row]);
#pragma unroll
        for (int w = 0; w < kTeams; ++w)
            row_l += group_l[w][row] * exp2_approx(group_m[w][row] - finite_max(row_m));
#pragma unroll
        for (int d0 = 0; d0 < DC; d0 += M::kJoin) {
            if (d0 >= (int)D)
                break;
            if (d0 > 0)
                __syncthreads();
            float *mine = join + group * H * M::kJoinRow;
#pragma unroll
            for (int d = 0; d < M::kJoin / 16; ++d)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t column = 16 * d + (CACHE8 ? lane / 4 * 2 + i / 2
                                                             : lane / 4 + i / 2 * 8);
                    float x = o[d0 / 16 + d][i];
                    if (kApart)
                        x = x * half_way[i & 1] * half_way[i & 1];
                    mine[(first + (i & 1)) * M::kJoinRow + column] = x * own[i & 1];
                }
            __syncthreads();
#pragma unroll
            for (uint32_t i = 0; i < M::kJoin / kLanes; ++i) {
                const uint32_t column = tid % kLanes + kLanes * i, d = d0 + column;
                const uint32_t at = row * M::kJoinRow + column;
                float v = join[at];
#pragma unroll
                for (int w = 1; w < kTeams; ++w)
                    v += join[w * H * M::kJoinRow + at];
                if (row >= u.rows || d >= D)
                    continue;
                if (UNITS && parts > 1)   // the ring is done with: nothing is left to fetch
                    reinterpret_cast<float *>(smem)[row * D + d] = v;
                else if (part < 0)
                    store_row<DT>(a.out + (uint64_t)done.b * a.sout, (u.head + row) * D + d,
                                  output_of(v, row_l));
                else
                    WorkSpace(a.work).o[((uint64_t)part * H + row) * D + d] = v;
            }
        }
        if (UNITS && parts > 1) {
            if (tid % kLanes == 0) {
                whole_m[row] = row_m;
                whole_l[row] = row_l;
            }
            float(*all)[32] = reinterpret_cast<float(*)[32]>(smem + H * DC * 4);
            static_assert(M::kRing >= H * DC * 4 + 2 * kMaxParts * 128, "both fit in the ring");
            join_cluster<DT, M::kThreads>(a, done.b, u, parts, rank,
                                          reinterpret_cast<const float *>(smem), whole_m, whole_l,
                                          H, all, all + kMaxParts);
        } else if (tid % kLanes == 0 && row < u.rows) {
            if (part >= 0)
                WorkSpace(a.work).ml[(uint32_t)part * H + row] = make_float2(row_m, row_l);
            else if (a.lse)
                a.lse[(uint64_t)done.b * a.heads + u.head + row] = lse_of(row_m, row_l);
        }
    }
    fetch_wait<0>();
}

}  // namespace ar
