// A mixture-of-experts layer for a few tokens, in two launches:
//
//   h = g / (1 + exp(-g)) * u,  g, u = the two halves of up[e] x[t]
//   out[t] = sum_k w[t, k] down[e] h
//
// Bound by memory: the weights of every expert that a token chose are read once.
// They are the 16-row operand of warp-wide products (E4M3 is exact in binary16), the
// pairs (token, choice) of the expert the 8 or 16 columns: x is scaled by a power of two
// for each 128 of a row so that binary16 holds it, in two parts where one would round it;
// h has two parts always.  A block of 128 along k gets its scales in binary32 when it is
// summed.
//
// Weights come by TMA, a warp's own tiles of 16 rows by 128 bytes, through a ring of two
// stages per warp: a stage is free as soon as its codes are in the lanes' registers, and
// the ring runs on across the ends of units.  (By loads to registers, 16 rows at a time,
// an SM's requests in flight ran out: 2.5 TB/s with 16 bytes a lane, 3.5 with 32.)  Rows
// that are not on 16-byte boundaries are read by bytes.  A lane takes 32 bytes of a row,
// and the order of k inside a block is that of the lanes (see place_of), for the columns
// too.
//
// First launch (up): a CTA takes 16 rows of both halves of one expert at a time, its
// warps share the blocks along k.  The columns lie in shared memory, converted when the
// expert changes (on the way they cost three times the weights' conversion).  Second
// launch (down): a CTA takes rows of the output, its warps share the blocks along k of
// all experts; each keeps its own sums of all tokens, which are added in order.
//
// One token, 8 of 64 experts of 8192 x 2048: 85 us (4.7 TB/s); 16 tokens, 8192 x 1024, 293 to
// 304 by box (4.7 to 4.8; the first launch 172, the second 112).
//
// Every wait is bounded; after one that ran out the output is NaN, all of it (first launch) or
// the rows of a CTA (second), and the status word says so.
#include "ar_mma.cuh"
#include "ar_ring.cuh"
#include "ar_rows.cuh"
#include "ar_tensor_map.cuh"

namespace ar {

constexpr int kMoePairs = AR_MOE_LAYER_PAIRS;
// Dynamic shared memory of a CTA that has an SM to itself.
constexpr size_t kMoeSmem = 226 * 1024;
constexpr int kColumns = 16;          // most pairs of an expert in one pass over its weights

__device__ __forceinline__ uint32_t smem_at(const void *p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}

struct MoeArgs {
    const uint8_t *x;
    const void *ids;
    const float *w;
    const uint8_t *up, *down;
    const float *up_scale, *down_scale;
    uint8_t *out;
    uint8_t *h;                       // T * K rows of sh bytes, see HiddenRow
    uint64_t sx, sout, sh;            // bytes between rows
    uint64_t ldup, lddown;
    uint32_t T, K, H, F, E;
    uint32_t hb, fb, ub;              // blocks of 128 along H, F and 2F
    uint32_t columns;                 // pairs that the first launch's shared memory holds
    uint32_t stages;                  // of its rings
    uint32_t part_row;                // of its sums: floats between rows
    int wide_x;
    int ids8;
    int *status;                      // the workspace's last word
    uint8_t *failed;                  // of each CTA of the first launch: a wait ran out
    uint32_t ups;                     // those CTAs
};

// ---- who goes where ---------------------------------------------------------------

// The pairs that are here, and the experts they go to in the order of their first pair.
struct Chosen {
    int16_t expert[kMoePairs];        // of a pair, or -1
    int16_t active[kMoePairs];
    int16_t pairs[kMoePairs];         // of an active expert
    int first[AR_MOE_MAX_EXPERTS];
    int count;                        // of active
    int warp_count[kMoePairs / 32];
};

__device__ __forceinline__ int expert_of(const MoeArgs &a, uint32_t p) {
    const int64_t id = a.ids8 ? static_cast<const int64_t *>(a.ids)[p]
                              : (int64_t) static_cast<const int32_t *>(a.ids)[p];
    return id >= 0 && id < (int64_t)a.E ? (int)id : -1;
}

// The pairs of expert e in order, by one warp: `list` receives those from `skip` on,
// at most `most`; returns how many there are in all.
__device__ __forceinline__ int list_pairs(const MoeArgs &a, const Chosen &c, int e, int skip,
                                          int most, int16_t *list) {
    const uint32_t pairs = a.T * a.K, lane = threadIdx.x & 31;
    int n = 0;
    for (uint32_t p0 = 0; p0 < pairs; p0 += 32) {
        const uint32_t p = p0 + lane;
        const bool mine = p < pairs && c.expert[p] == e;
        const uint32_t m = __ballot_sync(0xFFFFFFFFu, mine);
        const int at = n + __popc(m & ((1u << lane) - 1u)) - skip;
        if (mine && at >= 0 && at < most)
            list[at] = (int16_t)p;
        n += __popc(m);
    }
    __syncwarp();
    return n;
}

__device__ __forceinline__ void choose(const MoeArgs &a, Chosen &c) {
    const uint32_t pairs = a.T * a.K, lane = threadIdx.x & 31;
    if (pairs <= 32) {                // one warp sees them all
        if (threadIdx.x < 32) {
            const int e = lane < pairs ? expert_of(a, lane) : -1;
            const uint32_t like = __match_any_sync(0xFFFFFFFFu, e);
            const bool lead = e >= 0 && (like & ((1u << lane) - 1u)) == 0;
            const uint32_t leads = __ballot_sync(0xFFFFFFFFu, lead);
            c.expert[lane] = (int16_t)e;
            if (lead) {
                const int at = __popc(leads & ((1u << lane) - 1u));
                c.active[at] = (int16_t)e;
                c.pairs[at] = (int16_t)__popc(like);
            }
            if (lane == 0)
                c.count = __popc(leads);
        }
        __syncthreads();
        return;
    }
    for (uint32_t e = threadIdx.x; e < a.E; e += blockDim.x)
        c.first[e] = kMoePairs;
    __syncthreads();
    for (uint32_t p = threadIdx.x; p < pairs; p += blockDim.x) {
        const int e = expert_of(a, p);
        c.expert[p] = (int16_t)e;
        if (e >= 0)
            atomicMin(&c.first[e], (int)p);
    }
    __syncthreads();
    // the first pair of an expert stands for it
    for (uint32_t p = threadIdx.x; p < kMoePairs; p += blockDim.x) {
        const bool lead = p < pairs && c.expert[p] >= 0 && c.first[c.expert[p]] == (int)p;
        const uint32_t m = __ballot_sync(0xFFFFFFFFu, lead);
        if (lane == 0)
            c.warp_count[p / 32] = __popc(m);
    }
    __syncthreads();
    for (uint32_t p = threadIdx.x; p < kMoePairs; p += blockDim.x) {
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
    for (int i = threadIdx.x >> 5; i < c.count; i += blockDim.x >> 5) {
        const int n = list_pairs(a, c, c.active[i], 0, 0, nullptr);
        if (lane == 0)
            c.pairs[i] = (int16_t)n;
    }
    __syncthreads();
}

// ---- a block of 128 along k ----------------------------------------------------------

// Lane l holds row or column l / 4 of an operand and, with c = l % 4, the elements
// 32 c .. 32 c + 31 of the block: eight steps of a product's 16 (4 elements a lane).
// In memory, converted columns have the 8-element pieces of the four lanes side by side.
__device__ __forceinline__ uint32_t place_of(uint32_t k) {
    return (k & ~127u) + (k / 8 & 3) * 32 + (k / 32 & 3) * 8 + k % 8;
}

struct Words8 {
    uint4 lo, hi;
    __device__ __forceinline__ uint32_t operator[](int i) const {
        const uint4 &v = i < 4 ? lo : hi;
        return i % 4 == 0 ? v.x : i % 4 == 1 ? v.y : i % 4 == 2 ? v.z : v.w;
    }
};

// 16 codes of a weight row from k on, byte by byte; zeros past K.
__device__ __forceinline__ uint4 load_codes(const uint8_t *row, uint32_t k, uint32_t K) {
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    for (uint32_t i = 0; i < 16 && k + i < K; ++i)
        w[i / 4] |= (uint32_t)row[k + i] << (8 * (i & 3));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The lane's codes of MT tiles of 16 rows: [tile][row l / 4 or that + 8].
template <int MT> struct Codes {
    Words8 q[MT][2];
};

// A warp's ring of 1, 2 or 4 stages of `BOXES` tiles of 16 rows by 128 bytes, in 1024-byte
// units whose 16-byte pieces are exchanged by row (the map's 128-byte swizzle).
constexpr uint64_t kMoeWaitNs = 2000000000ull;
constexpr uint32_t kBox = 16 * 128;
template <int BOXES> struct Ring {
    static constexpr uint32_t kStage = BOXES * kBox;
    uint32_t at, bars;                // this warp's stages and barriers
    const uint8_t *memory;
    volatile int *failed;             // of the CTA
    RingSteps steps;

    __device__ __forceinline__ void begin(uint8_t *stages, uint64_t *barriers, int *flag,
                                          uint32_t stages_log2) {
        at = (uint32_t)__cvta_generic_to_shared(stages);
        bars = (uint32_t)__cvta_generic_to_shared(barriers);
        memory = stages;
        failed = flag;
        steps = {stages_log2, 0u, 0u};
    }
    // Boxes at (k, rows[b]) of matrix e to the next stage; by one lane.
    __device__ __forceinline__ void issue(const CUtensorMap *map, uint32_t k,
                                          const uint32_t *rows, int e) {
        const uint32_t s = steps.stage(steps.sent++), bar = bars + 8 * s;
        mbar_expect(bar, kStage);
#pragma unroll
        for (int b = 0; b < BOXES; ++b)
            tma_3d(at + s * kStage + b * kBox, map, (int)k, (int)rows[b], e, bar);
    }
    // Until the oldest stage is there; after a failure at once.
    __device__ __forceinline__ void wait() {
        const uint32_t bar = bars + 8 * steps.stage(steps.used);
        const uint32_t phase = steps.parity(steps.used);
        if (!__all_sync(0xFFFFFFFFu, mbar_test(bar, phase)))
            wait_slow(bar, phase);
    }
    __device__ __noinline__ void wait_slow(uint32_t bar, uint32_t phase) {
        const uint64_t deadline = globaltimer_ns() + kMoeWaitNs;
        while (!*failed && !mbar_test(bar, phase))
            if (globaltimer_ns() > deadline)
                *failed = 1;
        __syncwarp();
    }
    // This lane's codes of row r of box b.
    __device__ __forceinline__ Words8 codes(int b, uint32_t r) const {
        const uint8_t *row = memory + steps.stage(steps.used) * kStage + b * kBox + r * 128;
        const uint32_t c = (threadIdx.x & 3) * 2;
        Words8 w;
        w.lo = *reinterpret_cast<const uint4 *>(row + ((c ^ (r & 7)) << 4));
        w.hi = *reinterpret_cast<const uint4 *>(row + (((c + 1) ^ (r & 7)) << 4));
        return w;
    }
    // After a failure, by the lane that sends: until what is in flight has landed, so that
    // nothing comes to the CTA's memory once it has left.
    __device__ __forceinline__ void drain() const {
        for (uint32_t step = steps.oldest_open(); step != steps.sent; ++step) {
            const uint64_t deadline = globaltimer_ns() + kMoeWaitNs;
            while (!mbar_test(bars + 8 * steps.stage(step), steps.parity(step)) &&
                   globaltimer_ns() < deadline) {
            }
        }
    }
};

__device__ __forceinline__ uint32_t word_of(const uint4 &v, int i) {
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// part += codes * columns, which have PARTS parts.  column(nt, p, piece): eight of the lane's
// elements of part p of column l / 4 of tile nt, two steps' worth.
template <int MT, int NT, int PARTS, typename Column>
__device__ __forceinline__ void block_product(float (*part)[NT][4], const Codes<MT> &w,
                                              Column column) {
#pragma unroll
    for (int piece = 0; piece < 4; ++piece) {
        uint4 b[NT][PARTS];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int p = 0; p < PARTS; ++p)
                b[n][p] = column(n, p, piece);
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                uint32_t r[4];
                from_e4m3x4(w.q[m][0][2 * piece + k], r[0], r[2]);
                from_e4m3x4(w.q[m][1][2 * piece + k], r[1], r[3]);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int p = 0; p < PARTS; ++p)
                        mma16<AR_FP16>(part[m][n], r, word_of(b[n][p], 2 * k),
                                       word_of(b[n][p], 2 * k + 1));
            }
    }
}

// The lane's 32 binary32 values of a column to binary16: scaled by a power of two for the
// block, in one part or two.  Returns the inverse of the scale.
template <bool LO>
__device__ __forceinline__ float convert_column(const float *v, uint4 *hi, uint4 *lo) {
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i)
        top = fmaxf(top, fabsf(v[i]));
    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    float s, inverse;
    half_range(top, s, inverse);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float *x = v + 8 * j + 2 * i;
            a[i] = half2_of(x[0] * s, x[1] * s);
            b[i] = LO ? rest_of(a[i], x[0] * s, x[1] * s) : 0u;
        }
        hi[j] = make_uint4(a[0], a[1], a[2], a[3]);
        if (LO)
            lo[j] = make_uint4(b[0], b[1], b[2], b[3]);
    }
    return inverse;
}

// The lane's 32 elements of a row of type DT, as they lie in memory; zeros past K.
template <int DT> struct RawColumn {
    static constexpr int kSize = Elem<DT>::kSize, E = 16 / kSize;     // elements of a vector
    uint4 v[2 * kSize];
    __device__ __forceinline__ void load(const uint8_t *row, uint32_t kb, uint32_t K, bool wide,
                                         bool on) {
        const uint32_t k = kb * 128 + (threadIdx.x & 3) * 32;
#pragma unroll
        for (int i = 0; i < 2 * kSize; ++i) {
            v[i] = make_uint4(0u, 0u, 0u, 0u);
            if (on && wide && k + i * E + E <= K) {
                v[i] = ld_v4_l1(row + (uint64_t)(k + i * E) * kSize);
            } else if (on) {
                uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (k + i * E + e < K)
                        w[e * kSize / 4] |= ld_elem<DT>(row, k + i * E + e) << (8 * (e * kSize % 4));
                v[i] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    }
    // to binary16 in one part or two; returns the inverse of their scale
    template <bool LO> __device__ __forceinline__ float convert(uint4 *hi, uint4 *lo) const {
        float f[32];
#pragma unroll
        for (int i = 0; i < 2 * kSize; ++i)
            Rows<DT, true>::widen(v[i], f + i * E);
        return convert_column<LO>(f, hi, lo);
    }
};

// ---- h between the launches ----------------------------------------------------------

// Where the output is binary32, so is h.  Otherwise h is held as two binary16 numbers (21
// bits; one alone, 11 bits, took 81 and 282 us for one token and sixteen, not 85 and 293, but
// was a second rounding that showed: fp16 outputs were 1.5 times as far from exact, of four
// small experts) that 16 neighbours, a tile, have scaled by one power of two.  Its exponent goes in
// steps of 16, so that the tiles of a block nearly always have the same one and enter a
// product as they lie in memory: step j stands for 2^(120 - 16 j), which brings the tile's
// largest magnitude between 2^-1 and 2^15.  The four bits of j are the lowest ones of the
// second numbers of the tile's first four elements.  A block has 64 bytes for eight elements
// of each of its four lanes: first numbers, then second numbers; the last block has as many
// lanes as it has elements for.
template <int DT> struct HiddenRow {
    static constexpr bool kParts = DT != AR_FP32;
    static __host__ __device__ __forceinline__ uint64_t bytes(uint32_t F) {
        // rows are read by 16-byte vectors
        return kParts ? (uint64_t)(F + 31) / 32 * 128 : (uint64_t)(F + 3) / 4 * 16;
    }
    // bytes of eight elements of the lanes of the block that element f is in
    static __device__ __forceinline__ uint32_t piece(uint32_t f, uint32_t F) {
        const uint32_t left = (F - f / 128 * 128 + 31) / 32;
        return (left < 4 ? left : 4) * 16;
    }
};
// The step of a tile whose largest magnitude is `top`; 0 for one of zeros.
__device__ __forceinline__ uint32_t tile_step(float top) {
    const uint32_t e = __float_as_uint(top) >> 23;
    return e < 6u ? 0u : (e - 6u) / 16;
}
__device__ __forceinline__ float step_scale(uint32_t j) {
    return __uint_as_float((247u - 16u * j) << 23);
}
__device__ __forceinline__ float step_inverse(uint32_t j) {
    return __uint_as_float((7u + 16u * j) << 23);
}
// The bit of a step that element r < 4 of a tile carries, and the step from the tile's
// first two words.
__device__ __forceinline__ uint32_t step_bit(uint32_t j, uint32_t r) {
    return j >> ((r & 1) * 2 + r / 2) & 1u;
}
__device__ __forceinline__ uint32_t step_of(uint32_t w0, uint32_t w1) {
    const uint32_t x = (w0 & 0x10001u) | (w1 & 0x10001u) << 1;
    return (x | x >> 14) & 15u;
}
// v in binary16 with this lowest bit: the nearest such number, or next to it.
__device__ __forceinline__ uint32_t half_with_bit(float v, uint32_t bit) {
    const __half h = __float2half_rn(v);
    const uint32_t q = __half_as_ushort(h);
    if ((q & 1u) == bit)
        return q;
    const bool away = fabsf(v) >= fabsf(__half2float(h));     // and NaN stays one: q - 1
    return away ? q + 1 : q - 1;
}

// ---- first launch -------------------------------------------------------------

constexpr int kUpTiles = 2, kUpRows = 8 * kUpTiles;       // rows of each half
constexpr int kUpWarps = 16, kUpThreads = 32 * kUpWarps;
static_assert(kUpRows == 16, "a box of each half; and what shares an exponent of h");

struct UpShared {
    Chosen c;
    int16_t list[kUpWarps][kColumns];
    uint64_t bars[kUpWarps][2];
    int failed;
};
// Bytes of it with the sums of half of the warps.
static __host__ __device__ __forceinline__ uint32_t up_fixed(uint32_t part_row) {
    return (uint32_t)(sizeof(UpShared) + kUpWarps / 2 * 2 * kUpRows * part_row * 4 + 127) / 128 *
           128;
}
// A column in shared memory: blocks of 256 bytes, in one part or two, and an inverse
// scale each.  Columns start 64 bytes apart in the banks.
template <int DT> struct UpColumn {
    static constexpr int kParts = DT == AR_FP32 ? 2 : 1;
    static __host__ __device__ __forceinline__ uint32_t bytes(uint32_t hb) {
        return (kParts * hb * 256 + hb * 4 + 127) / 128 * 128 + 64;
    }
};

// The listed pairs' tokens to shared memory, a warp to a block.
template <int DT>
__device__ __forceinline__ void stage_columns(const MoeArgs &a, const int16_t *list, int n,
                                              uint8_t *xs) {
    using C = UpColumn<DT>;
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31, bytes = C::bytes(a.hb);
#pragma unroll 4
    for (uint32_t item = warp; item < n * a.hb; item += kUpWarps) {
        const uint32_t c = item / a.hb, kb = item - c * a.hb, k = kb * 128 + lane * 4;
        const uint8_t *row = a.x + (uint64_t)(list[c] / a.K) * a.sx;
        float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (a.wide_x && k + 4 <= a.H) {
            if (Elem<DT>::kSize == 4) {
                const float4 f = *reinterpret_cast<const float4 *>(row + (uint64_t)k * 4);
                v[0] = f.x;
                v[1] = f.y;
                v[2] = f.z;
                v[3] = f.w;
            } else {
                const uint2 u = *reinterpret_cast<const uint2 *>(row + (uint64_t)k * 2);
                const float2 f = widen2<DT == AR_FP32 ? AR_BF16 : DT>(u.x);
                const float2 g = widen2<DT == AR_FP32 ? AR_BF16 : DT>(u.y);
                v[0] = f.x;
                v[1] = f.y;
                v[2] = g.x;
                v[3] = g.y;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (k + i < a.H)
                    v[i] = widen1<DT>(ld_elem<DT>(row, k + i));
        }
        float top = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
        float s, inverse;
        half_range(top, s, inverse);
        uint8_t *column = xs + c * bytes;
        uint8_t *at = column + kb * 256 + place_of(lane * 4) * 2;
        const uint2 hi = make_uint2(half2_of(v[0] * s, v[1] * s), half2_of(v[2] * s, v[3] * s));
        *reinterpret_cast<uint2 *>(at) = hi;
        if (C::kParts == 2)
            *reinterpret_cast<uint2 *>(at + a.hb * 256) =
                make_uint2(rest_of(hi.x, v[0] * s, v[1] * s), rest_of(hi.y, v[2] * s, v[3] * s));
        if (lane == 0)
            reinterpret_cast<float *>(column + C::kParts * a.hb * 256)[kb] = inverse;
    }
}

// The weights that a warp of the first launch fetches, in the order in which it uses them:
// for each expert of the CTA's run, for each pass over its pairs, for each tile of rows,
// its blocks along k.
struct UpCursor {
    uint32_t i, tile, first, last, kb, pass;
    uint64_t left;                    // tiles of the run past this expert's
    bool done;

    __device__ __forceinline__ void begin(const MoeArgs &a, uint32_t tiles, uint64_t unit,
                                          uint64_t end) {
        const uint32_t warp = threadIdx.x >> 5;
        done = unit >= end || warp >= a.hb;
        i = (uint32_t)(unit / tiles);
        first = tile = (uint32_t)(unit - (uint64_t)i * tiles);
        last = end - unit < tiles - tile ? tile + (uint32_t)(end - unit) : tiles;
        left = end - unit - (last - tile);
        kb = warp;
        pass = 0;
    }
    __device__ __forceinline__ void next(const MoeArgs &a, const Chosen &c, uint32_t tiles) {
        kb += kUpWarps;
        if (kb < a.hb)
            return;
        kb = threadIdx.x >> 5;
        if (++tile < last)
            return;
        tile = first;
        if (++pass * a.columns < (uint32_t)c.pairs[i])
            return;
        pass = 0;
        ++i;
        first = tile = 0;
        last = left < tiles ? (uint32_t)left : tiles;
        left -= last;
        done = last == 0;
    }
};

// What a warp of the first launch works with.
struct UpWarp {
    Ring<2> ring;
    UpCursor cursor;
    const CUtensorMap *map;
    uint32_t tiles;

    // the next step's weights on their way, if there is one
    __device__ __forceinline__ void fetch(const MoeArgs &a, const Chosen &c) {
        if (cursor.done)
            return;
        if ((threadIdx.x & 31) == 0 && !*ring.failed) {
            const uint32_t rows[2] = {cursor.tile * kUpRows, a.F + cursor.tile * kUpRows};
            ring.issue(map, cursor.kb * 128, rows, c.active[cursor.i]);
        }
        cursor.next(a, c, tiles);
    }
};

// Rows f0.. of both halves of expert e times n listed pairs.  BULK: the weights come
// through the ring and the columns lie in shared memory at xs; otherwise both are read
// on the way.  parts: where half of the warps leave their sums.
template <int DT, bool BULK, int NT>
__device__ __forceinline__ void up_unit(const MoeArgs &a, UpShared &s, UpWarp &me, float *parts,
                                        const uint8_t *xs, int e, uint32_t f0, int n) {
    using C = UpColumn<DT>;
    constexpr bool kLo = C::kParts == 2;
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int16_t *list = s.list[warp];
    const uint8_t *w = a.up + (uint64_t)e * 2 * a.F * a.ldup;
    const float *ws = a.up_scale + (uint64_t)e * a.ub * a.hb;
    // rows past the last stand in for it: their sums go nowhere
    const uint8_t *rows[kUpTiles][2];
    uint32_t scales[kUpTiles][2];
#pragma unroll
    for (int m = 0; m < kUpTiles; ++m)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t f = f0 + m * 8 + lane / 4;
            const uint32_t r = (f < a.F ? f : a.F - 1) + i * a.F;
            rows[m][i] = w + (uint64_t)r * a.ldup;
            scales[m][i] = r / 128 * a.hb;
        }
    const uint32_t bytes = C::bytes(a.hb), first = lane % 4 * 2;
    const uint8_t *mine = xs + lane / 4 * bytes + lane % 4 * 16;
    const float *inverses = reinterpret_cast<const float *>(xs + first * bytes +
                                                            C::kParts * a.hb * 256);
    float sum[kUpTiles][NT][4] = {}, next_scale[kUpTiles][2];
    auto load_scales = [&](uint32_t kb) {
#pragma unroll
        for (int m = 0; m < kUpTiles; ++m)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                next_scale[m][i] = ws[scales[m][i] + kb];
    };
    if (warp < a.hb)
        load_scales(warp);
    for (uint32_t kb = warp; kb < a.hb; kb += kUpWarps) {
        float sc[kUpTiles][2];
#pragma unroll
        for (int m = 0; m < kUpTiles; ++m)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                sc[m][i] = next_scale[m][i];
        if (kb + kUpWarps < a.hb)
            load_scales(kb + kUpWarps);
        Codes<kUpTiles> now;
        if (BULK) {
            me.ring.wait();
#pragma unroll
            for (int m = 0; m < kUpTiles; ++m)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    now.q[m][i] = me.ring.codes(i, m * 8 + lane / 4);
            __syncwarp();
            ++me.ring.steps.used;
            me.fetch(a, s.c);
        } else {
            const uint32_t k = kb * 128 + lane % 4 * 32;
#pragma unroll
            for (int m = 0; m < kUpTiles; ++m)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    now.q[m][i].lo = load_codes(rows[m][i], k, a.H);
                    now.q[m][i].hi = load_codes(rows[m][i], k + 16, a.H);
                }
        }
        float part[kUpTiles][NT][4] = {}, inverse[NT][2];   // of this lane's columns
        if constexpr (BULK) {
            block_product<kUpTiles, NT, C::kParts>(part, now, [&](int nt, int p, int piece) {
                return nt * 8 + (int)lane / 4 < n
                           ? *reinterpret_cast<const uint4 *>(
                                 mine + nt * 8 * bytes + (p * a.hb + kb) * 256 + piece * 64)
                           : make_uint4(0u, 0u, 0u, 0u);
            });
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    inverse[nt][i] = nt * 8 + (int)first + i < n
                                         ? inverses[(nt * 8 + i) * (bytes / 4) + kb]
                                         : 0.0f;
        } else {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int c = nt * 8 + (int)lane / 4;
                RawColumn<DT> raw;
                raw.load(a.x + (uint64_t)(c < n ? list[c] / a.K : 0u) * a.sx, kb, a.H, a.wide_x,
                         c < n);
                uint4 hi[4], lo[4];
                const float inv = raw.template convert<kLo>(hi, lo);
                inverse[nt][0] = __shfl_sync(0xFFFFFFFFu, inv, lane % 4 * 8);
                inverse[nt][1] = __shfl_sync(0xFFFFFFFFu, inv, lane % 4 * 8 + 4);
                float one[kUpTiles][1][4] = {};
                block_product<kUpTiles, 1, C::kParts>(one, now, [&](int, int p, int piece) {
                    return p ? lo[piece] : hi[piece];
                });
#pragma unroll
                for (int m = 0; m < kUpTiles; ++m)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        part[m][nt][i] = one[m][0][i];
            }
        }
#pragma unroll
        for (int m = 0; m < kUpTiles; ++m)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sum[m][nt][i] += part[m][nt][i] * (inverse[nt][i & 1] * sc[m][i / 2]);
    }
    // the upper half of the warps hands its sums to the lower
    constexpr uint32_t kHalf = kUpWarps / 2;
    auto slot = [&](uint32_t w, int half, uint32_t r, uint32_t c) -> float & {
        return parts[((w * 2 + half) * kUpRows + r) * a.part_row + c];
    };
    auto each = [&](auto f) {
#pragma unroll
        for (int m = 0; m < kUpTiles; ++m)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    f(slot(warp % kHalf, i / 2, m * 8 + lane / 4, nt * 8 + lane % 4 * 2 + i % 2),
                      sum[m][nt][i]);
    };
    if (warp >= kHalf)
        each([](float &x, float v) { x = v; });
    __syncthreads();
    if (warp < kHalf)
        each([](float &x, float v) { x += v; });
    __syncthreads();
    // 16 lanes have the rows of one pair
    for (int c0 = (int)warp * 2; c0 < n; c0 += 2 * kUpWarps) {
        const int c = c0 + lane / kUpRows, r = lane % kUpRows;
        float h = 0.0f;
        if (c < n && f0 + r < a.F) {
            float g = 0.0f, u = 0.0f;
#pragma unroll
            for (uint32_t k = 0; k < kHalf; ++k) {
                g += slot(k, 0, r, c);
                u += slot(k, 1, r, c);
            }
            h = __fdiv_rn(g, 1.0f + expf(-g)) * u;
        }
        uint8_t *row = a.h + (uint64_t)(c < n ? list[c] : 0) * a.sh;
        if (!HiddenRow<DT>::kParts) {
            if (c < n && f0 + r < a.F)
                reinterpret_cast<float *>(row)[f0 + r] = h;
            continue;
        }
        float top = fabsf(h);
#pragma unroll
        for (int d = kUpRows / 2; d > 0; d >>= 1)
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
        if (c >= n)
            continue;
        const uint32_t step = tile_step(top), f = f0 + r, piece = HiddenRow<DT>::piece(f, a.F);
        const float v = h * step_scale(step);
        const uint32_t hi = __half_as_ushort(__float2half_rn(v));
        const float left = isinf(h) ? 0.0f : v - __half2float(__ushort_as_half(hi));
        uint8_t *at = row + (uint64_t)(f / 128) * 512 + f / 8 % 4 * piece + f / 32 % 4 * 16 +
                      f % 8 * 2;
        *reinterpret_cast<uint16_t *>(at) = (uint16_t)hi;
        *reinterpret_cast<uint16_t *>(at + 4 * piece) =
            (uint16_t)(r < 4 ? half_with_bit(left, step_bit(step, r))
                             : __half_as_ushort(__float2half_rn(left)));
    }
    __syncthreads();
}

template <int DT, bool BULK>
__global__ void __launch_bounds__(kUpThreads, 1)
k_moe_up(const __grid_constant__ MoeArgs a, const __grid_constant__ CUtensorMap map) {
    extern __shared__ uint8_t raw[];
    // the rings first: their swizzle wants 1024-byte boundaries
    uint8_t *rings = raw + ((1024u - (smem_at(raw) & 1023u)) & 1023u);
    UpShared &s = *reinterpret_cast<UpShared *>(
        rings + (BULK ? (uint32_t)kUpWarps * a.stages * Ring<2>::kStage : 0u));
    float *parts = reinterpret_cast<float *>(&s + 1);
    uint8_t *xs = reinterpret_cast<uint8_t *>(&s) + up_fixed(a.part_row);
    const uint32_t warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        s.failed = 0;
        for (int w = 0; w < kUpWarps; ++w)
            for (int i = 0; i < 2; ++i)
                mbar_init((uint32_t)__cvta_generic_to_shared(&s.bars[w][i]), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    // the second launch reads the choices and weights before its own wait, so it may come
    // only once what was before this one is done
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (blockIdx.x == 0 && threadIdx.x == 0)
        *a.status = AR_OK;
    choose(a, s.c);
    const uint32_t tiles = (a.F + kUpRows - 1) / kUpRows;
    // this CTA's run of (expert, rows)
    const uint64_t units = (uint64_t)s.c.count * tiles;
    uint64_t unit = units * blockIdx.x / gridDim.x;
    const uint64_t end = units * (blockIdx.x + 1) / gridDim.x;
    UpWarp me;
    me.map = &map;
    me.tiles = tiles;
    me.ring.begin(rings + warp * a.stages * Ring<2>::kStage, s.bars[warp], &s.failed, a.stages - 1);
    me.cursor.begin(a, tiles, unit, end);
    if (BULK)
        for (uint32_t i = 0; i < a.stages; ++i)
            me.fetch(a, s.c);
    while (unit < end) {
        const uint32_t i = (uint32_t)(unit / tiles), tile = (uint32_t)(unit - (uint64_t)i * tiles);
        const uint32_t last = end - unit < tiles - tile ? tile + (uint32_t)(end - unit) : tiles;
        const int e = s.c.active[i], all = s.c.pairs[i];
        for (int skip = 0; skip < all; skip += (int)a.columns) {
            int16_t *list = s.list[warp];
            list_pairs(a, s.c, e, skip, (int)a.columns, list);
            const int n = all - skip < (int)a.columns ? all - skip : (int)a.columns;
            if (BULK) {
                stage_columns<DT>(a, list, n, xs);
                __syncthreads();
            }
            for (uint32_t t = tile; t < last; ++t) {
                if (n <= 8)
                    up_unit<DT, BULK, 1>(a, s, me, parts, xs, e, t * kUpRows, n);
                else
                    up_unit<DT, BULK, 2>(a, s, me, parts, xs, e, t * kUpRows, n);
            }
        }
        unit += last - tile;
    }
    __syncthreads();
    if (BULK && s.failed && threadIdx.x % 32 == 0)
        me.ring.drain();
    if (threadIdx.x == 0)
        a.failed[blockIdx.x] = s.failed != 0;
}

// ---- second launch --------------------------------------------------------------

constexpr int kDownWarps = 8, kDownThreads = 32 * kDownWarps;
// (four stages: the same; three CTAs an SM with registers for two: 114 us for one token
// of 8192 x 2048, not 80, both with h in one binary16 number)
constexpr int kDownStagesLog2 = 1, kDownStages = 1 << kDownStagesLog2;
// Most tokens whose sums leave room for a second CTA beside tiles of 32 rows.
constexpr uint32_t kDownTokens = 32;

struct DownShared {
    Chosen c;
    int16_t list[kDownWarps][kColumns];
    uint64_t bars[kDownWarps][kDownStages];
    int failed;
    alignas(16) float sums[1];        // [warp][token][row]
};
template <int MT> static size_t down_smem(uint32_t T, bool bulk) {
    return (bulk ? 1024 + kDownWarps * kDownStages * Ring<MT>::kStage : 0) + sizeof(DownShared) +
           sizeof(float) * kDownWarps * 16 * MT * T;
}

// The steps of a warp of the second launch: its blocks of (expert, k), a run of them, and
// for each expert's share of it the passes over the expert's pairs.
struct DownCursor {
    uint32_t i, kb0, kb1, kb, pass, left;     // left: blocks past this expert's
    bool done;

    __device__ __forceinline__ void begin(const MoeArgs &a, uint32_t at, uint32_t end) {
        i = at / a.fb;
        kb = kb0 = at - i * a.fb;
        kb1 = end - at < a.fb - kb0 ? kb0 + (end - at) : a.fb;
        left = end - at - (kb1 - kb0);
        pass = 0;
        done = at >= end;
    }
    __device__ __forceinline__ void next(const MoeArgs &a, const Chosen &c) {
        if (++kb < kb1)
            return;
        kb = kb0;
        if (++pass * kColumns < (uint32_t)c.pairs[i])
            return;
        pass = 0;
        ++i;
        kb = kb0 = 0;
        kb1 = left < a.fb ? left : a.fb;
        left -= kb1;
        done = kb1 == 0;
    }
};

template <int MT> struct DownWarp {
    Ring<MT> ring;
    DownCursor cursor;
    const CUtensorMap *map;
    uint32_t r0;

    __device__ __forceinline__ void fetch(const MoeArgs &a, const Chosen &c) {
        if (cursor.done)
            return;
        if ((threadIdx.x & 31) == 0 && !*ring.failed) {
            uint32_t rows[MT];
#pragma unroll
            for (int m = 0; m < MT; ++m)
                rows[m] = r0 + 16 * m;
            ring.issue(map, cursor.kb * 128, rows, c.active[cursor.i]);
        }
        cursor.next(a, c);
    }
};

// The lane's elements of a row of h, block kb, in two parts.
template <int DT> struct Hidden;
template <> struct Hidden<AR_FP32> {
    RawColumn<AR_FP32> v;
    uint4 parts[2][4];
    __device__ __forceinline__ void load(const MoeArgs &a, const uint8_t *row, uint32_t kb,
                                         bool on) {
        v.load(row, kb, a.F, true, on);
    }
    // the inverse of the block's scale
    __device__ __forceinline__ float convert(const MoeArgs &, uint32_t) {
        return v.convert<true>(parts[0], parts[1]);
    }
};
template <int DT> struct Hidden {
    uint4 parts[2][4];
    __device__ __forceinline__ void load(const MoeArgs &a, const uint8_t *row, uint32_t kb,
                                         bool on) {
        const uint32_t c = threadIdx.x & 3, k = kb * 128 + c * 32;
        const uint32_t piece = HiddenRow<DT>::piece(kb * 128, a.F);
        row += (uint64_t)kb * 512 + c * 16;
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                parts[p][j] = make_uint4(0u, 0u, 0u, 0u);
                if (on && k + 16 * (j / 2) < a.F)
                    parts[p][j] = ld_v4_l1(row + (4 * p + j) * piece);
            }
    }
    // The inverse of the block's scale.  Tiles of several steps are brought to one scale in
    // binary32, as in Hidden<AR_FP32>.
    __device__ __forceinline__ float convert(const MoeArgs &a, uint32_t kb) {
        uint32_t step[2], most;
#pragma unroll
        for (int t = 0; t < 2; ++t)
            step[t] = step_of(parts[1][2 * t].x, parts[1][2 * t].y);
        most = max(step[0], step[1]);
        most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
        most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
        const float inverse = step_inverse(most);
        const uint32_t k = kb * 128 + (threadIdx.x & 3) * 32;
        if (__all_sync(0xFFFFFFFFu, (step[0] == most || k >= a.F) &&
                                        (step[1] == most || k + 16 >= a.F)))
            return inverse;
        float v[32];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const uint32_t down = 16 * (most - step[i / 8]);      // 240 at most
            const float by = down < 120 ? __uint_as_float((127 - down) << 23) : 0.0f;
            const float2 hi = widen2<AR_FP16>(word_of(parts[0][i / 4], i % 4));
            const float2 lo = widen2<AR_FP16>(word_of(parts[1][i / 4], i % 4));
            v[2 * i] = (hi.x + lo.x) * by;
            v[2 * i + 1] = (hi.y + lo.y) * by;
        }
        return inverse * convert_column<true>(v, parts[0], parts[1]);
    }
};
// The line that p is in to L1: a load that nothing waits for (prefetch.global.L1 did not
// bring it there).
__device__ __forceinline__ void touch_l1(const void *p) {
    asm volatile("{\n\t.reg .b32 unused;\n\tld.global.u32 unused, [%0];\n\t}" :: "l"(p));
}

// Blocks [kb0, kb1) along k of expert e times the listed pairs, added to this warp's
// sums of their tokens.
template <int DT, bool BULK, int MT, int NT>
__device__ __forceinline__ void down_part(const MoeArgs &a, const Chosen &c, DownWarp<MT> &me,
                                          const int16_t *list, float *sums, int e, uint32_t kb0,
                                          uint32_t kb1, int n) {
    const int lane = threadIdx.x & 31;
    const uint8_t *w = a.down + (uint64_t)e * a.H * a.lddown;
    const float *ws = a.down_scale + (uint64_t)e * a.hb * a.fb;
    // rows past the last stand in for it: their sums go nowhere
    auto row_of = [&](int m, int i) {
        const uint32_t r = me.r0 + 16 * m + i * 8 + lane / 4;
        return r < a.H ? r : a.H - 1;
    };
    // a tile's 16 rows lie in one block of 128
    const float *scales[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
        scales[m] = ws + (uint64_t)(row_of(m, 0) / 128) * a.fb;
    const uint8_t *columns[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int x = nt * 8 + lane / 4;
        columns[nt] = a.h + (uint64_t)(x < n ? list[x] : 0) * a.sh;
    }
    float sum[MT][NT][4] = {}, next_scale[MT];
    auto load_scales = [&](uint32_t kb) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
            next_scale[m] = scales[m][kb];
    };
    load_scales(kb0);
    for (uint32_t kb = kb0; kb < kb1; ++kb) {
        float sc[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m)
            sc[m] = next_scale[m];
        Hidden<DT> h;
        auto load_h = [&](int nt) { h.load(a, columns[nt], kb, nt * 8 + lane / 4 < n); };
        load_h(0);                    // on its way while the weights are waited for
        if (kb + 1 < kb1) {
            load_scales(kb + 1);
            // the next block's columns, a line of 128 bytes a lane: registers have no room
            // for them (one token: 85 us; without this 87.5; in registers a block ahead 97)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                if ((kb + 1) * 128 + lane % 4 * 32 < a.F)
                    touch_l1(columns[nt] + (uint64_t)(kb + 1) * 512 + lane % 4 * 128);
        }
        Codes<MT> now;
        if (BULK) {
            me.ring.wait();
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    now.q[m][i] = me.ring.codes(m, i * 8 + lane / 4);
            __syncwarp();
            ++me.ring.steps.used;
            me.fetch(a, c);
        } else {
            const uint32_t k = kb * 128 + lane % 4 * 32;
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint8_t *row = w + (uint64_t)row_of(m, i) * a.lddown;
                    now.q[m][i].lo = load_codes(row, k, a.F);
                    now.q[m][i].hi = load_codes(row, k + 16, a.F);
                }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if (nt > 0)
                load_h(nt);
            const float inv = h.convert(a, kb);
            const float inverse[2] = {__shfl_sync(0xFFFFFFFFu, inv, lane % 4 * 8),
                                      __shfl_sync(0xFFFFFFFFu, inv, lane % 4 * 8 + 4)};
            // (the parts' sums apart, two chains of half the length: 88 us for one token, not 85)
            float part[MT][1][4] = {};
            block_product<MT, 1, 2>(part, now, [&](int, int p, int piece) {
                return h.parts[p][piece];
            });
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sum[m][nt][i] += part[m][0][i] *
                                     (inverse[i & 1] * sc[m]);
        }
    }
    // columns of different pairs may be one token's (its choices of one expert): one
    // column at a time
    for (int x = 0; x < n; ++x) {
        const int p = list[x];
        const float g = a.w ? a.w[p] : 1.0f;
        if (lane % 4 == x % 8 / 2) {
            float *token = sums + (uint32_t)p / a.K * (16 * MT);
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    if (nt == x / 8)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            token[16 * m + i * 8 + lane / 4] +=
                                g * (x & 1 ? sum[m][nt][2 * i + 1] : sum[m][nt][2 * i]);
        }
        __syncwarp();
    }
}

// MT: tiles of 16 rows of the output.
template <int DT, bool BULK, int MT>
__global__ void __launch_bounds__(kDownThreads, 2)
k_moe_down(const __grid_constant__ MoeArgs a, const __grid_constant__ CUtensorMap map) {
    extern __shared__ uint8_t raw[];
    uint8_t *rings = raw + (BULK ? (1024u - (smem_at(raw) & 1023u)) & 1023u : 0u);
    DownShared &s = *reinterpret_cast<DownShared *>(
        rings + (BULK ? (uint32_t)kDownWarps * kDownStages * Ring<MT>::kStage : 0u));
    constexpr uint32_t kDownRows = 16 * MT;
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        s.failed = 0;
        for (int w = 0; w < kDownWarps; ++w)
            for (int i = 0; i < kDownStages; ++i)
                mbar_init((uint32_t)__cvta_generic_to_shared(&s.bars[w][i]), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    // before the wait: the choices and the first weights, which were there before the first
    // launch
    choose(a, s.c);
    const uint32_t each = a.T * kDownRows;
    float *mine = s.sums + (uint32_t)warp * each;
    for (uint32_t i = threadIdx.x; i < each * kDownWarps; i += kDownThreads)
        s.sums[i] = 0.0f;
    __syncthreads();
    DownWarp<MT> me;
    me.map = &map;
    me.r0 = blockIdx.x * kDownRows;
    me.ring.begin(rings + warp * kDownStages * Ring<MT>::kStage, s.bars[warp], &s.failed,
                  kDownStagesLog2);
    // this warp's run of (expert, block)
    const uint32_t steps = (uint32_t)s.c.count * a.fb;
    const uint32_t from = (uint32_t)((uint64_t)steps * warp / kDownWarps);
    const uint32_t end = (uint32_t)((uint64_t)steps * (warp + 1) / kDownWarps);
    me.cursor.begin(a, from, end);
    if (BULK)
        for (int i = 0; i < kDownStages; ++i)
            me.fetch(a, s.c);
    kernel_prologue();
    int failed = 0;
    for (uint32_t i = threadIdx.x; i < a.ups; i += kDownThreads)
        failed |= a.failed[i];
    for (uint32_t at = from; at < end;) {
        const uint32_t i = at / a.fb, kb0 = at - i * a.fb;
        const uint32_t kb1 = end - at < a.fb - kb0 ? kb0 + (end - at) : a.fb;
        const int e = s.c.active[i], all = s.c.pairs[i];
        for (int skip = 0; skip < all; skip += kColumns) {
            list_pairs(a, s.c, e, skip, kColumns, s.list[warp]);
            const int n = all - skip < kColumns ? all - skip : kColumns;
            if (n <= 8)
                down_part<DT, BULK, MT, 1>(a, s.c, me, s.list[warp], mine, e, kb0, kb1, n);
            else
                down_part<DT, BULK, MT, 2>(a, s.c, me, s.list[warp], mine, e, kb0, kb1, n);
        }
        at += kb1 - kb0;
    }
    if (BULK && *me.ring.failed && threadIdx.x % 32 == 0)
        me.ring.drain();
    failed = __syncthreads_or(failed | s.failed);
    if (failed && threadIdx.x == 0)
        *a.status = AR_ERR_TIMEOUT;
    for (uint32_t i = threadIdx.x; i < each; i += kDownThreads) {
        const uint32_t t = i / kDownRows, r = i % kDownRows;
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < kDownWarps; ++k)
            v += s.sums[k * each + i];
        if (failed)
            v = NAN;
        if (me.r0 + r < a.H)
            st_elem<DT>(a.out + t * a.sout, me.r0 + r, narrow1<DT>(v));
    }
}

// Columns of an expert that fit beside rings of this many stages, no more than there can
// be.
template <int DT> static uint32_t up_columns(const MoeArgs &a, uint32_t stages) {
    const size_t column = UpColumn<DT>::bytes(a.hb), pairs = (size_t)a.T * a.K;
    const size_t rings = 1024 + kUpWarps * stages * Ring<2>::kStage;
    size_t n = (kMoeSmem - rings - up_fixed(9)) / column;
    if (n > 8) {
        n = (kMoeSmem - rings - up_fixed(kColumns + 1)) / column;
        n = n < 8 ? 8 : n;
    }
    n = n < kColumns ? n : kColumns;
    return (uint32_t)(n < pairs ? n : pairs);
}

// The first launch; sets what the second needs to know of it.
template <int DT, bool BULK>
static cudaError_t launch_up(MoeArgs &a, const CUtensorMap &map, int sms, cudaStream_t s) {
    const cudaError_t e = opt_in_smem<k_moe_up<DT, BULK>>(kMoeSmem);
    if (e != cudaSuccess)
        return e;
    const uint64_t pairs = (uint64_t)a.T * a.K;
    size_t smem;
    if (BULK) {
        // Rings of two stages where the columns of nearly every expert fit beside them (8
        // tokens, top 8 of 64 experts of 8192 x 1024: 215 us; one stage 221), else of one
        // (16 tokens: 293; two stages, and a second pass over the weights for more than four
        // columns, 387).
        const uint32_t mean = (uint32_t)((pairs + a.E - 1) / a.E), likely = 2 * mean + 2;
        a.stages = up_columns<DT>(a, 2) >= (likely < a.T ? likely : a.T) ? 2 : 1;
        a.columns = up_columns<DT>(a, a.stages);
        a.part_row = a.columns <= 8 ? 9 : kColumns + 1;
        smem = 1024 + kUpWarps * a.stages * Ring<2>::kStage + up_fixed(a.part_row) +
               a.columns * UpColumn<DT>::bytes(a.hb);
    } else {
        a.columns = pairs < kColumns ? (uint32_t)pairs : kColumns;
        a.part_row = kColumns + 1;
        smem = 1024 + up_fixed(a.part_row);
    }
    const uint64_t units = (uint64_t)((a.F + kUpRows - 1) / kUpRows) * pairs;
    a.ups = (uint32_t)(units < (uint64_t)sms ? units : (uint64_t)sms);
    // The flags lie at the workspace's end, past the rows of h and before the status word.  A
    // pair has 4 F + 512 bytes there, of which its row leaves 388 at least.
    if (a.ups > 384)
        a.ups = 384;
    a.failed -= a.ups;
    return launch_kernel(k_moe_up<DT, BULK>, a.ups, kUpThreads, smem, s, true, a, map);
}
template <int DT, bool BULK, int MT>
static cudaError_t launch_down(const MoeArgs &a, const CUtensorMap &map, cudaStream_t s) {
    constexpr uint32_t most = MT == 1 ? AR_MOE_LAYER_TOKENS : kDownTokens;
    const cudaError_t e = opt_in_smem<k_moe_down<DT, BULK, MT>>(down_smem<MT>(most, BULK));
    if (e != cudaSuccess)
        return e;
    return launch_kernel(k_moe_down<DT, BULK, MT>, (a.H + 16 * MT - 1) / (16 * MT), kDownThreads,
                         down_smem<MT>(a.T, BULK), s, true, a, map);
}

template <int DT>
static cudaError_t moe_dt(MoeArgs a, bool bulk_up, bool bulk_down, cudaStream_t s) {
    const int sms = sm_count();
    if (sms < 1)
        return cudaErrorUnknown;
    a.sh = HiddenRow<DT>::bytes(a.F);
    CUtensorMap up = {}, down = {};
    // without room for a column the first launch reads them on the way
    bulk_up = bulk_up && up_columns<DT>(a, 1) > 0;
    if ((bulk_up || bulk_down) && !encoder())
        return cudaErrorNotSupported;
    if ((bulk_up && !encode(&up, a.up, a.H, 2 * (uint64_t)a.F, a.ldup, a.E, 16)) ||
        (bulk_down && !encode(&down, a.down, a.F, a.H, a.lddown, a.E, 16)))
        return cudaErrorInvalidValue;
    const cudaError_t e =
        bulk_up ? launch_up<DT, true>(a, up, sms, s) : launch_up<DT, false>(a, up, sms, s);
    if (e != cudaSuccess)
        return e;
    if (!bulk_down)
        return launch_down<DT, false, 1>(a, down, s);
    // 32 rows a CTA where that leaves no SM without one (8 and 16 tokens of 8192 x 1024: 215
    // and 293 us; 16 rows 225 and 308; one token of 8192 x 2048 85, so 86)
    return a.H / 32 >= (uint32_t)sms && a.T <= kDownTokens ? launch_down<DT, true, 2>(a, down, s)
                                                          : launch_down<DT, true, 1>(a, down, s);
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
    a.h = reinterpret_cast<uint8_t *>(work);
    a.sx = mx.stride;
    a.sout = mo.stride;
    a.ldup = mu.stride;
    a.lddown = md.stride;
    a.T = (uint32_t)T;
    a.K = (uint32_t)K;
    a.H = (uint32_t)H;
    a.F = (uint32_t)F;
    a.E = (uint32_t)E;
    a.hb = (uint32_t)hb;
    a.fb = (uint32_t)fb;
    a.ub = (uint32_t)ub;
    a.columns = a.ups = a.stages = a.part_row = 0;
    a.status = reinterpret_cast<int *>(work) + mw.bytes / 4 - 1;
    a.failed = reinterpret_cast<uint8_t *>(a.status);             // less a byte per CTA
    a.wide_x = wide(mx);
    a.ids8 = ids_bytes == 8;
    const bool bu = wide(mu), bd = wide(md);
    switch (dtype) {
    case AR_BF16: return launched(moe_dt<AR_BF16>(a, bu, bd, stream));
    case AR_FP16: return launched(moe_dt<AR_FP16>(a, bu, bd, stream));
    default: return launched(moe_dt<AR_FP32>(a, bu, bd, stream));
    }
}

}  // extern "C"
