// What the kernels of attention over the paged cache share: their arguments, the
// deal of tiles to CTAs, the workspace, and how a unit ends.
#pragma once

#include "ar_cache.cuh"

namespace ar {

constexpr int kPartRows = 14976;      // rows of partial results: two parts a CTA
constexpr int kMaxCtas = kPartRows / 2 / 8;
constexpr float kLog2E = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct AttnArgs {
    Pages g;
    const uint8_t *q;
    uint8_t *out;
    float *lse;
    float *work;
    uint64_t sq, sout;                // bytes between rows
    float scale2;                     // scale * log2 e
    uint32_t B, heads, group;         // group: query heads that share a key-value head
    uint32_t unit_rows;               // query heads of a unit: 8, 16 or 32
    uint32_t head_tiles;              // units of one key-value head
    uint32_t window;                  // 0: none
    int runs;                         // tiles begin at multiples of 16 positions
    uint32_t cluster;                 // CTAs of a unit that share it by rank; 0: runs of tiles
};

// The CTAs that a launch of `most` may have: parts for all of them fit.
inline int cta_limit(uint32_t unit_rows, int most) {
    const int limit = kPartRows / 2 / (int)unit_rows;
    return most < limit ? most : limit;
}

// The workspace: where a CTA's first unit that others finish is, then (m, l) and o
// of unit_rows rows for two parts of each CTA: part 0 continues a unit, part 1 begins
// one.
struct WorkSpace {
    int4 *meta;                       // sequence, unit, last CTA (-1: none)
    float2 *ml;
    float *o;
    __device__ __forceinline__ explicit WorkSpace(float *work)
        : meta(reinterpret_cast<int4 *>(work)),
          ml(reinterpret_cast<float2 *>(work + 4 * kMaxCtas)),
          o(work + 4 * kMaxCtas + 2 * kPartRows) {}
};
static_assert(4 * kMaxCtas + 2 * kPartRows + kPartRows <= AR_CACHE_WORK_ROWS * 3 &&
                  kPartRows <= AR_CACHE_WORK_ROWS,
              "the workspace has room for D = 1, and so for every D");
static_assert((4 * kMaxCtas + 2 * kPartRows) % 4 == 0, "o starts on a 16-byte boundary");

// The range of positions [lo, n) of a sequence; its first tile begins at `origin`.
struct Span {
    uint32_t lo, n, origin;
};
__device__ __forceinline__ Span span_of(const AttnArgs &a, uint32_t b) {
    const uint32_t n = a.g.length(b), lo = a.window && n > a.window ? n - a.window : 0u;
    return {lo, n, a.runs ? lo & ~15u : lo};
}
template <uint32_t TILE> __device__ __forceinline__ uint32_t tiles_of(Span s) {
    return (s.n - s.origin + TILE - 1) / TILE;
}

// Beginning and ending a unit costs about as much as this many tiles: the deal counts
// them, so that CTAs with many short units have fewer tiles (64 sequences of 256 to
// 16384, 64 / 8 heads of 128 in 8 bits: 113 us with the other changes of that step, 151
// without).  A unit of n tiles has kUnitCost + n places in the order; the first
// kUnitCost of them stand for no tile.
constexpr uint32_t kUnitCost = 2;

// A place in a CTA's run: tiles [t, t1) of a unit.
template <uint32_t TILE> struct Cursor {
    uint32_t b, unit, t, t1, tiles;
    Span span;
    uint64_t base;                    // place of the unit's first
    uint64_t left;                    // places of the run past the unit's

    __device__ __forceinline__ bool done() const { return t >= t1; }
    __device__ __forceinline__ void begin(const AttnArgs &a, uint64_t in) {
        // the run enters the unit at its place `in`
        const uint64_t all = kUnitCost + tiles, end = all - in < left ? all : in + left;
        left -= end - in;
        t = in > kUnitCost ? (uint32_t)(in - kUnitCost) : 0u;
        t1 = end > kUnitCost ? (uint32_t)(end - kUnitCost) : 0u;
        if (t >= t1 && left > 0)      // places for no tile only
            next_unit(a);
    }
    // Share `rank` of `parts` of one unit, counted over all sequences.
    __device__ __forceinline__ void share(const AttnArgs &a, uint32_t index, uint32_t rank,
                                          uint32_t parts) {
        const uint32_t units = a.g.heads * a.head_tiles;
        b = index / units;
        unit = index - b * units;
        span = span_of(a, b);
        tiles = tiles_of<TILE>(span);
        t = (uint32_t)((uint64_t)tiles * rank / parts);
        t1 = (uint32_t)((uint64_t)tiles * (rank + 1) / parts);
        left = 0;
    }
    __device__ __forceinline__ void next_unit(const AttnArgs &a) {
        t = t1 = 0;
        if (left == 0)
            return;
        base += kUnitCost + tiles;
        if (++unit == a.g.heads * a.head_tiles) {
            unit = 0;
            do {
                span = span_of(a, ++b);
                tiles = tiles_of<TILE>(span);
            } while (tiles == 0);     // `left` says that there is another
        }
        const uint64_t all = kUnitCost + tiles, end = all < left ? all : left;
        left -= end;
        t1 = end > kUnitCost ? (uint32_t)(end - kUnitCost) : 0u;
    }
    __device__ __forceinline__ void next(const AttnArgs &a) {
        if (++t >= t1)
            next_unit(a);
    }
};

// a / b; in 32 bits where that does, for a fraction of the time.
__device__ __forceinline__ uint64_t divide(uint64_t a, uint64_t b) {
    return (a | b) >> 32 ? a / b : (uint64_t)((uint32_t)a / (uint32_t)b);
}

// This CTA's run.  `part` is shared memory of 32 words.  *per: places of a run.
template <uint32_t TILE>
__device__ __forceinline__ Cursor<TILE> find_run(const AttnArgs &a, uint64_t *part,
                                                 uint64_t *per) {
    // every thread counts a run of sequences; their sums are scanned
    const uint32_t each = (a.B + blockDim.x - 1) / blockDim.x;
    const uint32_t b0 = threadIdx.x * each;
    const uint32_t b1 = b0 + each < a.B ? b0 + each : a.B;
    const uint32_t units = a.g.heads * a.head_tiles;
    auto places = [&](uint32_t b) -> uint64_t {
        const uint32_t n = tiles_of<TILE>(span_of(a, b));
        return n ? (uint64_t)(n + kUnitCost) * units : 0;
    };
    uint64_t mine = 0;
    for (uint32_t b = b0; b < b1; ++b)
        mine += places(b);
    uint64_t sum = mine;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint64_t other = __shfl_up_sync(0xFFFFFFFFu, sum, d);
        if (lane >= d)
            sum += other;
    }
    __shared__ uint32_t at[2];
    __shared__ uint64_t before;
    if (lane == 31)
        part[warp] = sum;
    if (threadIdx.x == 0)
        at[1] = 0;
    __syncthreads();
    uint64_t total = 0;
    for (int w = 0; w < (int)(blockDim.x >> 5); ++w) {
        if (w < warp)
            sum += part[w];
        total += part[w];
    }
    *per = divide(total + gridDim.x - 1, gridDim.x);
    const uint64_t start = *per * blockIdx.x;
    if (start >= sum - mine && start < sum) {
        uint64_t base = sum - mine;
        uint32_t b = b0;
        for (;; ++b) {
            const uint64_t n = places(b);
            if (start < base + n)
                break;
            base += n;
        }
        at[0] = b;
        at[1] = 1;
        before = base;
    }
    __syncthreads();
    Cursor<TILE> c = {};
    if (!at[1])
        return c;                         // past the last place
    c.b = at[0];
    c.span = span_of(a, c.b);
    c.tiles = tiles_of<TILE>(c.span);
    const uint64_t all = kUnitCost + c.tiles, in = start - before;
    c.unit = (uint32_t)divide(in, all);
    c.base = before + c.unit * all;
    c.left = total - start < *per ? total - start : *per;
    c.begin(a, in - c.unit * all);
    return c;
}

template <int DT> __device__ __forceinline__ void store_row(uint8_t *row, uint32_t d, float v) {
    st_elem<DT>(row, d, narrow1<DT>(v));
}

// Zeros (and -inf) for the sequences that have no position.
template <int DT, uint32_t TILE> __device__ __forceinline__ void empty_rows(const AttnArgs &a) {
    for (uint32_t b = blockIdx.x; b < a.B; b += gridDim.x) {
        if (tiles_of<TILE>(span_of(a, b)) != 0)
            continue;
        uint8_t *row = a.out + (uint64_t)b * a.sout;
        for (uint32_t i = threadIdx.x; i < a.heads * a.g.D; i += blockDim.x)
            store_row<DT>(row, i, 0.0f);
        if (a.lse)
            for (uint32_t h = threadIdx.x; h < a.heads; h += blockDim.x)
                a.lse[(uint64_t)b * a.heads + h] = -INFINITY;
    }
}

__device__ __forceinline__ float lse_of(float m, float l) {
    return l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
}
// o / l, and 0 for a row without a weight; NaN stays.
__device__ __forceinline__ float output_of(float o, float l) {
    return l == 0.0f ? 0.0f : __fdiv_rn(o, l);
}
// What the running maximum subtracts: a row of -inf alone keeps weights of 0.
__device__ __forceinline__ float finite_max(float m) { return m == -INFINITY ? 0.0f : m; }

// The running maximum follows a row's scores only when one is this far above it
// (as exponents of two): weights up to 2^4 cost nothing, new factors for all of o do.
constexpr float kSlack = 4.0f;

// Where a unit's rows go: first query head, rows.
struct UnitRows {
    uint32_t kv, head, rows;
};
__device__ __forceinline__ UnitRows unit_rows(const AttnArgs &a, uint32_t unit) {
    UnitRows u;
    u.kv = unit / a.head_tiles;
    const uint32_t r0 = unit % a.head_tiles * a.unit_rows;
    u.head = u.kv * a.group + r0;
    u.rows = a.group - r0 < a.unit_rows ? a.group - r0 : a.unit_rows;
    return u;
}

// How the cursor's segment ends: its unit is finished (-1), or it is a part for the
// join, and which.  Thread 0 notes the unit's last CTA.
template <uint32_t TILE>
__device__ __forceinline__ int segment_part(const AttnArgs &a, const Cursor<TILE> &c,
                                            uint64_t per) {
    if (c.t == 0 && c.t1 == c.tiles)
        return -1;
    if (c.t != 0)
        return 2 * blockIdx.x;
    if (threadIdx.x == 0) {
        const uint64_t last = (c.base + kUnitCost + c.tiles - 1) / per;
        WorkSpace(a.work).meta[blockIdx.x] = make_int4((int)c.b, (int)c.unit, (int)last, 0);
    }
    return 2 * blockIdx.x + 1;
}

// ar_cache_attention_mma.cu: the tensor-core form, for keys and values of one or two
// bytes whose rows are whole 16-byte vectors on 16-byte boundaries.  Sets the units of
// `a`; *grid: the CTAs whose parts a join has to look at, 0 if there are none.
cudaError_t launch_attention_mma(AttnArgs &a, int dtype, bool e4m3, int *grid, cudaStream_t s);
// ar_cache_attention_units.cu: its other form, without a join.  The first says whether it
// serves `a` where `room` CTAs run at a time, and sets a.cluster.
bool attention_units(AttnArgs &a, int room);
cudaError_t launch_attention_units(const AttnArgs &a, int dtype, bool e4m3, cudaStream_t s);

}  // namespace ar
