// Rows of keys and values into the pages of their sequences, and back.
//
//   as they are, or  scale = max(max |x|, 2^-96) / 448,  code = e4m3(x / scale)
//
// Bound by memory: every row is read once and written once (65536 rows of 8 heads of 128
// bf16 from 8 bits: 64.2 us, 6.3 TB/s; 8192 rows to 8 bits 11.2, about 3 of it launch and
// lookup).  Rows that are not 16-byte vectors go by elements (30000 rows of 7 x 101 bf16
// to 8 bits: 119 us, 1.1 TB/s).  A CTA takes a few rows of all heads; a line (one head's D elements of k or of v) belongs to a
// power of two of consecutive lanes, so that its largest magnitude is found by
// shuffles.  Writing, the rows' loads are issued before their places are looked
// up (offsets, length and page table depend on one another), reading after.
#include "ar_cache.cuh"

namespace ar {

struct MoveArgs {
    Pages g;
    uint8_t *k, *v;               // the rows
    uint64_t sk, sv;              // bytes between rows
    const int32_t *offsets;
    uint32_t T, B;
    uint32_t rows;                // rows of a job
    uint32_t slots;               // lanes of a row: 2 * heads << lane_bits
    uint32_t jobs_per_row;        // jobs that share one row (rows = 1 then)
    uint32_t lane_bits;
    Divide by_lines;              // the lines of a row
};

constexpr int kMoveThreads = 256;
constexpr int kMoveSlots = 2;     // slots of a thread in flight
constexpr int kMoveRows = 64;     // most rows of a job

// One lane's share of a line.  WIDE: N vectors of 16 bytes, vector i at unit
// lane + (i << bits).  Otherwise N = 8 single elements, element lane + 32 * i.
template <int DT, bool WIDE, int N> struct Line {
    static constexpr int kSize = Elem<DT>::kSize;
    static constexpr int E = WIDE ? 16 / kSize : 1;
    uint4 w[WIDE ? N : (N + 3) / 4];

    static __device__ __forceinline__ uint32_t at(uint32_t lane, int i, uint32_t bits) {
        return WIDE ? (lane + ((uint32_t)i << bits)) * E : lane + 32u * i;
    }
    __device__ __forceinline__ uint32_t &word(int i) { return (&w[i / 4].x)[i % 4]; }
    __device__ __forceinline__ void load(const uint8_t *line, uint32_t lane, uint32_t bits,
                                         uint32_t D) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t e = at(lane, i, bits);
            if (WIDE) {
                w[i] = make_uint4(0u, 0u, 0u, 0u);
                if (e < D)
                    w[i] = ld_v4_stream(line + (uint64_t)e * kSize);
            } else {
                word(i) = e < D ? ld_elem<DT>(line, e) : 0u;
            }
        }
    }
    __device__ __forceinline__ void store(uint8_t *line, uint32_t lane, uint32_t bits,
                                          uint32_t D) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t e = at(lane, i, bits);
            if (e >= D)
                continue;
            if (WIDE)
                st_v4(line + (uint64_t)e * kSize, w[i]);
            else
                st_elem<DT>(line, e, word(i));
        }
    }
    __device__ __forceinline__ void widen(int i, float *v) const {
        if (!WIDE) {
            v[0] = widen1<DT>((&w[i / 4].x)[i % 4]);
        } else {
            Rows<DT, true>::widen(w[i], v);
        }
    }
    __device__ __forceinline__ void narrow(int i, const float *v) {
        if (!WIDE) {
            word(i) = narrow1<DT>(v[0]);
        } else if (kSize == 2) {
            w[i] = make_uint4(narrow2<DT>(v[0], v[1]), narrow2<DT>(v[2], v[3]),
                              narrow2<DT>(v[4 % E], v[5 % E]), narrow2<DT>(v[6 % E], v[7 % E]));
        } else {
            w[i] = make_uint4(narrow1<DT>(v[0]), narrow1<DT>(v[1]), narrow1<DT>(v[2]),
                              narrow1<DT>(v[3]));
        }
    }
};

// Two binary32 values to two E4M3 codes, `a` in the low byte, and back.
__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b) {
    uint16_t q;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(q) : "f"(b), "f"(a));
    return q;
}
__device__ __forceinline__ uint32_t to_e4m3x4(const float t[4]) {
    uint32_t q;
    asm("{\n\t.reg .b16 x, y;\n\tcvt.rn.satfinite.e4m3x2.f32 x, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 y, %4, %3;\n\tmov.b32 %0, {x, y};\n\t}"
        : "=r"(q) : "f"(t[0]), "f"(t[1]), "f"(t[2]), "f"(t[3]));
    return q;
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t q) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)q));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// The larger magnitudes of two words of two elements; a NaN gives way to a number.
template <int DT> __device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b) {
    if (DT == AR_BF16) {
        const __nv_bfloat162 m = __hmax2(__habs2(*reinterpret_cast<const __nv_bfloat162 *>(&a)),
                                         __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&b)));
        return *reinterpret_cast<const uint32_t *>(&m);
    }
    const __half2 m = __hmax2(__habs2(*reinterpret_cast<const __half2 *>(&a)),
                              __habs2(*reinterpret_cast<const __half2 *>(&b)));
    return *reinterpret_cast<const uint32_t *>(&m);
}
// The same, whole lines: the largest magnitude among 1 << bits lanes' elements.
template <int DT, bool WIDE, int N>
__device__ __forceinline__ float largest(const Line<DT, WIDE, N> &line, bool on, uint32_t bits) {
    using L = Line<DT, WIDE, N>;
    if constexpr (WIDE && L::kSize == 2) {
        uint32_t top = 0u;
        if (on)
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const uint4 w = line.w[n];
                top = max_abs2<DT>(max_abs2<DT>(top, max_abs2<DT>(w.x, w.y)),
                                   max_abs2<DT>(w.z, w.w));
            }
        for (int d = (1 << bits) / 2; d > 0; d >>= 1)
            top = max_abs2<DT>(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
        const float2 f = widen2<DT>(top);
        return fmaxf(f.x, fmaxf(f.y, 0.0f));          // 0 where all are NaN
    } else {
        float top = 0.0f;
        if (on)
#pragma unroll
            for (int n = 0; n < N; ++n) {
                float v[8];
                line.widen(n, v);
#pragma unroll
                for (int e = 0; e < L::E; ++e)
                    top = fmaxf(top, fabsf(v[e]));
            }
        for (int d = (1 << bits) / 2; d > 0; d >>= 1)
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
        return top;
    }
}

// What one slot works on.
struct SlotOf {
    uint32_t row, head, lane;
    bool value, on;               // of v; there is such a slot
};
__device__ __forceinline__ SlotOf slot_of(const MoveArgs &a, uint32_t slot, uint32_t rows) {
    SlotOf s;
    const uint32_t line = slot >> a.lane_bits;
    s.lane = slot & ((1u << a.lane_bits) - 1u);
    s.row = a.by_lines(line);
    const uint32_t kv = line - s.row * 2u * a.g.heads;
    s.value = kv >= a.g.heads;
    s.head = s.value ? kv - a.g.heads : kv;
    s.on = s.row < rows;
    return s;
}

// CACHE8: the cache holds E4M3.  READ: out of the pages.
template <int DT, bool WIDE, int N, bool CACHE8, bool READ>
__global__ void __launch_bounds__(kMoveThreads)
k_cache_move(const __grid_constant__ MoveArgs a) {
    using L = Line<DT, WIDE, N>;
    __shared__ int2 places[kMoveRows];
    wait_for_input();
    const uint32_t group = blockIdx.x / a.jobs_per_row, part = blockIdx.x % a.jobs_per_row;
    const uint32_t row0 = group * a.rows;
    const uint32_t rows = a.T - row0 < a.rows ? a.T - row0 : a.rows;
    const uint32_t D = a.g.D;
    const uint32_t first = part * (kMoveThreads * kMoveSlots) + threadIdx.x;
    L line[kMoveSlots];
    SlotOf at[kMoveSlots];
    auto row_line = [&](const SlotOf &s) {
        return (s.value ? a.v + (uint64_t)(row0 + s.row) * a.sv
                        : a.k + (uint64_t)(row0 + s.row) * a.sk) +
               (uint64_t)s.head * D * L::kSize;
    };
#pragma unroll
    for (int i = 0; i < kMoveSlots; ++i) {
        at[i] = slot_of(a, first + i * kMoveThreads, rows);
        if (!READ && at[i].on)
            line[i].load(row_line(at[i]), at[i].lane, a.lane_bits, D);
    }
    for (uint32_t r = threadIdx.x / 32; r < rows; r += kMoveThreads / 32) {
        const int2 at = a.g.place(a.offsets, a.B, row0 + r);
        if (threadIdx.x % 32 == 0)
            places[r] = at;
    }
    __syncthreads();
    constexpr int kCell = CACHE8 ? 1 : L::kSize;          // bytes of a cached element
    if constexpr (READ) {
        // all loads before the first use
        uint2 codes[CACHE8 && WIDE ? kMoveSlots * N : 1];
        uint32_t code[CACHE8 && !WIDE ? kMoveSlots * N : 1];
        float scale[kMoveSlots];
#pragma unroll
        for (int i = 0; i < kMoveSlots; ++i) {
            scale[i] = 0.0f;
            const int2 p = at[i].on ? places[at[i].row] : make_int2(-1, 0);
            at[i].on = p.x >= 0;
            if (!at[i].on)
                continue;
            const uint8_t *cells = (at[i].value ? a.g.v : a.g.k) + (uint64_t)p.x * a.g.stride +
                                   (uint64_t)a.g.in_page(at[i].head, p.y) * kCell;
            if (!CACHE8) {
                line[i].load(cells, at[i].lane, a.lane_bits, D);
                continue;
            }
            scale[i] = (at[i].value ? a.g.vs : a.g.ks)[a.g.scale_at(p.x, at[i].head, p.y)];
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const uint32_t e = L::at(at[i].lane, n, a.lane_bits);
                if (WIDE) {
                    uint2 &c = codes[(i * N + n) % (sizeof(codes) / sizeof(codes[0]))];
                    c = make_uint2(0u, 0u);
                    if (e < D) {
                        if (L::E == 8)
                            c = *reinterpret_cast<const uint2 *>(cells + e);
                        else
                            c.x = *reinterpret_cast<const uint32_t *>(cells + e);
                    }
                } else {
                    code[(i * N + n) % (sizeof(code) / sizeof(code[0]))] = e < D ? cells[e] : 0u;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kMoveSlots; ++i) {
            if (!at[i].on)
                continue;
            if (CACHE8) {
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    float v[8];
                    if (WIDE) {
                        const uint2 c = codes[(i * N + n) % (sizeof(codes) / sizeof(codes[0]))];
#pragma unroll
                        for (int e = 0; e < L::E; e += 2) {
                            const uint32_t w = e < 4 ? c.x : c.y;
                            const float2 f = from_e4m3x2((w >> (8 * (e & 2))) & 0xFFFFu);
                            v[e] = f.x * scale[i];
                            v[(e + 1) % 8] = f.y * scale[i];
                        }
                    } else {
                        v[0] = from_e4m3x2(code[(i * N + n) % (sizeof(code) / sizeof(code[0]))])
                                   .x * scale[i];
                    }
                    line[i].narrow(n, v);
                }
            }
            line[i].store(row_line(at[i]), at[i].lane, a.lane_bits, D);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kMoveSlots; ++i) {
            // lines of no row take part with nothing: a warp's lanes stay together
            const float top = CACHE8 ? largest(line[i], at[i].on, a.lane_bits) : 0.0f;
            const int2 p = at[i].on ? places[at[i].row] : make_int2(-1, 0);
            if (p.x < 0)
                continue;
            uint8_t *cells = (at[i].value ? a.g.v : a.g.k) + (uint64_t)p.x * a.g.stride +
                             (uint64_t)a.g.in_page(at[i].head, p.y) * kCell;
            if (!CACHE8) {
                line[i].store(cells, at[i].lane, a.lane_bits, D);
                continue;
            }
            // the quotients are products with rounded reciprocals, as in ar_rmsnorm
            const float scale = fmaxf(top, kCacheLeast) * (1.0f / kCacheTop);
            const float inv = __frcp_rn(scale);
            if (at[i].lane == 0)
                (at[i].value ? a.g.vs : a.g.ks)[a.g.scale_at(p.x, at[i].head, p.y)] = scale;
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const uint32_t e = L::at(at[i].lane, n, a.lane_bits);
                if (e >= D)
                    continue;
                float v[8];
                line[i].widen(n, v);
                if constexpr (WIDE) {
                    uint32_t q[2];
#pragma unroll
                    for (int x = 0; x < L::E; x += 4) {
                        float t[4] = {v[x], v[x + 1], v[x + 2], v[x + 3]};
                        mul2(t, inv, inv);
                        mul2(t + 2, inv, inv);
                        q[x / 4] = to_e4m3x4(t);
                    }
                    if (L::E == 8)
                        *reinterpret_cast<uint2 *>(cells + e) = make_uint2(q[0], q[L::E / 4 - 1]);
                    else
                        *reinterpret_cast<uint32_t *>(cells + e) = q[0];
                } else {
                    cells[e] = (uint8_t)to_e4m3x2(v[0] * inv, 0.0f);
                }
            }
        }
    }
}

template <int DT, bool WIDE, int N, bool CACHE8, bool READ>
static cudaError_t move_form(MoveArgs a, cudaStream_t s) {
    using L = Line<DT, WIDE, N>;
    constexpr uint32_t kJob = kMoveThreads * kMoveSlots;
    const uint32_t lanes = WIDE ? (a.g.D + L::E * N - 1) / (L::E * N) : 32;
    a.lane_bits = 0;
    while ((1u << a.lane_bits) < lanes)
        ++a.lane_bits;
    a.slots = 2u * a.g.heads << a.lane_bits;
    a.by_lines = divide_by(2u * a.g.heads);
    a.jobs_per_row = (a.slots + kJob - 1) / kJob;
    a.rows = 1;
    if (a.jobs_per_row == 1) {
        // rows of a job: what fills it, less where that leaves SMs without one
        const uint32_t fill = kJob / a.slots, sms = (uint32_t)sm_count();
        const uint32_t spread = sms ? (a.T + 2 * sms - 1) / (2 * sms) : 1;
        a.rows = fill < spread ? fill : spread;
        if (a.rows > kMoveRows)
            a.rows = kMoveRows;
        if (a.rows < 1)
            a.rows = 1;
    }
    const uint64_t grid = (uint64_t)((a.T + a.rows - 1) / a.rows) * a.jobs_per_row;
    if (grid >= 1ull << 31)
        return cudaErrorInvalidConfiguration;
    return launch_kernel(k_cache_move<DT, WIDE, N, CACHE8, READ>, (unsigned)grid, kMoveThreads, 0,
                         s, true, a);
}

template <int DT, bool READ>
static cudaError_t move_dt(const MoveArgs &a, bool w, bool e4m3, cudaStream_t s) {
    if (!w)
        return e4m3 ? move_form<DT, false, 8, true, READ>(a, s)
                    : move_form<DT, false, 8, false, READ>(a, s);
    // 32 bytes of codes and twice or four times that of rows a lane: with half of it, every
    // line's address, scale and shuffles are paid for by fewer bytes (65536 rows of 8 x 128
    // bf16 from 8 bits 77.7 us, to 8 bits 99; so 64.2 and 70.4)
    constexpr int N = Elem<DT>::kSize == 4 ? 4 : 2;
    return e4m3 ? move_form<DT, true, N, true, READ>(a, s)
                : move_form<DT, true, N, false, READ>(a, s);
}

template <bool READ>
static int move(const void *k, size_t ldk, const void *v, size_t ldv, const void *kcache,
                const void *vcache, size_t ldpage, const float *kscale, const float *vscale,
                size_t pages, int page, const int32_t *table, size_t ldtable, size_t width,
                const int32_t *lens, const int32_t *offsets, size_t T, size_t B, int heads, int D,
                int dtype, int cache_dtype, cudaStream_t stream) {
    MoveArgs a;
    const PagesCheck c = check_pages(kcache, vcache, ldpage, kscale, vscale, pages, page, table,
                                     ldtable, width, lens, B, heads, D, dtype, cache_dtype, &a.g);
    if (c.rc != AR_OK)
        return c.rc;
    if (T >= (size_t)1 << 31)
        return AR_ERR_UNSUPPORTED;
    if (!offsets && T != B)
        return AR_ERR_INVALID;
    if (T == 0)
        return AR_OK;
    if (!k || !v)
        return AR_ERR_INVALID;
    const size_t row = (size_t)heads * D, size = elem_size(dtype);
    const Matrix mk = matrix(k, ldk, T, row, size), mv = matrix(v, ldv, T, row, size);
    const Matrix mo = matrix(offsets, 0, 1, B + 1, 4);
    if (!mk.ok || !mv.ok || !mo.ok)
        return AR_ERR_INVALID;
    // the outputs: no other buffer on them
    const bool clash = c.on(mk) || c.on(mv) ||
                       (READ ? meet(mk, mv) || c.indexed(mk) || c.indexed(mv) || meet(mk, mo) ||
                                   meet(mv, mo)
                             : meet(c.k, c.v) || c.indexed(c.k) || c.indexed(c.v) ||
                                   c.indexed(c.ks) || c.indexed(c.vs) || c.on(mo) ||
                                   meet(c.ks, c.vs) || meet(c.k, c.ks) || meet(c.k, c.vs) ||
                                   meet(c.v, c.ks) || meet(c.v, c.vs));
    if (clash)
        return AR_ERR_INVALID;
    if (B == 0 || pages == 0)
        return AR_OK;                                    // no row has a place
    a.k = static_cast<uint8_t *>(const_cast<void *>(k));
    a.v = static_cast<uint8_t *>(const_cast<void *>(v));
    a.sk = mk.stride;
    a.sv = mv.stride;
    a.offsets = offsets;
    a.T = (uint32_t)T;
    a.B = (uint32_t)B;
    const bool e4m3 = cache_dtype == AR_E4M3;
    const size_t cell = e4m3 ? 16 / size : 16;           // bytes of a vector's cache cells
    const bool w = wide(mk) && wide(mv) && (size_t)D * size % 16 == 0 && wide(c.k, cell) &&
                   wide(c.v, cell);
    switch (dtype) {
    case AR_BF16: return launched(move_dt<AR_BF16, READ>(a, w, e4m3, stream));
    case AR_FP16: return launched(move_dt<AR_FP16, READ>(a, w, e4m3, stream));
    default: return launched(move_dt<AR_FP32, READ>(a, w, e4m3, stream));
    }
}

}  // namespace ar

using namespace ar;

extern "C" {

int ar_cache_write(const void *k, size_t ldk, const void *v, size_t ldv, void *kcache,
                   void *vcache, size_t ldpage, float *kscale, float *vscale, size_t pages,
                   int page, const int32_t *table, size_t ldtable, size_t width,
                   const int32_t *lens, const int32_t *offsets, size_t T, size_t B, int heads,
                   int D, int dtype, int cache_dtype, cudaStream_t stream) {
    return move<false>(k, ldk, v, ldv, kcache, vcache, ldpage, kscale, vscale, pages, page, table,
                       ldtable, width, lens, offsets, T, B, heads, D, dtype, cache_dtype, stream);
}

int ar_cache_read(const void *kcache, const void *vcache, size_t ldpage, const float *kscale,
                  const float *vscale, size_t pages, int page, const int32_t *table,
                  size_t ldtable, size_t width, const int32_t *lens, const int32_t *offsets,
                  void *k, size_t ldk, void *v, size_t ldv, size_t T, size_t B, int heads, int D,
                  int dtype, int cache_dtype, cudaStream_t stream) {
    return move<true>(k, ldk, v, ldv, kcache, vcache, ldpage, kscale, vscale, pages, page, table,
                      ldtable, width, lens, offsets, T, B, heads, D, dtype, cache_dtype, stream);
}

}  // extern "C"
