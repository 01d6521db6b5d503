// The paged cache of keys and values: its arguments, where a position lies, and
// the host-side checks that its calls share.
#pragma once

#include "ar_rows.cuh"

namespace ar {

// An E4M3 row's largest magnitude counts as at least this, so that neither its
// scale nor the scale's reciprocal leaves the range of normal numbers.
constexpr float kCacheLeast = 0x1p-96f;
constexpr float kCacheTop = 448.0f;

// n / d for n < 2^31 without a division: (n * mul) >> shift, exact for mul =
// ceil(2^shift / d) with shift = 31 + ceil(log2 d).
struct Divide {
    uint32_t mul, shift;
    __host__ __device__ __forceinline__ uint32_t operator()(uint32_t n) const {
        return (uint32_t)(((uint64_t)n * mul) >> shift);
    }
};
inline Divide divide_by(uint32_t d) {
    uint32_t bits = 0;
    while (bits < 31 && (1u << bits) < d)
        ++bits;
    Divide x;
    x.shift = 31 + bits;
    x.mul = (uint32_t)((((uint64_t)1 << x.shift) + d - 1) / d);
    return x;
}

struct Pages {
    uint8_t *k, *v;
    float *ks, *vs;               // scales, or NULL
    const int32_t *table;
    const int32_t *lens;
    uint64_t stride;              // bytes between pages
    uint64_t ldtable;
    uint32_t count, page, width;  // pages in the pool, slots of one, pages of a sequence
    uint32_t heads, D;
    Divide by_page;

    // tokens of sequence b
    __host__ __device__ __forceinline__ uint32_t length(uint32_t b) const {
        const int32_t n = lens[b];
        const uint32_t most = width * page;
        return n < 0 ? 0u : (uint32_t)n < most ? (uint32_t)n : most;
    }
    // the page of position j of sequence b, or -1
    __host__ __device__ __forceinline__ int32_t page_of(uint32_t b, uint32_t j) const {
        const int32_t p = table[(uint64_t)b * ldtable + by_page(j)];
        return (uint32_t)p < count ? p : -1;
    }
    __host__ __device__ __forceinline__ uint32_t slot_of(uint32_t j) const {
        return j - by_page(j) * page;
    }
    // elements before slot s of head h in its page; rows before it in the pool
    __host__ __device__ __forceinline__ uint32_t in_page(uint32_t h, uint32_t s) const {
        return (h * page + s) * D;
    }
    __host__ __device__ __forceinline__ uint64_t scale_at(int32_t p, uint32_t h, uint32_t s) const {
        return ((uint64_t)p * heads + h) * page + s;
    }
    // The place of row t of a call's rows: its page (-1: none) and slot.  On the device by
    // a whole warp, all lanes with one answer.
    __host__ __device__ __forceinline__ int2 place(const int32_t *offsets, uint32_t B,
                                                   uint32_t t) const {
        int2 none;
        none.x = -1;
        none.y = 0;
        uint32_t b = t;
        int64_t back = 1;                     // tokens from the row to the sequence's end
        if (offsets) {
            // the last b with offsets[b] <= t, 32 words at a time: one wait for memory up to
            // 32 sequences, two up to 1024
            uint32_t lo = 0, hi = B;
            while (hi - lo > 1) {
                const uint32_t step = (hi - lo + 31) / 32;
                const uint32_t n = count_up_to(offsets, lo, hi, step, t);
                lo += (n > 0 ? n - 1 : 0) * step;
                hi = hi - lo < step ? hi : lo + step;
            }
            b = lo;
            const int64_t end = offsets[b + 1];
            if ((int64_t)offsets[b] > (int64_t)t || end <= (int64_t)t)
                return none;
            back = end - t;
        }
        // a length past the table counts as the table's end, as in length()
        const int64_t j = (int64_t)length(b) - back;
        if (j < 0)
            return none;
        int2 at;
        at.x = page_of(b, (uint32_t)j);
        at.y = (int)slot_of((uint32_t)j);
        return at;
    }
    // How many of the words offsets[lo + i * step] below hi, i < 32, are at most t.
    static __host__ __device__ __forceinline__ uint32_t count_up_to(const int32_t *offsets,
                                                                    uint32_t lo, uint32_t hi,
                                                                    uint32_t step, uint32_t t) {
#ifdef __CUDA_ARCH__
        const uint32_t at = (threadIdx.x & 31) * step;
        const bool in = at < hi - lo && (int64_t)offsets[lo + at] <= (int64_t)t;
        return __popc(__ballot_sync(0xFFFFFFFFu, in));
#else
        uint32_t n = 0;
        for (uint32_t i = 0; i < 32 && i * step < hi - lo; ++i)
            n += (int64_t)offsets[lo + i * step] <= (int64_t)t;
        return n;
#endif
    }
};

// The wait of kernel_prologue() without its call for the next kernel, which then comes
// when the CTAs of this one have ended.  For kernels that a kernel follows whose CTAs
// fill an SM to the last register: placed between warps that are still there, fewer of
// them fit, and the others wait for a second turn.
__device__ __forceinline__ void wait_for_input() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ---- host side -----------------------------------------------------------------

// The buffers of a cache argument.
struct PagesCheck {
    Matrix k, v, ks, vs, table, lens;
    int rc = AR_OK;               // what the call has to return, if not AR_OK
    bool on(const Matrix &o) const {          // o meets a part of the cache
        return meet(o, k) || meet(o, v) || meet(o, ks) || meet(o, vs);
    }
    bool indexed(const Matrix &o) const { return meet(o, table) || meet(o, lens); }
};

inline PagesCheck check_pages(const void *kcache, const void *vcache, size_t ldpage,
                              const float *kscale, const float *vscale, size_t pages, int page,
                              const int32_t *table, size_t ldtable, size_t width,
                              const int32_t *lens, size_t B, int heads, int D, int dtype,
                              int cache_dtype, Pages *g) {
    PagesCheck c;
    const bool e4m3 = cache_dtype == AR_E4M3;
    c.rc = AR_ERR_INVALID;
    if (!float_dtype(dtype) || !(e4m3 || cache_dtype == dtype) || heads < 1 || D < 1 || page < 1 ||
        width < 1)
        return c;
    const size_t most = (size_t)1 << 31;
    if (D > AR_CACHE_MAX_DIM || heads > AR_CACHE_MAX_HEADS || pages >= most || B >= most ||
        width >= most || width * (size_t)page >= most ||
        // offsets inside a page are 32 bits
        (size_t)heads * page * D >= most) {
        c.rc = AR_ERR_UNSUPPORTED;
        return c;
    }
    const size_t size = e4m3 ? 1 : elem_size(dtype), row = (size_t)heads * page * D;
    c.k = matrix(kcache, ldpage, pages, row, size);
    c.v = matrix(vcache, ldpage, pages, row, size);
    c.ks = matrix(kscale, 0, pages, (size_t)heads * page, 4);
    c.vs = matrix(vscale, 0, pages, (size_t)heads * page, 4);
    c.table = matrix(table, ldtable ? ldtable : width, B, width, 4);
    c.lens = matrix(lens, 0, 1, B, 4);
    if (!c.k.ok || !c.v.ok || !c.ks.ok || !c.vs.ok || !c.table.ok || !c.lens.ok)
        return c;
    if (B > 0 && (!table || !lens || (pages > 0 && (!kcache || !vcache))))
        return c;
    if (B > 0 && pages > 0 && (e4m3 != (kscale != nullptr) || e4m3 != (vscale != nullptr)))
        return c;
    g->k = static_cast<uint8_t *>(const_cast<void *>(kcache));
    g->v = static_cast<uint8_t *>(const_cast<void *>(vcache));
    g->ks = const_cast<float *>(kscale);
    g->vs = const_cast<float *>(vscale);
    g->table = table;
    g->lens = lens;
    g->stride = c.k.stride;
    g->ldtable = ldtable ? ldtable : width;
    g->count = (uint32_t)pages;
    g->page = (uint32_t)page;
    g->by_page = divide_by((uint32_t)page);
    g->width = (uint32_t)width;
    g->heads = (uint32_t)heads;
    g->D = (uint32_t)D;
    c.rc = AR_OK;
    return c;
}

}  // namespace ar
