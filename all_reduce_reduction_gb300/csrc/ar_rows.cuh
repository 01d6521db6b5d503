// Rows of a matrix, read and written by threads in units.
//
// A row of H elements is cut into units, one thread's share of it.  In the
// wide form a unit is one 16-byte vector (the row's address is a multiple of
// 16; the last unit may be short and is then accessed element by element).
// In the general form a unit is four elements, lane l of a warp holding
// elements l, l + 32, l + 64 and l + 96 of the warp's 128, so that each access
// of the warp is one contiguous run whatever the alignment.  Either way the
// units of 128 consecutive elements belong to consecutive lanes of one warp,
// kBlockLanes of them, which lets a block that shares a scale be reduced by
// shuffles alone.
#pragma once

#include <atomic>

#include "ar_device.cuh"

namespace ar {

// Two elements of a two-byte type in one word, and back.
template <int DT> __device__ __forceinline__ float2 widen2(uint32_t w) {
    if (DT == AR_BF16)
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
template <int DT> __device__ __forceinline__ uint32_t narrow2(float lo, float hi) {
    if (DT == AR_BF16) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&p);
    }
    const __half2 p = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}

template <int DT, bool WIDE> struct Rows {
    static constexpr int kSize = Elem<DT>::kSize;
    static constexpr int E = WIDE ? 16 / kSize : 4;               // elements per unit
    static constexpr int kBlockLanes = AR_SCALE_BLOCK / E;        // units per scale block
    static constexpr bool kPairs = WIDE && kSize == 2;            // two elements a word
    static_assert(kBlockLanes <= 32, "a scale block is at most one warp");

    // units that cover a row of H < 2^31 elements: whole scale blocks in the
    // general form, whose units interleave within 128 elements
    static __host__ __device__ __forceinline__ uint32_t units(uint32_t H) {
        return WIDE ? (H + E - 1) / E : (H + 127) / 128 * 32;
    }
    // the same, up to a whole number of warps
    static __host__ __device__ __forceinline__ uint32_t warp_units(uint32_t H) {
        return (units(H) + 31) / 32 * 32;
    }
    // element i of unit u
    static __device__ __forceinline__ uint32_t at(uint32_t u, int i) {
        return WIDE ? u * E + i : u / 32 * 128 + u % 32 + 32 * i;
    }
    static __device__ __forceinline__ bool whole(uint32_t u, uint32_t H) {
        return WIDE && u * E + E <= H;
    }
    // The unit's bits: words of packed elements (wide) or one element a word.
    // Elements past H read as zero.  REUSED data may stay in L1.
    template <bool REUSED = false>
    static __device__ __forceinline__ uint4 load(const void *row, uint32_t u, uint32_t H) {
        if (whole(u, H)) {
            const uint4 *p = reinterpret_cast<const uint4 *>(row) + u;
            return REUSED ? ld_v4_l1(p) : ld_v4_stream(p);
        }
        uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (at(u, i) < H) {
                const uint32_t b = ld_elem<DT>(row, at(u, i));
                if (kPairs)
                    w[i / 2] |= b << (16 * (i & 1));
                else
                    w[i & 3] = b;
            }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    // The same where `on` is true, zeros elsewhere.  The wide load is predicated,
    // not branched around, so that a run of them is issued without a wait.
    static __device__ __forceinline__ uint4 load_if(bool on, const void *row, uint32_t u,
                                                    uint32_t H) {
        if (!whole(u, H))
            return on ? load(row, u, H) : make_uint4(0u, 0u, 0u, 0u);
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t"
            "@p ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
            : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)
            : "l"(reinterpret_cast<const uint4 *>(row) + u), "r"((uint32_t)on));
        return v;
    }
    static __device__ __forceinline__ void widen(uint4 p, float v[E]) {
        const uint32_t w[4] = {p.x, p.y, p.z, p.w};
        if (kPairs) {
#pragma unroll
            for (int i = 0; i < E; i += 2) {
                const float2 f = widen2<DT>(w[i / 2]);
                v[i] = f.x;
                v[i + (E > 1)] = f.y;
            }
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i)
                v[i] = widen1<DT>(w[i & 3]);
        }
    }
    static __device__ __forceinline__ void store(void *row, uint32_t u, uint32_t H,
                                                 const float v[E]) {
        uint32_t w[4] = {0u, 0u, 0u, 0u};
        if (kPairs) {
#pragma unroll
            for (int i = 0; i < E; i += 2)
                w[i / 2] = narrow2<DT>(v[i], v[i + (E > 1)]);
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i)
                w[i & 3] = narrow1<DT>(v[i]);
        }
        if (whole(u, H)) {
            st_v4(reinterpret_cast<uint4 *>(row) + u, make_uint4(w[0], w[1], w[2], w[3]));
            return;
        }
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (at(u, i) < H)
                st_elem<DT>(row, at(u, i),
                            kPairs ? (w[i / 2] >> (16 * (i & 1))) & 0xFFFFu : w[i & 3]);
    }
};

// Two binary32 operations in one instruction, each rounded to nearest even on
// its own: x = x + y, x = x * y, x = a * b + x.
__device__ __forceinline__ void add2(float *x, float y0, float y1) {
    asm("{\n\t.reg .b64 t, u;\n\tmov.b64 t, {%2, %3};\n\tmov.b64 u, {%0, %1};\n\t"
        "add.rn.f32x2 u, u, t;\n\tmov.b64 {%0, %1}, u;\n\t}"
        : "+f"(x[0]), "+f"(x[1]) : "f"(y0), "f"(y1));
}
__device__ __forceinline__ void mul2(float *x, float y0, float y1) {
    asm("{\n\t.reg .b64 t, u;\n\tmov.b64 t, {%2, %3};\n\tmov.b64 u, {%0, %1};\n\t"
        "mul.rn.f32x2 u, u, t;\n\tmov.b64 {%0, %1}, u;\n\t}"
        : "+f"(x[0]), "+f"(x[1]) : "f"(y0), "f"(y1));
}
__device__ __forceinline__ void fma2(float *x, float a0, float a1, float b0, float b1) {
    asm("{\n\t.reg .b64 s, t, u;\n\t"
        "mov.b64 s, {%2, %3};\n\tmov.b64 t, {%4, %5};\n\tmov.b64 u, {%0, %1};\n\t"
        "fma.rn.f32x2 u, s, t, u;\n\tmov.b64 {%0, %1}, u;\n\t}"
        : "+f"(x[0]), "+f"(x[1]) : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    return v;
}

// Rows of a CTA at a time.
//   kOneRow:  the whole CTA works on a row.
//   kWarpRow: every warp on its own.
//   kGroups:  `warps` warps on each, groups of them side by side; the warps past
//             the last whole group have g == groups() and no row.
enum RowSplit { kOneRow, kWarpRow, kGroups };
template <RowSplit SPLIT> struct RowGroup {
    int warps_;
    __device__ __forceinline__ explicit RowGroup(int warps) : warps_(warps) {}
    __device__ __forceinline__ int warps() const {
        return SPLIT == kOneRow ? (int)(blockDim.x >> 5) : SPLIT == kWarpRow ? 1 : warps_;
    }
    __device__ __forceinline__ int groups() const {
        return SPLIT == kOneRow ? 1 : (int)(blockDim.x >> 5) / warps();
    }
    __device__ __forceinline__ int g() const {
        if (SPLIT == kOneRow)
            return 0;
        const int g = (int)(threadIdx.x >> 5) / warps();
        return g < groups() ? g : groups();
    }
    // this thread's place in its group, and the group's threads
    __device__ __forceinline__ uint32_t thread() const {
        return SPLIT == kOneRow    ? threadIdx.x
               : SPLIT == kWarpRow ? threadIdx.x & 31
                                   : threadIdx.x - (uint32_t)(g() * warps()) * 32;
    }
    __device__ __forceinline__ uint32_t threads() const {
        return SPLIT == kOneRow ? blockDim.x : (uint32_t)warps() * 32;
    }
    // Sum over the group, the same in each of its threads.  Called by the
    // whole CTA; `part` is shared memory of 32 floats, free again after the
    // CTA's next barrier.
    __device__ __forceinline__ float sum(float v, float *part) const {
        v = warp_sum(v);
        if (SPLIT == kWarpRow || warps() == 1)
            return v;
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        if (lane == 0)
            part[warp] = v;
        __syncthreads();
        return warp_sum(lane < warps() && g() < groups() ? part[g() * warps() + lane] : 0.0f);
    }
};

// ---- host-side checks ------------------------------------------------------

// A row-major matrix argument: its address, bytes between and in its rows, and
// bytes from its first to past its last element.
struct Matrix {
    uintptr_t p = 0;
    size_t rows = 0;
    size_t stride = 0;       // bytes between rows
    size_t width = 0;        // bytes of a row
    size_t bytes = 0;
    bool ok = true;
};

// ld = 0 stands for rows without gaps.  ok is false for a misaligned address,
// a leading dimension below the row, or a size past 2^62 bytes.
inline Matrix matrix(const void *p, size_t ld, size_t rows, size_t cols, size_t esz) {
    Matrix m;
    if (ld == 0)
        ld = cols;
    m.p = (uintptr_t)p;
    m.rows = rows;
    const size_t limit = (size_t)1 << 62;
    m.ok = m.p % esz == 0 && ld >= cols && ld <= limit / esz &&
           (rows == 0 || ld * esz <= limit / rows);
    if (m.ok) {
        m.stride = ld * esz;
        m.width = cols * esz;
        m.bytes = rows == 0 || cols == 0 ? 0 : (rows - 1) * m.stride + m.width;
    }
    return m;
}
// Whether the two share a byte.  Rows of one stride that lie in the gaps of the
// other's (column slices of one wider buffer) do not; for rows of different
// strides the answer is that of the whole ranges.
inline bool meet(const Matrix &a, const Matrix &b) {
    if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0 || a.p >= b.p + b.bytes ||
        b.p >= a.p + a.bytes)
        return false;
    const bool strided_a = a.rows > 1, strided_b = b.rows > 1;
    if (strided_a == strided_b && (!strided_a || a.stride != b.stride))
        return true;
    const size_t stride = strided_a ? a.stride : b.stride;
    // where rows of b start in those of a
    const size_t at = b.p >= a.p ? (b.p - a.p) % stride : (stride - (a.p - b.p) % stride) % stride;
    return at < a.width || at + b.width > stride;
}
// The same rows, for matrices of as many rows of one length.
inline bool same(const Matrix &a, const Matrix &b) {
    return a.p == b.p && (a.stride == b.stride || a.rows <= 1);
}
// the output o meets the input i otherwise than exactly
inline bool clash(const Matrix &o, const Matrix &i) { return meet(o, i) && !same(o, i); }
inline bool wide(const Matrix &m, size_t align = 16) {
    return m.p % align == 0 && m.stride % align == 0;
}

inline bool float_dtype(int d) { return d == AR_BF16 || d == AR_FP16 || d == AR_FP32; }

// SMs of the current device (asked once per device); 0 if it does not answer.
inline int sm_count() {
    static std::atomic<int> known[64];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0)
        return 0;
    if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0)
        return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    if (dev < 64)
        known[dev].store(n, std::memory_order_relaxed);
    return n;
}

// Opts a kernel in to `bytes` of dynamic shared memory, once per kernel and
// device: asking the runtime every time costs a launch 0.5 us.
template <auto KERNEL> inline cudaError_t opt_in_smem(size_t bytes) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
    if (done.load(std::memory_order_acquire) & bit)
        return cudaSuccess;
    e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess)
        done.fetch_or(bit, std::memory_order_release);
    return e;
}

// The launch's result as a status code.
inline int launched(cudaError_t e) {
    if (e == cudaSuccess)
        return AR_OK;
    (void)cudaGetLastError();
    return AR_ERR_CUDA;
}

}  // namespace ar
