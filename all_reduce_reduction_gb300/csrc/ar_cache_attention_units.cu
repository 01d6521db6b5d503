// Attention on the tensor cores for few units of few tiles: each has a CTA, or a cluster
// that joins its shares through its shared memory, in one launch (one sequence of 500
// positions: 5.8 us; dealt and joined by a second launch, as under a table with room for more
// than 4096 of them, 8.6).
#include "ar_cache_attention_mma.cuh"

namespace ar {

bool attention_units(AttnArgs &a, int room) {
    // tiles of a unit, as far as the host knows
    uint64_t most = (uint64_t)a.g.width * a.g.page;
    if (a.window && most > a.window)
        most = (uint64_t)a.window + 15;
    most = (most + kMmaTile - 1) / kMmaTile;
    const uint64_t units = (uint64_t)a.B * a.g.heads * a.head_tiles;
    uint32_t parts = 1;
    while (parts < kMaxParts && 2 * parts <= most && units * 2 * parts <= (uint64_t)room)
        parts *= 2;
    // up to eight tiles a CTA, or as much one CTA after the other
    a.cluster = units <= (uint64_t)room                                  ? (most <= 8 * parts ? parts : 0)
                : units <= 4ull * room && units * most <= 8ull * room ? 1
                                                                       : 0;
    return a.cluster > 0;
}

template <int DT, bool CACHE8, int DC, int HG>
static cudaError_t mma_form(const AttnArgs &a, cudaStream_t s) {
    using M = MmaForm<DT, CACHE8, DC, HG>;
    constexpr auto kernel = k_attention_mma<DT, CACHE8, DC, HG, true>;
    const cudaError_t e = opt_in_smem<kernel>(M::kSmem);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = (unsigned)(a.B * a.g.heads * a.head_tiles * a.cluster);
    cfg.blockDim = M::kThreads;
    cfg.dynamicSmemBytes = M::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int DT, bool CACHE8, int DC>
static cudaError_t mma_heads(const AttnArgs &a, cudaStream_t s) {
    return a.group <= 8    ? mma_form<DT, CACHE8, DC, 1>(a, s)
           : a.group <= 16 ? mma_form<DT, CACHE8, DC, 2>(a, s)
                           : mma_form<DT, CACHE8, DC, 4>(a, s);
}

template <int DT, bool CACHE8>
static cudaError_t mma_dim(const AttnArgs &a, cudaStream_t s) {
    return a.g.D <= 64    ? mma_heads<DT, CACHE8, 64>(a, s)
           : a.g.D <= 128 ? mma_heads<DT, CACHE8, 128>(a, s)
                          : mma_heads<DT, CACHE8, 256>(a, s);
}

cudaError_t launch_attention_units(const AttnArgs &a, int dtype, bool e4m3, cudaStream_t s) {
    if (dtype == AR_FP32)
        return mma_dim<AR_FP32, true>(a, s);
    if (dtype == AR_BF16)
        return e4m3 ? mma_dim<AR_BF16, true>(a, s) : mma_dim<AR_BF16, false>(a, s);
    return e4m3 ? mma_dim<AR_FP16, true>(a, s) : mma_dim<AR_FP16, false>(a, s);
}

}  // namespace ar
