// Attention on the tensor cores, tiles dealt to CTAs in runs of one length.
#include "ar_cache_attention_mma.cuh"

namespace ar {

template <int DT, bool CACHE8, int DC, int HG>
static cudaError_t mma_form(AttnArgs &a, int *grid, cudaStream_t s) {
    using M = MmaForm<DT, CACHE8, DC, HG>;
    constexpr auto kernel = k_attention_mma<DT, CACHE8, DC, HG, false>;
    const int sms = sm_count();
    if (sms < 1)
        return cudaErrorUnknown;
    a.unit_rows = M::kHeads;
    a.head_tiles = (a.group + M::kHeads - 1) / M::kHeads;
    a.runs = a.g.page % 16 == 0;
    if (attention_units(a, M::kCtas * sms)) {
        *grid = 0;
        return launch_attention_units(a, DT, CACHE8, s);
    }
    const cudaError_t e = opt_in_smem<kernel>(M::kSmem);
    if (e != cudaSuccess)
        return e;
    *grid = cta_limit(a.unit_rows, M::kCtas * sms);
    return launch_kernel(kernel, *grid, M::kThreads, M::kSmem, s, true, a);
}

template <int DT, bool CACHE8, int DC>
static cudaError_t mma_heads(AttnArgs &a, int *grid, cudaStream_t s) {
    return a.group <= 8    ? mma_form<DT, CACHE8, DC, 1>(a, grid, s)
           : a.group <= 16 ? mma_form<DT, CACHE8, DC, 2>(a, grid, s)
                           : mma_form<DT, CACHE8, DC, 4>(a, grid, s);
}

template <int DT, bool CACHE8>
static cudaError_t mma_dim(AttnArgs &a, int *grid, cudaStream_t s) {
    return a.g.D <= 64    ? mma_heads<DT, CACHE8, 64>(a, grid, s)
           : a.g.D <= 128 ? mma_heads<DT, CACHE8, 128>(a, grid, s)
                          : mma_heads<DT, CACHE8, 256>(a, grid, s);
}

cudaError_t launch_attention_mma(AttnArgs &a, int dtype, bool e4m3, int *grid, cudaStream_t s) {
    if (dtype == AR_FP32)
        return mma_dim<AR_FP32, true>(a, grid, s);
    if (dtype == AR_BF16)
        return e4m3 ? mma_dim<AR_BF16, true>(a, grid, s) : mma_dim<AR_BF16, false>(a, grid, s);
    return e4m3 ? mma_dim<AR_FP16, true>(a, grid, s) : mma_dim<AR_FP16, false>(a, grid, s);
}

}  // namespace ar
