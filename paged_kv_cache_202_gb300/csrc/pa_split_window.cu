// Split paged decode with a sliding window and sinks (pa_decode_window): the
// kernels of pa_split.cu over the pages that hold a visible token (split_body's
// WIN), for the few segments so long that a cluster each (pa_window_decode.cu)
// would leave SMs idle for many rounds.
//
// The visible pages of all sequences form one page stream, which every warp of
// the grid takes an equal part of; the partial results go through memory and a
// merge kernel. That second kernel and the finding of a warp's place in the
// stream cost about 4 us, and for long windows the even split of the stream over
// all SMs is worth more: one sequence, one kv head, W = 32768, 17.4 us against
// 27.7 in a cluster of 8 blocks, W = 65536, 22.3 against 46.4. (The calls that
// come here are chosen in pa_api.cu.)
#include "pa_split.cuh"

namespace pa {
namespace split {

template <int D, int BS, int NT>
__global__ void __launch_bounds__(NT == 2 ? 32 * kQsMaxWarps : 256, 1)
    mma_window_kernel(const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap, const SplitWindowArgs a) {
    split_body<D, BS, MmaState<D, kChunkTokens, NT, NT == 2>, false, false, false, true>(&kmap, &vmap, a);
}

using WindowFn = void (*)(CUtensorMap, CUtensorMap, SplitWindowArgs);

WindowFn select_window(const SplitLaunch& L) {
    if (L.kind != kSplitMma || L.mq || L.fused || L.append || (L.NT != 1 && L.NT != 2)) return nullptr;
    if (L.D == 128 && L.BS == 16) return L.NT == 1 ? mma_window_kernel<128, 16, 1> : mma_window_kernel<128, 16, 2>;
    if (L.D == 128 && L.BS == 32) return L.NT == 1 ? mma_window_kernel<128, 32, 1> : mma_window_kernel<128, 32, 2>;
    if (L.D == 64 && L.BS == 16) return L.NT == 1 ? mma_window_kernel<64, 16, 1> : mma_window_kernel<64, 16, 2>;
    if (L.D == 64 && L.BS == 32) return L.NT == 1 ? mma_window_kernel<64, 32, 1> : mma_window_kernel<64, 32, 2>;
    return nullptr;
}

}  // namespace split

int split_window_blocks_per_sm(const SplitLaunch& L, cudaError_t* status) {
    split::WindowFn fn = split::select_window(L);
    int n = 0;
    // For every call in the process, whatever its size (as in pa_split.cu).
    *status = fn ? cudaFuncSetAttribute(reinterpret_cast<const void*>(fn),
                                        cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        static_cast<int>(kScanSmemLimit))
                 : cudaErrorInvalidValue;
    if (*status == cudaSuccess)
        *status = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, reinterpret_cast<const void*>(fn),
                                                                L.warps * 32, L.smem);
    return *status == cudaSuccess ? n : 0;
}

cudaError_t launch_split_window(const SplitLaunch& L, const CUtensorMap& kmap,
                                const CUtensorMap& vmap, const SplitWindowArgs& a,
                                cudaStream_t stream) {
    split::WindowFn fn = split::select_window(L);
    if (!fn) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(L.blocks);
    cfg.blockDim = dim3(L.warps * 32);
    cfg.dynamicSmemBytes = L.smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, kmap, vmap, a);
}

}  // namespace pa
