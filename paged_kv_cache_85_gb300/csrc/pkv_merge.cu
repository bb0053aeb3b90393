// The kernel that merges the pieces of split streams (pkv_merge.cuh), one warp
// per (sequence, query head).
#include "pkv_merge.cuh"

namespace pkv {

template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32) merge_pieces_kernel(const DecodeParams p)
{
    grid_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * kMergeWarps + warp;
    if (row >= (long long)p.B * p.Hq)
        return;
    merge_row<D>(p, row, lane);
}

cudaError_t launch_merge(int D, int G, const DecodeParams &p, cudaStream_t stream)
{
    (void)G;
    const long long rows = (long long)p.B * p.Hq;
    if (rows == 0)
        return cudaSuccess;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)((rows + kMergeWarps - 1) / kMergeWarps));
    cfg.blockDim = dim3(kMergeWarps * 32);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (D == 128)
        return cudaLaunchKernelEx(&cfg, merge_pieces_kernel<128>, p);
    if (D == 64)
        return cudaLaunchKernelEx(&cfg, merge_pieces_kernel<64>, p);
    return cudaErrorInvalidValue;
}

} // namespace pkv
