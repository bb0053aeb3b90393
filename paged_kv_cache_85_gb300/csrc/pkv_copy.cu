// copy_blocks: block `dst` of every tensor becomes block `src`, for each pair of a list.
//
// The tensors are what lies under the cache's block ids (caches, scales, recorded
// weights, of one layer or of many), so a block's pieces are large runs of bytes (32 KB
// for 16 bf16 tokens of 8 heads) next to tiny ones (32 B of scales).  A warp therefore
// takes a piece of 4 KB, sixteen-byte loads, eight of them in flight per lane; a tiny
// piece costs one warp's turn, not a CTA's.  Bound by HBM (read and write): 4000 blocks of
// 16 bf16 tokens of 8 heads, K and V of two layers (1.05 GB in all), 158 us, 6.6 TB/s, 0.98
// of the measured copy; the last blocks of eight forks in eight tensors 3.6 us.
#include "pkv_kernels.h"
#include "pkv_ptx.cuh"
#include "pkv_scaled.h"

namespace pkv {

constexpr int kCopyThreads = 256;

template <typename V>
__device__ __forceinline__ void copy_piece(uint8_t *dst, const uint8_t *src, int bytes, int lane)
{
    constexpr int IN = 8;  // loads in flight per lane
    V *d = reinterpret_cast<V *>(dst);
    const V *s = reinterpret_cast<const V *>(src);
    const int n = bytes / (int)sizeof(V);
    for (int i0 = lane; i0 < n; i0 += 32 * IN) {
        V v[IN];
#pragma unroll
        for (int k = 0; k < IN; k++)
            if (i0 + 32 * k < n)
                v[k] = s[i0 + 32 * k];
#pragma unroll
        for (int k = 0; k < IN; k++)
            if (i0 + 32 * k < n)
                d[i0 + 32 * k] = v[k];
    }
}

__global__ void __launch_bounds__(kCopyThreads) copy_blocks_kernel(const __grid_constant__ CopyParams p)
{
    grid_launch_dependents();
    grid_dependency_wait();  // what is copied may have just been written
    const int lane = threadIdx.x & 31;
    const long long warps = (long long)gridDim.x * (kCopyThreads / 32);
    const long long units = (long long)p.n * p.chunks;
    for (long long u = (long long)blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5); u < units; u += warps) {
        const int i = (int)(u / p.chunks);
        int c = (int)(u - (long long)i * p.chunks);
        const int2 pair = p.pairs[i];
        const bool in = pair.x >= 0 && pair.x < p.NB && pair.y >= 0 && pair.y < p.NB;
        if (!in || pair.x == pair.y) {
            if (!in && (pair.x != -1 || pair.y != -1) && c == 0 && lane == 0)
                flag_error(p.err_flag, 0x2 /* PKV_FLAG_BAD_BLOCK */);
            continue;
        }
        int t = 0;
        while (c >= p.t[t].chunks)
            c -= p.t[t++].chunks;
        const CopyTensor &x = p.t[t];
        const long long at = (long long)c * kCopyChunk;
        const int bytes = (int)min((long long)kCopyChunk, x.block_bytes - at);
        const uint8_t *src = x.base + pair.x * x.block_bytes + at;
        uint8_t *dst = x.base + pair.y * x.block_bytes + at;
        if (x.vec == 16)
            copy_piece<uint4>(dst, src, bytes, lane);
        else if (x.vec == 4)
            copy_piece<uint32_t>(dst, src, bytes, lane);
        else
            copy_piece<uint8_t>(dst, src, bytes, lane);
    }
}

cudaError_t launch_copy_blocks(const CopyParams &p, int sms, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    constexpr int W = kCopyThreads / 32;
    const long long need = ((long long)p.n * p.chunks + W - 1) / W, most = 8LL * sms;
    cfg.gridDim = dim3((unsigned)(need < most ? need : most));
    cfg.blockDim = dim3(kCopyThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, copy_blocks_kernel, p);
}

} // namespace pkv
