// Attention weights of a decode step, added to the cache's weight table.
//
// The decode kernel left, per box of a stream, the scores s[g][t] (log2
// units) of its tokens for the G query heads of the group, and, per (sequence,
// query head), the log-sum-exp lse of all its scores (the merge kernel for
// streams split over workers).  A token's weight in this step is the sum of
// its G softmax values,
//     w = sum_g 2^(s[g][t] - lse[g]),
// added to weights[block, kv head, offset], or stored there for the step's
// newest token, whose slot may hold what an earlier owner of the block left.
//
// One thread per four tokens of a box (16-byte loads of the scores and one
// 16-byte addition to the weights, which lie next to each other in a block).
// Every (token, KV head) gets exactly one addition per call, so the sums do not
// depend on the order of the threads; they are atomic because two sequences of
// a batch may share a prefix block (then their two additions may come in either
// order).
#include "pkv_kernels.h"
#include "pkv_ptx.cuh"

namespace pkv {

constexpr int kAddThreads = 256;

template <int G, int BT>
__global__ void __launch_bounds__(kAddThreads)
    add_weights_kernel(const DecodeParams p, float *__restrict__ weights)
{
    constexpr int kQuads = BT / 4;  // threads per box
    // scores, descriptors and log-sum-exps come from the kernels just before
    grid_dependency_wait();
    const int per_head = p.ws_hdr[kWsHeaderInts + p.B];  // boxes per KV head
    const long long n = (long long)per_head * p.Hkv * kQuads;
    for (long long idx = (long long)blockIdx.x * kAddThreads + threadIdx.x; idx < n;
         idx += (long long)gridDim.x * kAddThreads) {
        const int box = (int)(idx / kQuads), i = (int)(idx % kQuads) * 4;
        const int4 m = p.ws_box[box];
        float4 s[G];
        const float *sc = p.ws_score + (size_t)box * G * BT + i;
#pragma unroll
        for (int g = 0; g < G; g++)
            s[g] = *reinterpret_cast<const float4 *>(sc + g * BT);
        const int nvalid = m.w & (kBoxNewest - 1);
        if (m.y < 0 || i >= nvalid)
            continue;
        const int h = box / per_head;
        const float *lse = p.ws_lse + (size_t)m.x * p.Hq + (size_t)h * G;
        float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int g = 0; g < G; g++) {
            const float l = lse[g];
            w.x += fast_exp2(s[g].x - l);
            w.y += fast_exp2(s[g].y - l);
            w.z += fast_exp2(s[g].z - l);
            w.w += fast_exp2(s[g].w - l);
        }
        float *dst = weights + ((size_t)m.y * p.Hkv + h) * p.bs + m.z + i;
        const bool newest = (m.w & kBoxNewest) != 0;
        if (i + 4 <= nvalid - (newest ? 1 : 0)) {
            atomicAdd(reinterpret_cast<float4 *>(dst), w);
        } else {  // the context's last tokens: none past it, and the newest one is set
            const float x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int k = 0; k < 4; k++) {
                if (newest && i + k == nvalid - 1)
                    dst[k] = x[k];
                else if (i + k < nvalid)
                    atomicAdd(dst + k, x[k]);
            }
        }
    }
}

cudaError_t launch_add_weights(int G, int bt, const DecodeParams &p, float *weights, long long max_boxes,
                               int sms, cudaStream_t stream)
{
    const long long need = (max_boxes * (bt / 4) + kAddThreads - 1) / kAddThreads;
    const long long most = (long long)sms * (2048 / kAddThreads);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)(need < most ? need : most));
    cfg.blockDim = dim3(kAddThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
#define PKV_ADD(GG)                                                                               \
    case GG:                                                                                      \
        return bt == 2 * kBox ? cudaLaunchKernelEx(&cfg, add_weights_kernel<GG, 2 * kBox>, p, weights) \
                              : cudaLaunchKernelEx(&cfg, add_weights_kernel<GG, kBox>, p, weights);
    switch (G) {
        PKV_ADD(1)
        PKV_ADD(2)
        PKV_ADD(4)
        PKV_ADD(8)
    default: return cudaErrorInvalidValue;
    }
#undef PKV_ADD
}

} // namespace pkv
