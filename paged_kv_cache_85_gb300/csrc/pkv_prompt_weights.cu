// Attention weights of a prefill step, added to the cache's weight table.
//
// The prefill kernel left every (new token, query head)'s log-sum-exp lse of
// its scores (log2 units).  The weight that token t of a sequence received
// from the observing queries is
//     w[t] = sum over observing new tokens i that see t, and over the G heads
//            of the group, of 2^(s[i, g, t] - lse[i, g]),
// which needs the final lse of every row, so the scores are made again here.
// It is added to weights[block, kv head, offset], or stored there for the
// step's new tokens, whose slots may hold what an earlier owner left.
//
// One thread per cached token: its K row stays in registers and the query rows
// pass by in shared memory.
#include "pkv_kernels.h"
#include "pkv_prefill.h"
#include "pkv_ptx.cuh"

namespace pkv {

constexpr int kPwTokens = 128;  // tokens (threads) per CTA
constexpr int kPwRows = 32;     // (new token, head) rows in shared memory at a time

template <int D>
__global__ void __launch_bounds__(kPwTokens)
    prompt_weights_kernel(const PrefillParams p, const uint16_t *k_cache, float *weights, int window)
{
    __shared__ __align__(16) float sq[kPwRows][D];
    __shared__ float slse[kPwRows];
    grid_dependency_wait();
    const int b = blockIdx.z, h = blockIdx.y, tid = threadIdx.x;
    const int G = p.Hq / p.Hkv;
    const int cq0 = p.cu_q[b], cq1 = p.cu_q[b + 1], ck0 = p.cu_k[b], ck1 = p.cu_k[b + 1];
    const int q_len = cq1 - cq0, k_len = ck1 - ck0, base = k_len - q_len;
    if (cq0 < 0 || q_len < 0 || (long long)cq1 > p.Tq || k_len < q_len ||
        (long long)k_len > (long long)p.MBS * p.bs || q_len > p.max_q)
        return;  // skipped by the attention as well, which reports it
    const int t0 = blockIdx.x * kPwTokens, t = t0 + tid;
    if (q_len == 0 || t0 >= k_len)
        return;
    int blk = -1, off = 0;
    if (t < k_len) {
        blk = p.block_tables[(size_t)b * p.MBS + t / p.bs];
        off = t % p.bs;
        if (blk < 0 || blk >= p.NB)
            blk = -1;
    }
    uint32_t kr[D / 2];
#pragma unroll
    for (int i = 0; i < D / 2; i++)
        kr[i] = 0;
    if (blk >= 0) {
        const uint4 *src = reinterpret_cast<const uint4 *>(
            k_cache + (((size_t)blk * p.bs + off) * p.Hkv + h) * D);
#pragma unroll
        for (int i = 0; i < D / 8; i++) {
            const uint4 x = src[i];
            kr[4 * i] = x.x;
            kr[4 * i + 1] = x.y;
            kr[4 * i + 2] = x.z;
            kr[4 * i + 3] = x.w;
        }
    }
    const float sl = p.neg_scale ? -p.scale_log2 : p.scale_log2;
    int i0 = max(0, t0 - base);  // first new token that sees any of these tokens
    if (window > 0)
        i0 = max(i0, q_len - window);
    float w = 0.f;
    for (int r0 = i0 * G; r0 < q_len * G; r0 += kPwRows) {
        const int nr = min(kPwRows, q_len * G - r0);
        __syncthreads();
        for (int e = tid; e < nr * (D / 2); e += kPwTokens) {
            const int r = e / (D / 2), c = e % (D / 2);
            const int i = (r0 + r) / G, g = (r0 + r) % G;
            const uint32_t x = reinterpret_cast<const uint32_t *>(
                p.q + ((size_t)(cq0 + i) * p.Hq + (size_t)h * G + g) * D)[c];
            const float2 f = bf16x2_to_float2(x);
            sq[r][2 * c] = f.x;
            sq[r][2 * c + 1] = f.y;
        }
        if (tid < nr) {
            const int i = (r0 + tid) / G, g = (r0 + tid) % G;
            slse[tid] = p.lse[((size_t)h * p.Tq + cq0 + i) * G + g];
        }
        __syncthreads();
        for (int r = 0; r < nr; r++) {
            if (t > base + (r0 + r) / G)
                continue;  // that query does not see this token
            float s = 0.f;
#pragma unroll
            for (int c = 0; c < D / 4; c++) {
                const float4 x = *reinterpret_cast<const float4 *>(&sq[r][4 * c]);
                const float2 k0 = bf16x2_to_float2(kr[2 * c]), k1 = bf16x2_to_float2(kr[2 * c + 1]);
                s = fmaf(x.x, k0.x, s);
                s = fmaf(x.y, k0.y, s);
                s = fmaf(x.z, k1.x, s);
                s = fmaf(x.w, k1.y, s);
            }
            w += fast_exp2(fmaf(s, sl, -slse[r]));
        }
    }
    if (blk >= 0) {
        float *dst = weights + ((size_t)blk * p.Hkv + h) * p.bs + off;
        if (t >= base)
            *dst = w;
        else
            atomicAdd(dst, w);
    }
}

cudaError_t launch_prompt_weights(int D, const PrefillParams &p, const void *k_cache, float *weights,
                                  int window, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)(((long long)p.MBS * p.bs + kPwTokens - 1) / kPwTokens),
                       (unsigned)p.Hkv, (unsigned)p.B);
    cfg.blockDim = dim3(kPwTokens);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const uint16_t *k = static_cast<const uint16_t *>(k_cache);
    return D == 128 ? cudaLaunchKernelEx(&cfg, prompt_weights_kernel<128>, p, k, weights, window)
                    : cudaLaunchKernelEx(&cfg, prompt_weights_kernel<64>, p, k, weights, window);
}

} // namespace pkv
