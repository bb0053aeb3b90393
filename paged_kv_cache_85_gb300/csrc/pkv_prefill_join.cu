// Joins the splits of the 128-key prefill kernel's items.
//
// Split i of a row's keys left o_i = sum 2^(s - lse_i) v (fp32, normalised) and
// lse_i = log2 sum 2^s.  With L = log2 sum_i 2^lse_i,
//     out = sum_i 2^(lse_i - L) o_i,
// and L is the row's log-sum-exp for the attention weights (+inf where no split
// could read a key: weight 0, output 0).  The splits of a row follow from its
// sequence's lengths as in the prefill kernel.
//
// One warp at a time per (row, query head).  Read once.  Where few rows meet long
// contexts from some KB to 60 MB (151 items in three splits): bound by its latency
// where they are few, which is why the sequences' boundaries are searched in
// shared memory.  Where only the last round's items are split, up to 80 MB; the
// other items' rows cost one load.
#include <cuda_bf16.h>

#include "pkv_kernels.h"
#include "pkv_prefill.h"
#include "pkv_ptx.cuh"

namespace pkv {

constexpr int kJoinWarps = 8;

template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) prefill_join_kernel(const PrefillParams p)
{
    __shared__ int cq[kJoinMaxSeqs + 1], ck[kJoinMaxSeqs + 1];
    constexpr int DPL = D / 32;
    constexpr unsigned FULL = 0xffffffffu;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_launch_dependents();
    grid_dependency_wait();
    for (int i = threadIdx.x; i <= p.B; i += kJoinWarps * 32) {
        cq[i] = p.cu_q[i];
        ck[i] = p.cu_k[i];
    }
    __syncthreads();
    // Warp w takes rows w, w + warps, ... (so that the rows of the items that were
    // split, which lie next to each other, spread over all warps) and looks at 32 of
    // them at once for those that were not.
    const int G = p.Hq / p.Hkv;
    const long long rows = p.Tq * p.Hq, warps = (long long)gridDim.x * kJoinWarps;
    const size_t stride = (size_t)rows;
    auto lse_of = [&](long long at) {
        const int row = (int)(at / p.Hq), hq = (int)(at % p.Hq);
        return ((size_t)(hq / G) * p.Tq + row) * G + hq % G;
    };
    auto join = [&](long long at) {
        const int row = (int)(at / p.Hq), hq = (int)(at % p.Hq);
        const size_t lse_at = lse_of(at);
        // the sequence that holds the row: boundaries need not be sane, so every one is
        // looked at
        int b = -1;
        for (int i = lane; i < p.B; i += 32)
            if (cq[i] <= row && row < cq[i + 1])
                b = i;
        b = __reduce_max_sync(FULL, b);
        if (b < 0)
            return;
        const int q_len = cq[b + 1] - cq[b], k_len = ck[b + 1] - ck[b];
        // the sequences that the attention takes (prefill_seq_sane)
        if (cq[b] < 0 || (long long)cq[b + 1] > p.Tq || k_len < q_len ||
            (long long)k_len > (long long)p.MBS * p.bs || q_len > p.max_q)
            return;
        // key tiles of the row's item: a pair of query tiles of 128 / G tokens each
        const int tpc = kPrefillRows / G, tok0 = (row - cq[b]) / (2 * tpc) * (2 * tpc);
        const int nkt = (k_len - q_len + min(q_len, tok0 + 2 * tpc) - 1) / 128 + 1;
        const int chunk = wide_chunk(nkt, p.splits, p.least), n = (nkt + chunk - 1) / chunk;

        float M = -INFINITY;
        for (int i = lane; i < n; i += 32)
            M = fmaxf(M, p.part_lse[i * stride + lse_at]);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            M = fmaxf(M, __shfl_xor_sync(FULL, M, off));
        // a NaN log-sum-exp (NaN scores) does not show in the maximum: it comes in here
        float acc[DPL], W = 0.f;
#pragma unroll
        for (int c = 0; c < DPL; c++)
            acc[c] = 0.f;
        const float *o = p.part_out + ((size_t)row * p.Hq + hq) * D + lane * DPL;
#pragma unroll 4
        for (int i = 0; i < n; i++) {
            const float lse = p.part_lse[i * stride + lse_at];
            const float w = lse == -INFINITY ? 0.f : fast_exp2(lse - (M == -INFINITY ? 0.f : M));
            W += w;
            float x[DPL];
#pragma unroll
            for (int c = 0; c < DPL; c++)
                x[c] = o[i * stride * D + c];
            if (lse != -INFINITY)
#pragma unroll
                for (int c = 0; c < DPL; c++)
                    acc[c] += w * x[c];
        }
        const float inv = W > 0.f ? 1.f / W : 0.f;
        uint16_t *dst = p.out + ((size_t)row * p.Hq + hq) * D + lane * DPL;
#pragma unroll
        for (int c = 0; c < DPL; c += 2)
            *reinterpret_cast<uint32_t *>(dst + c) = pack_bf16x2(acc[c] * inv, acc[c + 1] * inv);
        if (lane == 0 && p.lse)
            p.lse[lse_at] = W == 0.f ? INFINITY : (M == -INFINITY ? 0.f : M) + log2f(W);
    };
    for (long long at0 = (long long)blockIdx.x * kJoinWarps + warp; at0 < rows; at0 += 32 * warps) {
        const long long mine = at0 + lane * warps;
        const bool split = mine < rows && p.part_lse[lse_of(mine)] != INFINITY;
        for (unsigned todo = __ballot_sync(FULL, split); todo; todo &= todo - 1)
            join(at0 + (__ffs(todo) - 1) * warps);
    }
}

cudaError_t launch_prefill_join(int D, const PrefillParams &p, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    const long long need = (p.Tq * p.Hq + kJoinWarps - 1) / kJoinWarps, most = 8 * kWideSms;
    cfg.gridDim = dim3((unsigned)(need < most ? need : most));
    cfg.blockDim = dim3(kJoinWarps * 32);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return D == 128 ? cudaLaunchKernelEx(&cfg, prefill_join_kernel<128>, p)
                    : cudaLaunchKernelEx(&cfg, prefill_join_kernel<64>, p);
}

} // namespace pkv
