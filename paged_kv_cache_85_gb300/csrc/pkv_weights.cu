// The second kernel of a decode step that records attention weights: the merge
// of split streams' outputs (pkv_merge.cuh) and, by other CTAs of the same
// launch, the weights added to the cache's table.
//
// The decode kernel left, per box of a stream, the scores s[g][t] (log2
// units) of its tokens for the G query heads of the group.  A token's weight
// in this step is the sum of its G softmax values,
//     w = sum_g 2^(s[g][t] - lse[g]),
// added to weights[block, kv head, offset].  The slot of the step's newest token,
// which may hold what an earlier owner of the block left, was cleared by the
// decode kernel: sequences may share the block it lies in, so that all additions
// have to come after that.
// lse[g] is the row's log-sum-exp: left by the worker that read the whole
// stream, or M + log2(sum_i 2^(m_i - M) l_i) over the pieces (m_i, l_i) of a
// split one, which each warp forms for the streams it meets, so that the
// weights need not wait for the merge (one launch less in the call's chain).
//
// One thread per four tokens of a box (16-byte loads of the scores and one
// 16-byte addition to the weights, which lie next to each other in a block).
// Every (token, KV head) gets exactly one addition per call, so the sums do not
// depend on the order of the threads; they are atomic because two sequences of
// a batch may share a prefix block (then their two additions may come in either
// order).
//
// Bound by the traffic of scores and weights and, on small calls, by three
// dependent reads: 16 us for 512 FP8 contexts (24 MB of scores, 24 of weights),
// 4 us beyond the plain call for 64 bf16 ones (17 MB in all).
#include "pkv_kernels.h"
#include "pkv_merge.cuh"
#include "pkv_ptx.cuh"

namespace pkv {

constexpr int kAddThreads = kMergeWarps * 32;

// The decode kernel's slicing (as in merge_row).
struct Slices {
    int P, Wr, R, per_head;
};

// Log-sum-exps of the G rows of stream (b, h), by the whole warp.
template <int D, int G>
__device__ __forceinline__ void stream_lse(const DecodeParams &p, const Slices &S, int b, int h, int lane,
                                           float (&lse)[G])
{
    constexpr unsigned FULL = 0xffffffffu;
    const int *pb = p.ws_hdr + kWsHeaderInts;
    const int p0 = pb[b], nb = pb[b + 1] - p0;
    const int r = S.R == p.Hkv ? h : 0;
    const int s = (S.R == p.Hkv ? 0 : h * S.per_head) + p0;
    const int w0 = r * S.Wr + s / S.P, w1 = r * S.Wr + (s + nb - 1) / S.P;
    if (w0 == w1) {
#pragma unroll
        for (int g = 0; g < G; g++)
            lse[g] = p.ws_lse[(size_t)b * p.Hq + (size_t)h * G + g];
        return;
    }
    const int n = w1 - w0 + 1, slot0 = s % S.P == 0 ? 0 : 1;
    float M[G], L[G];
#pragma unroll
    for (int g = 0; g < G; g++) {
        M[g] = -INFINITY;
        L[g] = 0.f;
    }
    for (int i = lane; i < n; i += 32) {
        const float *pc = p.ws_part + ((size_t)(w0 + i) * 2 + (i == 0 ? slot0 : 0)) * G * (D + 4);
#pragma unroll
        for (int g = 0; g < G; g++) {
            const float2 ml = *reinterpret_cast<const float2 *>(pc + g * (D + 4) + D);
            const float m = fmaxf(M[g], ml.x);
            // a piece none of whose keys could be read has m = -inf, l = 0
            L[g] = L[g] * (M[g] == -INFINITY ? 0.f : fast_exp2(M[g] - m)) +
                   ml.y * (ml.x == -INFINITY ? 0.f : fast_exp2(ml.x - m));
            M[g] = m;
        }
    }
#pragma unroll
    for (int g = 0; g < G; g++) {
        float m = M[g];
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            m = fmaxf(m, __shfl_xor_sync(FULL, m, off));
        float l = M[g] == -INFINITY ? L[g] : L[g] * fast_exp2(M[g] - m);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            l += __shfl_xor_sync(FULL, l, off);
        lse[g] = l == 0.f ? INFINITY : m + log2f(l);
    }
}

// TM: the scores are token-major ([BT][G], FP8 caches), else [G][BT].
template <int D, int G, int BT, bool TM>
__global__ void __launch_bounds__(kAddThreads, G == 8 ? 4 : 8)
    merge_and_add_kernel(const DecodeParams p, int add_ctas)
{
    constexpr unsigned FULL = 0xffffffffu;
    constexpr int kQuads = BT / 4;  // threads per box
    const int lane = threadIdx.x & 31;
    grid_launch_dependents();
    if ((int)blockIdx.x >= add_ctas) {
        const long long row = (long long)(blockIdx.x - add_ctas) * kMergeWarps + (threadIdx.x >> 5);
        if (row < (long long)p.B * p.Hq)
            merge_row<D>(p, row, lane);
        return;
    }
    // scores, descriptors and the pieces' sums come from the decode kernel
    grid_dependency_wait();
    const Slices S = {p.ws_hdr[1], p.ws_hdr[2], p.ws_hdr[4], p.ws_hdr[kWsHeaderInts + p.B]};
    // each warp takes a run of boxes next to each other, 32 / kQuads at a time,
    // so that it meets few streams; the next boxes are read ahead
    const int boxes = S.per_head * p.Hkv;
    const int warps = add_ctas * kMergeWarps;
    constexpr int kStep = 32 / kQuads;
    const int run = ((boxes + warps - 1) / warps + kStep - 1) / kStep * kStep;
    const long long first = (long long)(blockIdx.x * kMergeWarps + (threadIdx.x >> 5)) * run;
    if (first >= boxes)
        return;
    const int end = (int)min((long long)boxes, first + run);
    const int i = lane % kQuads * 4;  // this thread's tokens of its box
    int4 mn = make_int4(0, -1, 0, 0);
    float4 sn[G];
    auto read = [&](int box) {
        mn = make_int4(0, -1, 0, 0);
        if (box < end) {
            mn = p.ws_box[box];
            const float *sc = p.ws_score + (size_t)box * G * BT + (TM ? i * G : i);
#pragma unroll
            for (int g = 0; g < G; g++)
                sn[g] = *reinterpret_cast<const float4 *>(sc + g * (TM ? 4 : BT));
        }
    };
    read((int)first + lane / kQuads);
    int b1 = -1, h1 = -1;  // the stream whose log-sum-exps are in l1
    float l1[G];
    for (int box0 = (int)first; box0 < end; box0 += kStep) {
        const int box = box0 + lane / kQuads;
        const int4 m = mn;
        float4 s[G];
#pragma unroll
        for (int g = 0; g < G; g++)
            s[g] = sn[g];
        read(box + kStep);
        const int h = box / S.per_head;
        // a decode kernel that gave up waiting leaves descriptors unwritten: what
        // stands there then is checked before it is an address
        const int nvalid = min(m.w, BT);
        const bool valid = (unsigned)m.y < (unsigned)p.NB && (unsigned)m.x < (unsigned)p.B &&
                           (unsigned)m.z <= (unsigned)(p.bs - BT) && m.z % BT == 0 && i < nvalid;
        // the streams of these boxes, one after the other (mostly one, and the
        // same as before)
        float lse[G];
        for (unsigned todo = __ballot_sync(FULL, valid); todo;) {
            const int src = __ffs(todo) - 1;
            const int b2 = __shfl_sync(FULL, m.x, src), h2 = __shfl_sync(FULL, h, src);
            if (b2 != b1 || h2 != h1) {
                b1 = b2;
                h1 = h2;
                stream_lse<D, G>(p, S, b1, h1, lane, l1);
            }
            const bool mine = valid && m.x == b1 && h == h1;
            if (mine) {
#pragma unroll
                for (int g = 0; g < G; g++)
                    lse[g] = l1[g];
            }
            todo &= ~__ballot_sync(FULL, mine);
        }
        if (!valid)
            continue;
        float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
        if constexpr (TM) {
            // s holds 4 G values, token by token
            const float *v = reinterpret_cast<const float *>(s);
#pragma unroll
            for (int g = 0; g < G; g++) {
                w.x += fast_exp2(v[g] - lse[g]);
                w.y += fast_exp2(v[G + g] - lse[g]);
                w.z += fast_exp2(v[2 * G + g] - lse[g]);
                w.w += fast_exp2(v[3 * G + g] - lse[g]);
            }
        } else {
#pragma unroll
            for (int g = 0; g < G; g++) {
                w.x += fast_exp2(s[g].x - lse[g]);
                w.y += fast_exp2(s[g].y - lse[g]);
                w.z += fast_exp2(s[g].z - lse[g]);
                w.w += fast_exp2(s[g].w - lse[g]);
            }
        }
        float *dst = p.weights + ((size_t)m.y * p.Hkv + h) * p.bs + m.z + i;
        if (i + 4 <= nvalid) {
            atomicAdd(reinterpret_cast<float4 *>(dst), w);
        } else {  // none past the context's last token
            const float x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int k = 0; k < 3; k++)
                if (i + k < nvalid)
                    atomicAdd(dst + k, x[k]);
        }
    }
}

cudaError_t launch_merge_and_add(int D, int G, int bt, bool token_major, const DecodeParams &p,
                                 long long max_boxes, int sms, cudaStream_t stream)
{
    const long long rows = (long long)p.B * p.Hq;
    const long long merge = (rows + kMergeWarps - 1) / kMergeWarps;
    const long long need = (max_boxes * (bt / 4) + kAddThreads - 1) / kAddThreads;
    // one wave of CTAs with runs of several steps (their first step waits for
    // three dependent reads), beside the merge's
    const long long most = (long long)sms * 6;
    const long long add = need < most ? need : most;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)(add + merge));
    cfg.blockDim = dim3(kAddThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
#define PKV_ADD(DD, GG, BB, TM)                                  \
    if (D == DD && G == GG && bt == BB && token_major == TM) \
        return cudaLaunchKernelEx(&cfg, merge_and_add_kernel<DD, GG, BB, TM>, p, (int)add);
#define PKV_ADD2(DD, GG) \
    PKV_ADD(DD, GG, kBox, false) PKV_ADD(DD, GG, kBox, true) PKV_ADD(DD, GG, 2 * kBox, true)
    PKV_ADD2(64, 1) PKV_ADD2(64, 2) PKV_ADD2(64, 4) PKV_ADD2(64, 8)
    PKV_ADD2(128, 1) PKV_ADD2(128, 2) PKV_ADD2(128, 4) PKV_ADD2(128, 8)
#undef PKV_ADD2
#undef PKV_ADD
    return cudaErrorInvalidValue;
}

} // namespace pkv
