// evict_kvcache: trim contexts to a budget by accumulated attention weight.
//
// For a sequence of n > budget tokens and each KV head, the `recent` last
// tokens stay and, of the n - recent before them, the budget - recent with the
// largest weight; on equal weights the lower index stays, and NaN counts as
// larger than every number.  The tokens that stay move, in their order, to
// positions 0 .. budget - 1 of the sequence's own blocks (K, V and weight).
//
// Two kernels:
//   select  one CTA per (sequence, KV head): a radix select over the weights
//           as order-preserving 32-bit keys (11 + 11 + 10 bits, a histogram in
//           shared memory each) gives the smallest key that stays and how many
//           tokens of exactly that key do; one more pass in token order ranks
//           the tokens that stay (ballots and a scan of the warps' counts),
//           writes the slots they come from, and moves their weights.
//   move    copies the K and V rows.  Token j comes from a position >= j, so
//           rows may be moved in place in ascending order: a CTA reads a tile
//           of rows into registers, waits until all its threads have, writes
//           them, and goes on; every later source lies past this tile.  CTAs
//           share no bytes: each takes one (sequence, KV head) and a fixed run
//           of 16-byte units of every row, which is where the parallelism of
//           few long sequences comes from.
// HBM-bound: 4 bytes per token and KV head read for the weights, and the rows
// that move read and written once.
#include "pkv_evict.h"
#include "pkv_kernels.h"
#include "pkv_ptx.cuh"

namespace pkv {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelBins = 2048;
constexpr int kMoveThreads = 256;
constexpr int kMoveDepth = 8;  // 16-byte loads in flight per thread

// Weight -> 32-bit key, larger weight = larger key: NaN (any) above +inf, and
// -0 equal to +0.
__device__ __forceinline__ uint32_t weight_key(float w)
{
    if (w != w)
        return 0xffffffffu;
    const uint32_t u = __float_as_uint(w + 0.f);  // -0 + 0 = +0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictParams p)
{
    __shared__ uint32_t hist[kSelBins];
    __shared__ uint32_t scan[kSelWarps * 2];
    __shared__ uint32_t s_prefix, s_left;
    __shared__ int s_first;
    const int h = blockIdx.x, b = blockIdx.y;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr unsigned FULL = 0xffffffffu;
    grid_dependency_wait();

    const int n = p.context_lens[b];
    int2 *moved = p.ws_moved + (size_t)b * p.Hkv + h;
    bool cut = n > p.budget;
    if (n < 0 || (long long)n > (long long)p.MBS * p.bs) {
        if (h == 0 && tid == 0)
            flag_error(p.err_flag, 0x4 /* PKV_FLAG_BAD_CONTEXT_LEN */);
        cut = false;
    }
    const int32_t *table = p.block_tables + (size_t)b * p.MBS;
    if (cut) {
        bool bad = false;
        for (int i = tid; i < (n - 1) / p.bs + 1; i += kSelThreads) {
            const int blk = table[i];
            bad |= blk < 0 || blk >= p.NB;
        }
        if (__syncthreads_or(bad)) {
            if (h == 0 && tid == 0)
                flag_error(p.err_flag, 0x2 /* PKV_FLAG_BAD_BLOCK */);
            cut = false;
        }
    }
    if (!cut) {  // nothing to trim, or a sequence left alone
        if (tid == 0)
            *moved = make_int2(0, 0);
        return;
    }
    const int old = n - p.recent;         // tokens the weights decide on
    const int want = p.budget - p.recent; // of them, how many stay (< old)
    auto at = [&](int t) -> float * {
        const int j = t / p.bs;
        return p.weights + ((size_t)table[j] * p.Hkv + h) * p.bs + (t - j * p.bs);
    };

    // ---- the smallest key that stays (prefix) and how many tokens of it (left)
    uint32_t prefix = 0xffffffffu, left = 0;
    if (want > 0) {
        prefix = 0;
        left = (uint32_t)want;
#pragma unroll 1
        for (int pass = 0; pass < 3; pass++) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
            const uint32_t bins = pass == 2 ? 1024u : 2048u;
            const uint32_t above = pass == 0 ? 0u : pass == 1 ? 0xffe00000u : 0xfffffc00u;
            for (uint32_t i = tid; i < bins; i += kSelThreads)
                hist[i] = 0;
            __syncthreads();
            for (int t = tid; t < old; t += kSelThreads) {
                const uint32_t u = weight_key(*at(t));
                if ((u & above) == (prefix & above))
                    atomicAdd(&hist[(u >> shift) & (bins - 1)], 1u);
            }
            __syncthreads();
            // thread i owns bins 2i, 2i + 1 counted from the top; the bin in
            // which the running count from the top reaches `left`
            const uint32_t per = bins / kSelThreads;  // 2 or 1
            uint32_t own[2] = {0, 0};
            for (uint32_t i = 0; i < per; i++)
                own[i] = hist[bins - 1 - (tid * per + i)];
            uint32_t sum = own[0] + own[1], incl = sum;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const uint32_t y = __shfl_up_sync(FULL, incl, off);
                if (lane >= off)
                    incl += y;
            }
            if (lane == 31)
                scan[warp] = incl;
            __syncthreads();
            uint32_t before = incl - sum;
            for (int w = 0; w < warp; w++)
                before += scan[w];
            for (uint32_t i = 0; i < per; i++) {
                if (before < left && left <= before + own[i]) {
                    s_prefix = prefix | ((bins - 1 - (tid * per + i)) << shift);
                    s_left = left - before;
                }
                before += own[i];
            }
            __syncthreads();
            prefix = s_prefix;
            left = s_left;
            __syncthreads();
        }
    }

    // ---- rank the tokens that stay, in order; record their slots, move weights
    int32_t *src = p.ws_src + ((size_t)b * p.Hkv + h) * p.keep;
    int32_t *dst = p.ws_dst + (size_t)b * p.keep;
    uint32_t kept0 = 0, equal0 = 0;  // tokens kept, and of the border key, before this chunk
    int first = p.budget;            // first token that moves
    if (tid == 0)
        s_first = p.budget;
    for (int c0 = 0; c0 < n; c0 += kSelThreads) {
        const int t = c0 + tid;
        float w = 0.f;
        int slot = 0;
        bool over = false, border = false;
        if (t < n) {
            const int j = t / p.bs, o = t - j * p.bs, blk = table[j];
            slot = blk * p.bs + o;
            w = p.weights[((size_t)blk * p.Hkv + h) * p.bs + o];
            const uint32_t u = weight_key(w);
            over = t >= old || (want > 0 && u > prefix);
            border = t < old && want > 0 && u == prefix;
            if (h == 0 && t < p.budget)
                dst[t] = slot;
        }
        const uint32_t lower = (1u << lane) - 1u;
        const uint32_t mo = __ballot_sync(FULL, over), mb = __ballot_sync(FULL, border);
        if (lane == 0) {
            scan[warp] = __popc(mo);
            scan[kSelWarps + warp] = __popc(mb);
        }
        __syncthreads();  // also: every weight of the chunk has been read
        uint32_t o_before = 0, b_before = 0, o_all = 0, b_all = 0;
        for (int x = 0; x < kSelWarps; x++) {
            const uint32_t co = scan[x], cb = scan[kSelWarps + x];
            if (x < warp) {
                o_before += co;
                b_before += cb;
            }
            o_all += co;
            b_all += cb;
        }
        // of the border tokens the first `left` stay
        const uint32_t eq = equal0 + b_before + __popc(mb & lower);
        const uint32_t eq_kept = min(eq, left);
        if (over || (border && eq < left)) {
            const int j = (int)(kept0 + o_before + __popc(mo & lower) + (eq_kept - min(equal0, left)));
            src[j] = slot;
            if (j != t) {
                *at(j) = w;
                first = min(first, j);
            }
        }
        kept0 += o_all + (min(equal0 + b_all, left) - min(equal0, left));
        equal0 += b_all;
        __syncthreads();  // scan[] is free again
    }
    first = __reduce_min_sync(FULL, first);
    if (lane == 0)
        atomicMin(&s_first, first);
    __syncthreads();
    if (tid == 0)
        *moved = make_int2(s_first, p.budget);
}

__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictParams p)
{
    const int slice = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
    grid_dependency_wait();
    const int2 moved = p.ws_moved[(size_t)b * p.Hkv + h];
    if (slice == 0 && h == 0 && threadIdx.x == 0) {
        // here, not in the selection: its CTAs all read the length, and
        // out_lens may be context_lens.  The fence makes it visible to a next
        // kernel that starts as soon as this one's CTAs have left.
        const int n = p.context_lens[b];
        p.out_lens[b] = moved.y > 0 ? p.budget : n;
        __threadfence();
    }
    if (moved.x >= moved.y)
        return;
    // this CTA's units of every row: K's are 0 .. units - 1, V's the next
    const int per = 2 * p.units / p.slices;  // a power of two
    const int u0 = slice * per + (int)(threadIdx.x % per);
    uint4 *cache = u0 < p.units ? p.k_cache : p.v_cache;
    const int unit = u0 % p.units;
    const int rows = kMoveThreads / per;  // tokens per step of the tile
    const int32_t *src = p.ws_src + ((size_t)b * p.Hkv + h) * p.keep;
    const int32_t *dst = p.ws_dst + (size_t)b * p.keep;
    auto at = [&](int slot) { return cache + ((size_t)slot * p.Hkv + h) * p.units + unit; };
    for (int j0 = moved.x + (int)threadIdx.x / per; j0 - (int)threadIdx.x / per < moved.y;
         j0 += rows * kMoveDepth) {
        uint4 x[kMoveDepth];
#pragma unroll
        for (int i = 0; i < kMoveDepth; i++) {
            const int j = j0 + i * rows;
            if (j < moved.y)
                x[i] = *at(src[j]);
        }
        __syncthreads();  // the tile's rows are all in registers
#pragma unroll
        for (int i = 0; i < kMoveDepth; i++) {
            const int j = j0 + i * rows;
            if (j < moved.y)
                *at(dst[j]) = x[i];
        }
    }
}

static cudaLaunchConfig_t evict_config(dim3 grid, int threads, cudaLaunchAttribute *attr,
                                       cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

cudaError_t launch_evict_select(const EvictParams &p, cudaStream_t stream)
{
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg =
        evict_config(dim3((unsigned)p.Hkv, (unsigned)p.B), kSelThreads, attr, stream);
    return cudaLaunchKernelEx(&cfg, evict_select_kernel, p);
}

cudaError_t launch_evict_move(const EvictParams &p, cudaStream_t stream)
{
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = evict_config(
        dim3((unsigned)p.slices, (unsigned)p.Hkv, (unsigned)p.B), kMoveThreads, attr, stream);
    return cudaLaunchKernelEx(&cfg, evict_move_kernel, p);
}

} // namespace pkv
