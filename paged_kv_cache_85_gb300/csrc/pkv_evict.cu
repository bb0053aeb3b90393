// evict_kvcache: trim contexts to a budget by accumulated attention weight.
//
// For a sequence of n > budget tokens and each KV head, the `recent` last
// tokens stay and, of the n - recent before them, the budget - recent with the
// largest weight; on equal weights the lower index stays, and NaN counts as
// larger than every number.  The tokens that stay move, in their order, to
// positions 0 .. budget - 1 of the sequence's own blocks (K, V and weight).
//
// Two kernels:
//   select  one CTA per (sequence, KV head), or a cluster of up to eight that
//           split its tokens where there are few of them: the weights are read
//           once into shared memory as order-preserving 32-bit keys; a radix
//           select over them (11 + 11 + 10 bits, a histogram each; a cluster's
//           CTAs add their non-empty bins to the first one's through distributed
//           shared memory) gives the leading bits of the smallest key that
//           stays and how many tokens with exactly those bits do.  It ends as
//           soon as that is all of them: with distinct weights the third
//           histogram is rarely needed.  One more
//           pass in token order ranks the tokens that stay and writes the slots
//           they come from.
//   move    copies the K and V rows and the weights.  Token j comes from a
//           position >= j, so rows may be moved in place in ascending order: a
//           CTA reads a tile of rows into registers, waits until all its
//           threads have, writes them, and goes on; every later source lies
//           past this tile, so the next tile is read before this one is
//           written.  CTAs share no bytes: each takes one (sequence, KV head)
//           and a fixed run of 16-byte units of every row (one more CTA the
//           weights), which is where the parallelism of few long sequences
//           comes from.
// HBM-bound: 4 bytes per token and KV head read for the weights, and the rows
// that move read and written once.
#include <cooperative_groups.h>

#include "pkv_evict.h"
#include "pkv_kernels.h"
#include "pkv_ptx.cuh"

namespace cg = cooperative_groups;

namespace pkv {

constexpr int kSelThreads = 256;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelBins = 2048;
constexpr int kMoveThreads = 128;
constexpr int kMoveDepth = 4;  // 16-byte loads per thread and tile; two tiles in flight

__device__ __forceinline__ int divide(int n, FastDiv f)
{
    return (int)((__umulhi(f.mul, (uint32_t)n) + (uint32_t)n) >> f.shift);
}

// Weight -> 32-bit key, larger weight = larger key: NaN (any) above +inf, and
// -0 equal to +0.
__device__ __forceinline__ uint32_t weight_key(float w)
{
    if (w != w)
        return 0xffffffffu;
    const uint32_t u = __float_as_uint(w + 0.f);  // -0 + 0 = +0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

struct SelShared {
    uint32_t hist[3][kSelBins];
    uint32_t scan[2][kSelWarps];
    uint32_t over, border;  // this CTA's tokens over the border key and on it
    uint32_t prefix, left, whole;
    int first, bad;
};

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictParams p)
{
    extern __shared__ __align__(16) uint8_t smem[];
    SelShared &S = *reinterpret_cast<SelShared *>(smem);
    uint4 *keys = reinterpret_cast<uint4 *>(smem + align_up(sizeof(SelShared), 16));
    const cg::cluster_group cluster = cg::this_cluster();
    const int C = p.cluster, rank = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr unsigned FULL = 0xffffffffu;
    auto sync_all = [&]() {  // the CTAs of this (sequence, KV head)
        if (C > 1)
            cluster.sync();
        else
            __syncthreads();
    };
    grid_dependency_wait();

    const int n = p.context_lens[b];
    const bool lead = rank == 0 && tid == 0;
    int2 *moved = p.ws_moved + (size_t)b * p.Hkv + h;
    const bool bad_len = n < 0 || (long long)n > (long long)p.MBS * p.bs;
    if (bad_len || n <= p.budget) {  // nothing to trim, or a sequence left alone
        if (lead) {
            if (bad_len && h == 0)
                flag_error(p.err_flag, 0x4 /* PKV_FLAG_BAD_CONTEXT_LEN */);
            *moved = make_int2(0, 0);
        }
        return;
    }
    const int32_t *table = p.block_tables + (size_t)b * p.MBS;
    const int old = n - p.recent;         // tokens the weights decide on
    const int want = p.budget - p.recent; // of them, how many stay (< old)
    // this CTA's tokens: [t0, t1), in quads of four (a quad never leaves its block)
    const int seg = ((n + C - 1) / C + 3) & ~3;
    const int t0 = min(n, rank * seg), t1 = min(n, t0 + seg);
    const int quads = (t1 - t0 + 3) / 4;
    auto load = [&](int q, bool &bad) -> uint4 {
        const int t = t0 + 4 * q, j = divide(t, p.block);
        const int blk = __ldg(table + j);
        if (blk < 0 || blk >= p.NB) {
            bad = true;
            return make_uint4(0, 0, 0, 0);
        }
        const float4 w = *reinterpret_cast<const float4 *>(
            p.weights + ((size_t)blk * p.Hkv + h) * p.bs + (t - j * p.bs));
        return make_uint4(weight_key(w.x), weight_key(w.y), weight_key(w.z), weight_key(w.w));
    };
    // keys of a quad: from shared memory, or again from the table where it is full
    auto quad = [&](int q) -> uint4 {
        bool bad = false;
        return 4 * q < p.cap ? keys[q] : load(q, bad);
    };
    {
        if (tid == 0) {
            S.bad = 0;
            S.first = p.budget;
            S.over = S.border = 0;
        }
        bool bad = false;
#pragma unroll 4
        for (int q = tid; q < quads; q += kSelThreads) {
            const uint4 k = load(q, bad);
            if (4 * q < p.cap)
                keys[q] = k;
        }
        __syncthreads();
        if (bad)
            S.bad = 1;
        for (int i = tid; i < 3 * kSelBins; i += kSelThreads)
            (&S.hist[0][0])[i] = 0;
        sync_all();
        int any = S.bad;
        if (C > 1) {
            if (any && tid < C)  // tell every CTA of the cluster
                *cluster.map_shared_rank(&S.bad, tid) = 1;
            cluster.sync();
            any = S.bad;
        }
        if (any) {
            if (lead) {
                if (h == 0)
                    flag_error(p.err_flag, 0x2 /* PKV_FLAG_BAD_BLOCK */);
                *moved = make_int2(0, 0);
            }
            return;
        }
    }

    // ---- the leading bits (mask) of the smallest key that stays, and how many
    // tokens with exactly those bits do (left)
    uint32_t prefix = 0xffffffffu, mask = 0xffffffffu, left = 0;
    if (want > 0) {
        prefix = 0;
        left = (uint32_t)want;
#pragma unroll 1
        for (int pass = 0; pass < 3; pass++) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
            const uint32_t bins = pass == 2 ? 1024u : 2048u;
            const uint32_t above = pass == 0 ? 0u : pass == 1 ? 0xffe00000u : 0xfffffc00u;
            uint32_t *hist = S.hist[pass];
            for (int q = tid; q < quads; q += kSelThreads) {
                const uint4 k = quad(q);
                const uint32_t u[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
                for (int i = 0; i < 4; i++)
                    if (t0 + 4 * q + i < min(old, t1) && (u[i] & above) == (prefix & above))
                        atomicAdd(&hist[(u[i] >> shift) & (bins - 1)], 1u);
            }
            __syncthreads();
            if (C > 1) {
                if (rank > 0) {
                    uint32_t *sum = cluster.map_shared_rank(hist, 0);
                    for (uint32_t i = tid; i < bins; i += kSelThreads)
                        if (hist[i])
                            atomicAdd(sum + i, hist[i]);
                }
                cluster.sync();
            }
            // thread i owns `per` bins counted from the top; the bin in which the
            // running count from the top reaches `left` holds the border key (in a
            // cluster the first CTA finds it and tells the others)
            const int per = (int)bins / kSelThreads;  // 8 or 4
            uint32_t own[kSelBins / kSelThreads], sum = 0;
#pragma unroll
            for (int i = 0; i < kSelBins / kSelThreads; i++) {
                own[i] = i < per ? hist[bins - 1 - (uint32_t)(tid * per + i)] : 0u;
                sum += own[i];
            }
            uint32_t incl = sum;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const uint32_t y = __shfl_up_sync(FULL, incl, off);
                if (lane >= off)
                    incl += y;
            }
            if (lane == 31)
                S.scan[0][warp] = incl;
            __syncthreads();
            uint32_t before = incl - sum;
            for (int w = 0; w < warp; w++)
                before += S.scan[0][w];
            if (rank == 0 && before < left && left <= before + sum) {
#pragma unroll
                for (int i = 0; i < kSelBins / kSelThreads; i++) {
                    if (before < left && left <= before + own[i]) {
                        for (int c = 0; c < C; c++) {
                            SelShared &to = C > 1 ? *cluster.map_shared_rank(&S, c) : S;
                            to.prefix = prefix | ((bins - 1 - (uint32_t)(tid * per + i)) << shift);
                            to.left = left - before;
                            to.whole = left - before == own[i];
                        }
                    }
                    before += own[i];
                }
            }
            sync_all();
            prefix = S.prefix;
            left = S.left;
            mask = 0xffffffffu << shift;
            const bool whole = S.whole;
            __syncthreads();  // read before the next pass writes them
            if (whole)
                break;
        }
    }

    // ---- rank the tokens that stay, in token order, and record their slots
    auto classes = [&](int q, const uint4 &k, uint32_t &over, uint32_t &border) {  // 4-bit masks
        const uint32_t u[4] = {k.x, k.y, k.z, k.w};
        over = border = 0;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int t = t0 + 4 * q + i;
            if (t < t1) {
                over |= (t >= old || (want > 0 && (u[i] & mask) > prefix) ? 1u : 0u) << i;
                border |= (t < old && want > 0 && (u[i] & mask) == prefix ? 1u : 0u) << i;
            }
        }
    };
    uint32_t o_before = 0, b_before = 0;  // in the CTAs before this one
    if (C > 1) {
        uint32_t o = 0, e = 0;
        for (int q = tid; q < quads; q += kSelThreads) {
            uint32_t mo, mb;
            classes(q, quad(q), mo, mb);
            o += __popc(mo);
            e += __popc(mb);
        }
        o = __reduce_add_sync(FULL, o);
        e = __reduce_add_sync(FULL, e);
        if (lane == 0) {
            atomicAdd(&S.over, o);
            atomicAdd(&S.border, e);
        }
        cluster.sync();
        for (int c = 0; c < rank; c++) {
            o_before += *cluster.map_shared_rank(&S.over, c);
            b_before += *cluster.map_shared_rank(&S.border, c);
        }
    }
    int32_t *src = p.ws_src + ((size_t)b * p.Hkv + h) * p.keep;
    int32_t *dst = p.ws_dst + (size_t)b * p.keep;
    int first = p.budget;  // first token that moves
    for (int q0 = 0; q0 < quads; q0 += kSelThreads) {
        const int q = q0 + tid;
        uint32_t mo = 0, mb = 0;
        if (q < quads)
            classes(q, quad(q), mo, mb);
        const uint32_t no = __popc(mo), nb = __popc(mb);
        uint32_t io = no, ib = nb;  // inclusive scans over the warp
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t yo = __shfl_up_sync(FULL, io, off), yb = __shfl_up_sync(FULL, ib, off);
            if (lane >= off) {
                io += yo;
                ib += yb;
            }
        }
        if (lane == 31) {
            S.scan[0][warp] = io;
            S.scan[1][warp] = ib;
        }
        __syncthreads();
        uint32_t o = o_before + io - no, e = b_before + ib - nb;
#pragma unroll
        for (int w = 0; w < kSelWarps; w++) {
            const uint32_t co = S.scan[0][w], cb = S.scan[1][w];
            if (w < warp) {
                o += co;
                e += cb;
            }
            o_before += co;
            b_before += cb;
        }
        const int t = t0 + 4 * q;
        const bool to_dst = h == 0 && t < p.budget && q < quads;
        if ((mo | mb) || to_dst) {
            const int j = divide(t, p.block);
            const int slot = __ldg(table + j) * p.bs + (t - j * p.bs);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                // of the border tokens the first `left` stay
                const bool over = (mo >> i) & 1u, border = (mb >> i) & 1u;
                if (over || (border && e < left)) {
                    const int at = (int)(o + min(e, left));
                    src[at] = slot + i;
                    if (at != t + i)
                        first = min(first, at);
                }
                o += over;
                e += border;
                if (to_dst && t + i < p.budget)
                    dst[t + i] = slot + i;
            }
        }
        __syncthreads();  // scan[] is free again
    }
    first = __reduce_min_sync(FULL, first);
    if (lane == 0)
        atomicMin(&S.first, first);
    sync_all();
    if (lead) {
        first = S.first;
        for (int c = 1; c < C; c++)
            first = min(first, *cluster.map_shared_rank(&S.first, c));
        *moved = make_int2(first, p.budget);
    }
    if (C > 1)
        cluster.sync();  // the other CTAs' shared memory stays until it is read
}

// Copies tokens [first, end) of one (sequence, KV head): `lanes` threads take a
// token, thread i of them its i-th unit; get reads a token's source, put writes
// it.  Double-buffered tiles, indexes one tile further ahead.
template <typename T, typename Get, typename Put>
__device__ __forceinline__ void move_tiles(int first, int end, int lanes, const int32_t *src,
                                           const int32_t *dst, Get get, Put put)
{
    const int rows = kMoveThreads / lanes;  // tokens per step
    const int tile = rows * kMoveDepth;
    const int r = (int)threadIdx.x / lanes;
    int si[kMoveDepth], di[kMoveDepth];
    T x[2][kMoveDepth];
    auto index = [&](int j0, const int32_t *list, int (&to)[kMoveDepth]) {
#pragma unroll
        for (int i = 0; i < kMoveDepth; i++) {
            const int j = j0 + r + i * rows;
            to[i] = j < end ? __ldg(list + j) : -1;
        }
    };
    auto read = [&](T (&to)[kMoveDepth]) {
#pragma unroll
        for (int i = 0; i < kMoveDepth; i++)
            if (si[i] >= 0)
                to[i] = get(si[i]);
    };
    index(first, src, si);
    read(x[0]);
    index(first + tile, src, si);
    for (int j0 = first; j0 < end; j0 += 2 * tile) {
#pragma unroll
        for (int u = 0; u < 2; u++) {
            const int at = j0 + u * tile;
            if (at < end) {  // the same for the whole CTA
                index(at, dst, di);
                read(x[u ^ 1]);                  // tile at + tile: its sources lie past this tile
                index(at + 2 * tile, src, si);
                __syncthreads();                 // this tile is in every thread's registers
#pragma unroll
                for (int i = 0; i < kMoveDepth; i++)
                    if (di[i] >= 0)
                        put(di[i], x[u][i]);
            }
        }
    }
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
    const int32_t *src = p.ws_src + ((size_t)b * p.Hkv + h) * p.keep;
    const int32_t *dst = p.ws_dst + (size_t)b * p.keep;
    if (slice == p.slices) {  // the weights, fp32 [NB, Hkv, bs]
        auto at = [&](int slot) {
            const int blk = divide(slot, p.block);
            return p.weights + ((size_t)blk * p.Hkv + h) * p.bs + (slot - blk * p.bs);
        };
        move_tiles<float>(
            moved.x, moved.y, 1, src, dst, [&](int slot) { return *at(slot); },
            [&](int slot, float w) { *at(slot) = w; });
        return;
    }
    // this CTA's units of every row: K's are 0 .. units - 1, V's the next
    const int per = 2 * p.units / p.slices;  // a power of two
    const int u0 = slice * per + (int)(threadIdx.x % per);
    uint4 *base = (u0 < p.units ? p.k_cache : p.v_cache) + (size_t)h * p.units + u0 % p.units;
    const size_t row = (size_t)p.Hkv * p.units;
    move_tiles<uint4>(
        moved.x, moved.y, per, src, dst, [&](int slot) { return base[(size_t)slot * row]; },
        [&](int slot, const uint4 &x) { base[(size_t)slot * row] = x; });
}

size_t evict_select_smem_bytes(int cap)
{
    return align_up(sizeof(SelShared), 16) + (size_t)cap * sizeof(uint32_t);
}

const void *evict_select_kernel_fn() { return reinterpret_cast<const void *>(&evict_select_kernel); }

cudaError_t launch_evict_select(const EvictParams &p, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)p.cluster, (unsigned)p.Hkv, (unsigned)p.B);
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = evict_select_smem_bytes(p.cap);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, evict_select_kernel, p);
}

cudaError_t launch_evict_move(const EvictParams &p, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)p.slices + 1, (unsigned)p.Hkv, (unsigned)p.B);
    cfg.blockDim = dim3(kMoveThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, evict_move_kernel, p);
}

} // namespace pkv
