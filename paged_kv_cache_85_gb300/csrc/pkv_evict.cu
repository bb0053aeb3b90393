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
// that move read and written once.  Measured with nothing trimmed before, bf16,
// D = 128, 8 KV heads: 64 contexts up to 4096 tokens to 1024 in 88 us (select 12,
// move 70: 392 MB of DRAM traffic, 74% of its throughput in runs of 256 bytes),
// 8 of 32768 to 4096 in 71 (23 + 44).  Both in one kernel: 110 and 93.
#include <cooperative_groups.h>

#include "pkv_evict.h"
#include "pkv_kernels.h"
#include "pkv_ptx.cuh"

namespace cg = cooperative_groups;

namespace pkv {

constexpr int kSelThreads = 256;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelBins = 2048;
constexpr int kMoveThreads = 256;  // at most
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

struct __align__(16) SelShared {
    uint32_t hist[3][kSelBins];
    uint32_t scan[2][kSelWarps];
    uint32_t counts[8], borders[8];  // per CTA of the cluster: tokens over the border key, on it
    uint32_t mine, mine_border;      // this CTA's
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
    for (int i = tid; i < 3 * kSelBins / 4; i += kSelThreads)
        reinterpret_cast<uint4 *>(&S.hist[0][0])[i] = make_uint4(0, 0, 0, 0);
    if (tid == 0) {
        S.bad = 0;
        S.first = p.budget - p.recent;
        S.mine = S.mine_border = 0;
    }
    grid_dependency_wait();

    const int n = p.context_lens[b];
    const bool lead = rank == 0 && tid == 0;
    int2 *moved = p.ws_moved + (size_t)b * p.Hkv + h;
    const bool bad_len = n < 0 || (long long)n > (long long)p.MBS * p.bs;
    if (bad_len || n <= p.budget) {  // nothing to trim, or a sequence left alone
        if (lead) {
            if (bad_len && h == 0)
                flag_error(p.err_flag, 0x4 /* PKV_FLAG_BAD_CONTEXT_LEN */);
            *moved = make_int2(n, n);
        }
        return;
    }
    const int32_t *table = p.block_tables + (size_t)b * p.MBS;
    const int old = n - p.recent;         // tokens the weights decide on
    const int want = p.budget - p.recent; // of them, how many stay (< old)
    // this CTA's part of them: [t0, t1), in runs of eight, which never leave
    // their block
    const int seg = ((old + C - 1) / C + 7) & ~7;
    const int t0 = min(old, rank * seg), t1 = min(old, t0 + seg);
    const int runs = (t1 - t0 + 7) / 8;
    // the keys of a run; 0, below every weight's, past `old`
    auto load = [&](int q, uint4 &k0, uint4 &k1) -> bool {
        const int t = t0 + 8 * q, j = divide(t, p.block);
        const int blk = __ldg(table + j);
        k0 = k1 = make_uint4(0, 0, 0, 0);
        if (blk < 0 || blk >= p.NB)
            return false;
        const float4 *w = reinterpret_cast<const float4 *>(
            p.weights + ((size_t)blk * p.Hkv + h) * p.bs + (t - j * p.bs));
        const float4 a = w[0], c = w[1];
        k0 = make_uint4(weight_key(a.x), weight_key(a.y), weight_key(a.z), weight_key(a.w));
        k1 = make_uint4(weight_key(c.x), weight_key(c.y), weight_key(c.z), weight_key(c.w));
        if (t + 8 > old) {
            uint32_t *u = reinterpret_cast<uint32_t *>(&k0), *v = reinterpret_cast<uint32_t *>(&k1);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                u[i] = t + i < old ? u[i] : 0u;
                v[i] = t + 4 + i < old ? v[i] : 0u;
            }
        }
        return true;
    };
    // from shared memory, or again from the table where that is full
    auto run = [&](int q, uint4 &k0, uint4 &k1) {
        if (8 * q < p.cap) {
            k0 = keys[2 * q];
            k1 = keys[2 * q + 1];
        } else {
            load(q, k0, k1);
        }
    };
    __syncthreads();  // the histograms are clear
    {
        bool bad = false;
#pragma unroll 2
        for (int q = tid; q < runs; q += kSelThreads) {
            uint4 k0, k1;
            bad |= !load(q, k0, k1);
            if (8 * q < p.cap) {
                keys[2 * q] = k0;
                keys[2 * q + 1] = k1;
            }
            const uint32_t u[8] = {k0.x, k0.y, k0.z, k0.w, k1.x, k1.y, k1.z, k1.w};
#pragma unroll
            for (int i = 0; i < 8; i++)
                atomicAdd(&S.hist[0][u[i] >> 21], 1u);
        }
        // the recent tokens' blocks
        for (int j = old / p.bs + tid; j <= (n - 1) / p.bs; j += kSelThreads) {
            const int blk = __ldg(table + j);
            bad |= blk < 0 || blk >= p.NB;
        }
        if (bad)
            S.bad = 1;
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
                *moved = make_int2(n, n);
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
            uint32_t *hist = S.hist[pass];
            if (pass > 0) {  // the first one was counted while the weights came in
                for (int q = tid; q < runs; q += kSelThreads) {
                    uint4 k0, k1;
                    run(q, k0, k1);
                    const uint32_t u[8] = {k0.x, k0.y, k0.z, k0.w, k1.x, k1.y, k1.z, k1.w};
#pragma unroll
                    for (int i = 0; i < 8; i++)
                        if ((u[i] & mask) == prefix)
                            atomicAdd(&hist[(u[i] >> shift) & (bins - 1)], 1u);
                }
                __syncthreads();
            }
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
            if (rank == 0) {
                constexpr int kMost = kSelBins / kSelThreads;
                const int per = (int)bins / kSelThreads;  // 8 or 4
                uint32_t own[kMost], sum = 0;  // ascending bins
#pragma unroll
                for (int i = 0; i < kMost; i += 4) {
                    uint4 x = make_uint4(0, 0, 0, 0);
                    if (i < per)
                        x = *reinterpret_cast<const uint4 *>(hist + bins - per * (tid + 1) + i);
                    own[i] = x.x;
                    own[i + 1] = x.y;
                    own[i + 2] = x.z;
                    own[i + 3] = x.w;
                    sum += x.x + x.y + x.z + x.w;
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
#pragma unroll
                for (int w = 0; w < kSelWarps; w++)
                    before += w < warp ? S.scan[0][w] : 0u;
                if (before < left && left <= before + sum) {
#pragma unroll
                    for (int i = kMost - 1; i >= 0; i--) {
                        if (before < left && left <= before + own[i]) {
                            const uint32_t bin = bins - (uint32_t)(per * (tid + 1)) + (uint32_t)i;
                            for (int c = 0; c < C; c++) {
                                SelShared &to = C > 1 ? *cluster.map_shared_rank(&S, c) : S;
                                to.prefix = prefix | (bin << shift);
                                to.left = left - before;
                                to.whole = left - before == own[i];
                            }
                        }
                        before += own[i];
                    }
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
    auto classes = [&](int q, uint32_t &over, uint32_t &border) {  // a bit per token
        uint4 k0, k1;
        run(q, k0, k1);
        const uint32_t u[8] = {k0.x, k0.y, k0.z, k0.w, k1.x, k1.y, k1.z, k1.w};
        over = border = 0;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            over |= (u[i] & mask) > prefix ? 1u << i : 0u;
            border |= (u[i] & mask) == prefix ? 1u << i : 0u;
        }
    };
    int32_t *src = p.ws_src + ((size_t)b * p.Hkv + h) * p.keep;
    int first = want;  // first token that moves (the recent ones all do)
    if (want > 0) {
        uint32_t o_before = 0, b_before = 0;  // in the CTAs before this one
        if (C > 1) {
            uint32_t o = 0, e = 0;
            for (int q = tid; q < runs; q += kSelThreads) {
                uint32_t mo, mb;
                classes(q, mo, mb);
                o += __popc(mo);
                e += __popc(mb);
            }
            o = __reduce_add_sync(FULL, o);
            e = __reduce_add_sync(FULL, e);
            if (lane == 0) {
                atomicAdd(&S.mine, o);
                atomicAdd(&S.mine_border, e);
            }
            __syncthreads();
            if (tid < C) {
                SelShared &to = *cluster.map_shared_rank(&S, tid);
                to.counts[rank] = S.mine;
                to.borders[rank] = S.mine_border;
            }
            cluster.sync();
            for (int c = 0; c < rank; c++) {
                o_before += S.counts[c];
                b_before += S.borders[c];
            }
        }
        for (int q0 = 0, buf = 0; q0 < runs; q0 += kSelThreads, buf ^= 1) {
            const int q = q0 + tid;
            uint32_t mo = 0, mb = 0;
            if (q < runs)
                classes(q, mo, mb);
            // both counts in one word: a step holds 2048 tokens
            const uint32_t own = __popc(mo) | (__popc(mb) << 16);
            uint32_t incl = own;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const uint32_t y = __shfl_up_sync(FULL, incl, off);
                if (lane >= off)
                    incl += y;
            }
            if (lane == 31)
                S.scan[buf][warp] = incl;
            __syncthreads();
            uint32_t before = incl - own, all = 0;
#pragma unroll
            for (int w = 0; w < kSelWarps; w++) {
                const uint32_t x = S.scan[buf][w];
                before += w < warp ? x : 0u;
                all += x;
            }
            if (mo | mb) {
                uint32_t o = o_before + (before & 0xffffu), e = b_before + (before >> 16);
                const int t = t0 + 8 * q, j = divide(t, p.block);
                const int slot = __ldg(table + j) * p.bs + (t - j * p.bs);
#pragma unroll
                for (int i = 0; i < 8; i++) {
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
                }
            }
            o_before += all & 0xffffu;
            b_before += all >> 16;
        }
    }
    for (int i = rank * kSelThreads + tid; i < p.recent; i += C * kSelThreads) {
        const int t = old + i, j = divide(t, p.block);
        src[want + i] = __ldg(table + j) * p.bs + (t - j * p.bs);
    }
    first = __reduce_min_sync(FULL, first);
    if (lane == 0)
        atomicMin(C > 1 ? cluster.map_shared_rank(&S.first, 0) : &S.first, first);
    sync_all();  // also: no CTA of a cluster leaves before the others are done with it
    if (lead)
        *moved = make_int2(S.first, p.budget);
}

// Copies tokens [first, end) of one (sequence, KV head): `lanes` threads take a
// token, thread i of them its i-th unit; src lists the slots they come from,
// slot_of gives a position's slot; get reads a slot, put writes it.
// Double-buffered tiles, sources looked up one tile further ahead.
template <typename T, typename Slot, typename Get, typename Put>
__device__ __forceinline__ void move_tiles(int first, int end, int lanes, const int32_t *src,
                                           Slot slot_of, Get get, Put put)
{
    const int rows = (int)blockDim.x / lanes;  // tokens per step
    const int tile = rows * kMoveDepth;
    const int r = (int)threadIdx.x / lanes;
    int si[kMoveDepth], di[kMoveDepth];
    T x[2][kMoveDepth];
    auto sources = [&](int j0) {
#pragma unroll
        for (int i = 0; i < kMoveDepth; i++) {
            const int j = j0 + r + i * rows;
            si[i] = j < end ? __ldg(src + j) : -1;
        }
    };
    auto read = [&](T (&to)[kMoveDepth]) {
#pragma unroll
        for (int i = 0; i < kMoveDepth; i++)
            if (si[i] >= 0)
                to[i] = get(si[i]);
    };
    sources(first);
    read(x[0]);
    sources(first + tile);
    for (int j0 = first; j0 < end; j0 += 2 * tile) {
#pragma unroll
        for (int u = 0; u < 2; u++) {
            const int at = j0 + u * tile;
            if (at < end) {  // the same for the whole CTA
#pragma unroll
                for (int i = 0; i < kMoveDepth; i++) {
                    const int j = at + r + i * rows;
                    di[i] = j < end ? slot_of(j) : -1;
                }
                read(x[u ^ 1]);          // tile at + tile: its sources lie past this tile
                sources(at + 2 * tile);
                __syncthreads();         // this tile is in every thread's registers
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
    // here, not in the selection: its CTAs all read the lengths, and out_lens may be
    // (or overlap) context_lens
    if (slice == 0 && h == 0 && threadIdx.x == 0)
        p.out_lens[b] = moved.y;
    if (moved.x >= moved.y)
        return;
    const int32_t *src = p.ws_src + ((size_t)b * p.Hkv + h) * p.keep;
    const int32_t *table = p.block_tables + (size_t)b * p.MBS;
    auto slot_of = [&](int t) {
        const int j = divide(t, p.block);
        return __ldg(table + j) * p.bs + (t - j * p.bs);
    };
    if (slice == p.slices) {  // the weights, fp32 [NB, Hkv, bs]
        auto at = [&](int slot) {
            const int blk = divide(slot, p.block);
            return p.weights + ((size_t)blk * p.Hkv + h) * p.bs + (slot - blk * p.bs);
        };
        move_tiles<float>(
            moved.x, moved.y, 1, src, slot_of, [&](int slot) { return *at(slot); },
            [&](int slot, float w) { *at(slot) = w; });
        return;
    }
    // this CTA's units of every row: K's are 0 .. units - 1, V's the next
    const int per = 2 * p.units / p.slices;  // a power of two
    const int u0 = slice * per + (int)(threadIdx.x % per);
    uint4 *base = (u0 < p.units ? p.k_cache : p.v_cache) + (size_t)h * p.units + u0 % p.units;
    const size_t row = (size_t)p.Hkv * p.units;
    move_tiles<uint4>(
        moved.x, moved.y, per, src, slot_of, [&](int slot) { return base[(size_t)slot * row]; },
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
    cfg.blockDim = dim3((unsigned)p.move_threads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, evict_move_kernel, p);
}

} // namespace pkv
