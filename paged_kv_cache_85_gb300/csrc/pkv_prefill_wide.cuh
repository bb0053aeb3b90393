// Paged prefill attention with 128-key tiles, for the call that also records
// attention weights (it leaves every row's log-sum-exp for pkv_prompt_weights.cu
// and clears the weights of the new tokens).
//
// What it computes, its work items, their order, its precision (scores in bf16,
// P.V in f16, fp32 sums) and its flags are those of pkv_prefill_tc.cuh; the
// rounding of P differs where the running max moves at other keys.  What
// differs is the tile and with it the schedule:
//
//  * Key tiles of 128 (that kernel: 64).  A score MMA of N = 64 reads its 128
//    query rows from shared memory again for half the columns and runs at 48
//    cycles per 16 of the head dimension for 32 cycles of work; at N = 128 both
//    are 64.  Per pair of query tiles and 128 keys the tensor pipe has 2048
//    cycles of work, and shared memory (128 B a cycle) as many for the operands.
//  * One score buffer per query tile (128 columns; with the two outputs that is
//    all of TMEM).  P_t(j), 64 columns of f16 pairs, is written over S_t(j), so a
//    tile's chain is S_t(j) -> softmax -> P.V_t(j) -> S_t(j + 1); the other
//    tile's MMAs fill the pipe during its softmax.
//  * Nothing but the softmax lies on that chain: each softmax group converts its
//    half of V tile j + 1 to f16 right after P_t(j) is handed over, while the
//    MMAs P.V_t(j) and S_t(j + 1) run.
//  * A thread's 128 scores are read in two halves of 64: both for the maximum;
//    then the second half, still in registers, is exponentiated and its P
//    written over the last quarter of the score columns, and the first half is
//    read again and its P written over the first quarter.
//
//  * Few rows over long contexts (a short chunk on a long prefix) leave most SMs
//    without an item: the host then splits every item's key tiles over up to
//    p.splits CTAs.  Each leaves its rows' outputs (fp32) and log-sum-exps in
//    the workspace; pkv_prefill_join.cu puts them together.  So are the items of
//    an incomplete last round, where there are few rounds of long ones
//    (wide_split).
//
// Measured: 261 us for 8 sequences of 2048 new tokens (16 heads, 296 GFLOP: 1136
// TFLOP/s, tensor pipe 52%), where the 64-key kernel takes 298.  Bound by the
// chain above: 3200 cycles per pair of query tiles and 128 keys, of which a
// softmax group works 2700; an item's ends are another 7400.
//
// Warps (352 threads): 0..3 softmax of query tile A, 4..7 of tile B (thread =
// row = TMEM lane); 8 producer; 9, 10 the MMAs of tiles A and B.
// TMEM columns: O_A [0, D), O_B [128, 128 + D), S_A [256, 384), S_B [384, 512);
// P_t: keys 0..63 at S_t + 0, keys 64..127 at S_t + 96.
// Shared memory (D = 128): Q 64 KB, two stages of K and three of V, 32 KB each.
#pragma once

#include "pkv_prefill_tc.cuh"

namespace pkv {

// A lock in shared memory, taken by one thread per warp.
struct Turn {
    uint32_t *word;
    __device__ __forceinline__ bool take() const
    {
        uint64_t t0 = 0;
        while (atomicCAS_block(word, 0u, 1u) != 0u) {
            if (t0 == 0)
                t0 = sm_clock();
            else if (sm_clock() - t0 > kPollLimitCycles)
                return false;
        }
        return true;
    }
    __device__ __forceinline__ void pass() const { atomicExch_block(word, 0u); }
};

constexpr int kWKeys = 128;
constexpr int kWKStages = 2;  // K ring
constexpr int kWVStages = 3;  // V ring: one more, a V tile is held from its copy through
                              // the conversion to the second query tile's P.V
// q_full[2], q_empty[2], k_full, k_empty [kWKStages] each, v_full, v_empty, v_conv
// [kWVStages] each, per query tile s_full, pv_ready[2 halves], pv_done, o_free,
// then item_ready[2], item_free[2], mma_done
constexpr int kWBars = 4 + 2 * kWKStages + 3 * kWVStages + 10 + 4 + 1;

// An item's share of the key tiles: tiles j0 .. j0 + nkt[t] - 1 of query tile t.
struct WideItem {
    PrefillItem f;
    int j0, split;
    int clean;  // V's codes come without NaN (the kernel over scaled E4M3 caches)
    int pad;
};

struct WideSmem {
    size_t q, k, v, bars, items, slot, total;
};

__host__ __device__ inline WideSmem wide_smem_layout(int D)
{
    WideSmem L;
    size_t o = 0;
    L.q = o;  // [tile][D/64 halves][128 rows][128 B]
    o += (size_t)2 * (D / 64) * kTcRows * 128;
    L.k = o;  // stages of [D/64 halves][128 keys][128 B]
    o += (size_t)kWKStages * (D / 64) * kWKeys * 128;
    L.v = o;  // stages of [64-key run, or 16-key box][D/64 halves][keys][128 B]
    o += (size_t)kWVStages * (D / 64) * kWKeys * 128;
    L.bars = o;
    o += 8 * kWBars;
    L.items = align_up(o, 16);  // two published work items
    o = L.items + 2 * sizeof(WideItem);
    L.slot = o;  // TMEM base, and the MMA warps' lock
    o += 16;
    L.total = align_up(o, 16) + 1024;
    if (L.total < kTcMinSmem)
        L.total = kTcMinSmem;
    return L;
}

// SPLIT: p.splits > 1.  Of its own, for the others' items are 4% slower with it
// where they are short.
template <int D, int G, bool SPLIT>
__global__ void __launch_bounds__(kTcThreads, 1)
    paged_prefill_wide_kernel(const __grid_constant__ CUtensorMap tmq,
                              const __grid_constant__ CUtensorMap tmk,
                              const __grid_constant__ CUtensorMap tmv, const PrefillParams p)
{
    constexpr int TPC = kTcRows / G;               // query tokens per tile
    constexpr int HALVES = D / 64;
    constexpr uint32_t kQHalf = kTcRows * 128;     // 16 KB
    constexpr uint32_t kQTile = HALVES * kQHalf;
    constexpr uint32_t kKHalf = kWKeys * 128;      // 16 KB
    constexpr uint32_t kTile = HALVES * kKHalf;    // one K (or V) tile
    constexpr uint32_t kBoxBytes = kBox * D * 2;
    constexpr int kBoxes = kWKeys / kBox;          // 16-token boxes per tile
    constexpr unsigned FULL = 0xffffffffu;
    constexpr float kLazy = 8.f;
    const int splits = SPLIT ? p.splits : 1, whole = SPLIT ? p.whole : 0;
    const long long units = SPLIT ? whole + (long long)(p.n_items - whole) * splits : p.n_items;

    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const WideSmem L = wide_smem_layout(D);
    uint64_t *q_full = reinterpret_cast<uint64_t *>(smem + L.bars);  // [2] Q tile t landed
    uint64_t *q_empty = q_full + 2;               // [2] tile t's last S of the item completed
    uint64_t *k_full = q_empty + 2;
    uint64_t *k_empty = k_full + kWKStages;       // both tiles' S of the K tile completed
    uint64_t *v_full = k_empty + kWKStages;
    uint64_t *v_empty = v_full + kWVStages;       // both tiles' P.V of the V tile completed
    uint64_t *v_conv = v_empty + kWVStages;       // the V tile converted to f16 (8 warps)
    uint64_t *s_full = v_conv + kWVStages;        // [2] S_t written
    uint64_t *pv_ready = s_full + 2;              // [half of the keys][2] P_t written (4 warps)
    uint64_t *pv_done = pv_ready + 4;             // [2] P.V_t completed
    uint64_t *o_free = pv_done + 2;               // [2] O_t read out by its epilogue (4 warps)
    uint64_t *item_ready = o_free + 2;            // [2] item parameters published
    uint64_t *item_free = item_ready + 2;         // [2] ... no longer needed
    uint64_t *mma_done = item_free + 2;           // every MMA of the CTA completed
    uint32_t *slot = reinterpret_cast<uint32_t *>(smem + L.slot);
    const Turn turn{slot + 1};
    WideItem *items = reinterpret_cast<WideItem *>(smem + L.items);
    uint8_t *sQ = smem + L.q, *sK = smem + L.k, *sV = smem + L.v;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_launch_dependents();
    if (warp == kTcProducerWarp && lane == 0) {
        for (int t = 0; t < 2; t++) {
            mbar_init(&q_full[t], 1);
            mbar_init(&q_empty[t], 1);
            mbar_init(&s_full[t], 1);
            mbar_init(&pv_ready[t], 4);
            mbar_init(&pv_ready[2 + t], 4);
            mbar_init(&pv_done[t], 1);
            mbar_init(&o_free[t], 4);
            mbar_init(&item_ready[t], 1);
            mbar_init(&item_free[t], 10);  // two MMA warps, eight softmax warps
        }
        for (int s = 0; s < kWKStages; s++) {
            mbar_init(&k_full[s], 1);
            mbar_init(&k_empty[s], 2);  // both MMA warps
        }
        for (int s = 0; s < kWVStages; s++) {
            mbar_init(&v_full[s], 1);
            mbar_init(&v_empty[s], 2);
            mbar_init(&v_conv[s], 8);
        }
        mbar_init(mma_done, 2);
        *turn.word = 0;
        fence_mbarrier_init();
    } else if (warp == kTcMmaWarp) {
        tc::alloc(smem_u32(slot), kTcCols);
        tc::relinquish();
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = *slot;
    const int nC = (int)gridDim.x;
    const int c = (int)blockIdx.x;

    if (warp == kTcProducerWarp) {
        // ------------------------------------------------------------ producer
        if (lane == 0) {
            prefetch_tensormap(&tmq);
            prefetch_tensormap(&tmk);
            prefetch_tensormap(&tmv);
        }
        grid_dependency_wait();  // K/V may have just been written by store_kvcache
        if (p.ticket && c == 0) {  // the weights kernel's counters
            if (lane == 0)
                *p.ticket = 0;
            for (int i = lane; p.pw_count && i < kPwFewUnits * 8; i += 32)
                p.pw_count[i] = 0;
        }
        int gk = 0, gv = 0;       // K and V tiles issued so far (all items)
        int q_loads[2] = {0, 0};  // Q tiles A and B loaded so far
        bool ok = true;
        int n = 0;                // items published
        int k = 0;                // walk rounds
        for (;;) {
            // ---- the next item with work (round k: forward, then backward), or the end
            WideItem item{{-1, 0, 0, 0, 0, 0, {0, 0}}, 0, 0, 0, 0};
            PrefillItem &it = item.f;
            for (; ok; k++) {
                const long long at = (long long)k * nC + ((k & 1) ? nC - 1 - c : c);
                if (at >= units)
                    break;
                // the split items' first pieces, then their second ones: items that turn
                // out too short to be split fill the SMs like any others
                int pos = (int)at, piece = -1;
                if (SPLIT && at >= whole) {
                    piece = ((int)at - whole) / (p.n_items - whole);
                    pos -= piece * (p.n_items - whole);
                }
                const PrefillWork w = p.B <= 32 ? prefill_schedule<2 * TPC, 1>(p, lane, pos)
                                                : prefill_schedule<2 * TPC, kSchedChunks>(p, lane, pos);
                int cq0 = w.cq0, cq1 = w.cq1, ck0 = w.ck0, ck1 = w.ck1;
                if (w.b >= 0 && cq0 == kNotLoaded) {
                    cq0 = __ldg(p.cu_q + w.b);
                    cq1 = __ldg(p.cu_q + w.b + 1);
                    ck0 = __ldg(p.cu_k + w.b);
                    ck1 = __ldg(p.cu_k + w.b + 1);
                }
                const bool sane = w.b >= 0 && prefill_seq_sane(p, cq0, cq1, ck0, ck1);
                if (w.b >= 0 && !sane && lane == 0)
                    flag_error(p.err_flag, 0x4 /* PKV_FLAG_BAD_CONTEXT_LEN */);
                const int tok0 = w.tile * 2 * TPC;
                if (sane && tok0 < cq1 - cq0) {
                    it.kvh = w.kvh;
                    it.tok0 = tok0;
                    it.cq0 = cq0;
                    it.q_len = cq1 - cq0;
                    it.k_len = ck1 - ck0;
                    const int base = it.k_len - it.q_len;
                    it.nkt[0] = (base + min(it.q_len, tok0 + TPC) - 1) / kWKeys + 1;
                    it.nkt[1] = tok0 + TPC < it.q_len
                                    ? (base + min(it.q_len, tok0 + 2 * TPC) - 1) / kWKeys + 1
                                    : 0;
                    if constexpr (SPLIT)
                        item.split = -1;
                    if (SPLIT && piece >= 0) {
                        const int nkt = max(it.nkt[0], it.nkt[1]);
                        const int chunk = wide_chunk(nkt, splits, p.least);
                        item.j0 = piece * chunk;
                        if (item.j0 >= nkt)
                            continue;  // the item has fewer splits
                        if (nkt > chunk) {
                            item.split = piece;
                            for (int t = 0; t < 2; t++)
                                it.nkt[t] = min(max(it.nkt[t] - item.j0, 0), chunk);
                        }
                    }
                    it.b = w.b;
                    k++;
                    break;
                }
                // up to kSchedMaxSeqs sequences, ranks are longest first, so
                // the first empty item ends this CTA's work (but for further pieces)
                if (!SPLIT && p.B <= kSchedMaxSeqs && w.b < 0) {
                    k = 0x3fffffff;
                    break;
                }
            }
            // ---- publish it in slot n & 1, once the item two back is done with it
            const int sl = n & 1;
            if (n >= 2 && !(ok = ok && __all_sync(FULL, mbar_wait(&item_free[sl], ((n >> 1) & 1) ^ 1))))
                break;  // the other warps time out on item_ready and stop
            if (!ok)
                it.b = -1;
            if (lane == 0) {
                items[sl] = item;
                mbar_arrive(&item_ready[sl]);
            }
            __syncwarp();
            if (it.b < 0)
                break;
            // ---- the item's new tokens start from weight 0: the weights kernel, which
            // waits for this one, only adds (to blocks that other sequences may share).
            // Here, where the producer would wait for the last item's Q: 16k step 411 ->
            // 415 us; after the item's last copy 420, by the softmax threads 422.
            if (!SPLIT || item.split <= 0) {
                const int t0 = it.k_len - it.q_len + it.tok0, nt = min(2 * TPC, it.q_len - it.tok0);
                for (int i = lane; i < nt; i += 32) {
                    const int t = t0 + i, blk = __ldg(p.block_tables + (size_t)it.b * p.MBS + t / p.bs);
                    if (blk >= 0 && blk < p.NB)
                        p.weights[((size_t)blk * p.Hkv + it.kvh) * p.bs + t % p.bs] = 0.f;
                }
            }
            // ---- Q tiles, each once its tile's last S of the previous item completed
            for (int t = 0; t < 2 && ok; t++) {
                if (it.nkt[t] == 0)
                    continue;
                if (n >= 1 && !(ok = __all_sync(FULL, mbar_wait(&q_empty[t], (n - 1) & 1))))
                    break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&q_full[t], HALVES * kQHalf);
#pragma unroll
                    for (int h = 0; h < HALVES; h++)
                        tma_load_4d(sQ + t * kQTile + h * kQHalf, &tmq, 0, h, it.kvh * G,
                                    it.cq0 + it.tok0 + t * TPC, &q_full[t]);
                }
                ++q_loads[t];
            }
            if (!ok)
                break;
            n++;
            // ---- K and V tiles through the two rings: whichever can go.  Lanes 0-7
            // resolve one 16-token box each, a tile ahead of its copy.
            const int nkt = max(it.nkt[0], it.nkt[1]);
            const int j0 = SPLIT ? item.j0 : 0;
            const int32_t *table = p.block_tables + (size_t)it.b * p.MBS;
            auto entry = [&](int j) -> int {
                const int key0 = (j0 + j) * kWKeys + lane * kBox;
                return (lane < kBoxes && j < nkt && key0 < it.k_len) ? __ldg(table + key0 / p.bs) : -1;
            };
            int next_k = entry(0), next_v = next_k;
            // tokens per copy: a 64-token run where blocks hold whole runs, else a box
            const int per = p.tile_copies ? kPrefillKeys : kBox;
            auto issue = [&](int j, int g, bool is_k) {
                uint64_t *fb = is_k ? k_full : v_full;
                const int s = g % (is_k ? kWKStages : kWVStages);
                const int blk = is_k ? next_k : next_v;
                (is_k ? next_k : next_v) = entry(j + 1);
                const int key0 = (j0 + j) * kWKeys + lane * kBox;
                int row = -1;
                if (lane < kBoxes && key0 < it.k_len) {
                    if (blk >= 0 && blk < p.NB)
                        row = blk * p.bs + key0 % p.bs;
                    else
                        flag_error(p.err_flag, 0x2 /* PKV_FLAG_BAD_BLOCK */);
                }
                // rows past k_len of a run come along: their scores are masked and
                // their V rows zeroed
                const bool copies = row >= 0 && (lane * kBox) % per == 0;
                const uint32_t mask = __ballot_sync(FULL, copies);
                if (lane == 0)
                    mbar_arrive_expect_tx(&fb[s], (uint32_t)__popc(mask) * per * D * 2);
                __syncwarp();
                if (copies) {
                    if (is_k) {
                        // K: [half][128 rows], one stride along the keys
#pragma unroll
                        for (int h = 0; h < HALVES; h++)
                            tma_load_4d(sK + (size_t)s * kTile + h * kKHalf + lane * (kBox * 128), &tmk, 0, h,
                                        it.kvh, row, &fb[s]);
                    } else {
                        // V: one copy per run or box, both halves
                        tma_load_4d(sV + (size_t)s * kTile + lane * kBoxBytes, &tmv, 0, row, it.kvh, 0,
                                    &fb[s]);
                    }
                }
            };
            int jk = 0, jv = 0;
            uint64_t t_last = sm_clock();
            while (jk < nkt || jv < nkt) {
                bool prog = false;
                if (jk < nkt) {
                    const bool free_k = tc::test_wait(smem_u32(&k_empty[gk % kWKStages]),
                                                      ((gk / kWKStages) & 1) ^ 1);
                    if (__shfl_sync(FULL, free_k, 0)) {
                        issue(jk++, gk++, true);
                        prog = true;
                    }
                }
                if (jv < jk) {
                    const bool free_v = tc::test_wait(smem_u32(&v_empty[gv % kWVStages]),
                                                      ((gv / kWVStages) & 1) ^ 1);
                    if (__shfl_sync(FULL, free_v, 0)) {
                        issue(jv++, gv++, false);
                        prog = true;
                    }
                }
                if (prog) {
                    t_last = sm_clock();
                } else {
                    __nanosleep(32);
                    if (__shfl_sync(FULL, sm_clock() - t_last > kPollLimitCycles, 0)) {
                        ok = false;
                        break;
                    }
                }
            }
            if (!ok)
                break;  // the other warps time out on their barriers and stop
        }
        if (lane == 0) {
            if (!ok)
                flag_error(p.err_flag, 0x8 /* PKV_FLAG_TIMEOUT */);
            // copies still in flight land before the CTA may exit
            for (int t = 0; t < 2; t++)
                if (q_loads[t] >= 1)
                    mbar_wait(&q_full[t], (q_loads[t] - 1) & 1);
            for (int g = max(0, gk - kWKStages); g < gk; g++)
                mbar_wait(&k_full[g % kWKStages], (g / kWKStages) & 1);
            for (int g = max(0, gv - kWVStages); g < gv; g++)
                mbar_wait(&v_full[g % kWVStages], (g / kWVStages) & 1);
        }
        __syncwarp();
    } else if (warp == kTcMmaWarp || warp == kTcMmaWarp + 1) {
        // ----------------------------------------------------------------- MMA
        // One warp per query tile t.  Per key tile j: P.V_t(j), then, once it has
        // read P_t(j), S_t(j + 1) into the same buffer.  The two warps take turns (a
        // lock in shared memory) with such a pair: a tile's MMAs then run back to
        // back while the other tile's softmax works.  Without it both tiles' MMAs
        // share the pipe, both softmax groups get their scores at the same time, and
        // the pipe idles while both work (4707 cycles per pair of tiles and 128 keys).
        // A K, V or Q stage is released by one arrival per query tile: V by this warp,
        // which waits for its P.V, K and Q by the softmax group as it finds S_t(j), or
        // by this warp, for a stage its tile does not read, once that stage's tile has
        // landed (so that the arrival counts towards that tile's phase).  Plain
        // arrivals: each further commit costs the issuing thread about 100 cycles.
        const int t = warp - kTcMmaWarp;
        bool ok = true;
        const uint32_t qt = smem_u32(sQ) + (uint32_t)t * kQTile;
        // a negative scale is applied by negating Q (bit 13 of the descriptor)
        const uint32_t idS = tc::idesc_bf16(kTcRows, kWKeys, false) | (p.neg_scale ? 1u << 13 : 0u);
        const uint32_t idO = tc::idesc_f16(kTcRows, D, true);
        const uint32_t dS = tmem + 256u + 128u * (uint32_t)t, dO = tmem + 128u * (uint32_t)t;
        // 16 keys of a V tile: two 64-column halves v_lbo apart
        const uint32_t v_lbo = p.tile_copies ? (uint32_t)kPrefillKeys * 128 : (uint32_t)kBox * 128;
        if (tc::elect_one()) {
            int g0 = 0;    // K/V tiles of the previous items
            int gq = 0;    // S/P tiles of this query tile so far
            int used = 0;  // items in which this query tile had work
            for (int n = 0; ok; n++) {
                if (!(ok = mbar_wait(&item_ready[n & 1], (n >> 1) & 1)))
                    break;
                const PrefillItem it = items[n & 1].f;
                if (it.b < 0)
                    break;
                const int nk = it.nkt[t];
                const int nkt = max(it.nkt[0], it.nkt[1]);
                if (nk > 0 && !(ok = mbar_wait(&q_full[t], used & 1)))
                    break;
                tc::fence_after();
                if (nk == 0)
                    mbar_arrive(&q_empty[t]);  // this tile reads no Q this item
                // S_t(j), its K tile landed and S_t's buffer free
                auto scores = [&](int j) {
                    const int s = (g0 + j) % kWKStages;
                    tc::fence_after();
                    const uint32_t ka = smem_u32(sK + (size_t)s * kTile);
#pragma unroll
                    for (int kq = 0; kq < D / 16; kq++) {
                        const uint32_t off = (uint32_t)(kq >> 2) * kQHalf + (uint32_t)(kq & 3) * 32;
                        tc::mma_ss(dS, tc::smem_desc(qt + off, 16, 1024), tc::smem_desc(ka + off, 16, 1024),
                                   idS, kq > 0);
                    }
                    tc::commit(smem_u32(&s_full[t]));
                };
                auto landed = [&](int j) {
                    return mbar_wait(&k_full[(g0 + j) % kWKStages], ((g0 + j) / kWKStages) & 1);
                };
                if (nk > 0) {
                    // the buffer is free: this warp saw the previous item's last P.V complete
                    if (!(ok = landed(0)) || !(ok = turn.take()))
                        break;
                    scores(0);
                    turn.pass();
                }
                for (int j = 0; j < nk; j++) {
                    // P.V_t(j) once P_t(j) is written and V tile j converted; and, so that
                    // nothing is waited for that the other warp may owe while the turn is
                    // held, K tile j + 1 landed
                    const int s = (g0 + j) % kWVStages;
                    if (!(ok = mbar_wait(&v_conv[s], ((g0 + j) / kWVStages) & 1)))
                        break;
                    // the item's first P.V overwrites O: the tile's previous epilogue
                    // must have read it out
                    if (j == 0 && used >= 1 && !(ok = mbar_wait(&o_free[t], (used - 1) & 1)))
                        break;
                    if (j + 1 < nk && !(ok = landed(j + 1)))
                        break;
                    // keys 64 .. 127 first: their P is written first, and their MMAs run
                    // while the softmax is at the other half
                    const uint32_t va = smem_u32(sV + (size_t)s * kTile);
                    auto pv = [&](int half, bool add) {
                        tc::fence_after();
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            const int kk = 4 * half + i;
                            const uint32_t vk = p.tile_copies ? (uint32_t)half * (kPrefillKeys * 128 * HALVES) +
                                                                    (uint32_t)i * 2048
                                                              : (uint32_t)kk * kBoxBytes;
                            tc::mma_ts(dO, dS + 96u * half + 8u * i, tc::smem_desc(va + vk, v_lbo, 1024), idO,
                                       (add || i > 0) ? 1u : 0u);
                        }
                    };
                    if (!(ok = mbar_wait(&pv_ready[2 + t], gq & 1)) || !(ok = turn.take()))
                        break;
                    pv(1, j > 0);
                    turn.pass();
                    if (!(ok = mbar_wait(&pv_ready[t], gq & 1)) || !(ok = turn.take()))
                        break;
                    pv(0, true);
                    tc::commit(smem_u32(&pv_done[t]));
                    // S_t(j + 1) overwrites P_t(j)
                    ok = mbar_wait(&pv_done[t], gq & 1);
                    gq++;
                    if (ok) {
                        mbar_arrive(&v_empty[s]);
                        if (j + 1 < nk)
                            scores(j + 1);
                    }
                    turn.pass();
                    if (!ok)
                        break;
                }
                // K and V tiles that this query tile does not read
                for (int j = nk; ok && j < nkt; j++) {
                    const int s = (g0 + j) % kWVStages;
                    if (!(ok = landed(j)))
                        break;
                    mbar_arrive(&k_empty[(g0 + j) % kWKStages]);
                    if (!(ok = mbar_wait(&v_conv[s], ((g0 + j) / kWVStages) & 1)))
                        break;
                    mbar_arrive(&v_empty[s]);
                }
                if (!ok)
                    break;
                g0 += nkt;
                used += nk > 0 ? 1 : 0;
                mbar_arrive(&item_free[n & 1]);
            }
            if (!ok)
                flag_error(p.err_flag, 0x8 /* PKV_FLAG_TIMEOUT */);
            tc::commit(smem_u32(mma_done));  // every MMA completes before TMEM is released
        }
        __syncwarp();
        mbar_wait(mma_done, 0);
        __syncwarp();
    } else {
        // ------------------------------------------------------------- softmax
        const int tq = warp >> 2;            // query tile of this group (A = 0, B = 1)
        const int r = threadIdx.x & 127;     // row = TMEM lane
        const uint32_t tl = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t tO = tmem + 128u * tq + tl, tS = tmem + 256u + 128u * tq + tl;
        const float sl = p.scale_log2;
        const float2 sl2 = make_float2(sl, sl);
        bool ok = true;
        int g0 = 0, gq = 0;
        for (int n = 0; ok; n++) {
            ok = __all_sync(FULL, mbar_wait(&item_ready[n & 1], (n >> 1) & 1));
            if (!ok)
                break;
            const WideItem item = items[n & 1];
            const PrefillItem &it = item.f;
            if (it.b < 0)
                break;
            const int nkt = it.nkt[tq], all = max(it.nkt[0], it.nkt[1]);
            const int j0 = SPLIT ? item.j0 : 0;
            const int tok = it.tok0 + tq * TPC + r / G, g = r % G;
            const bool valid = tok < it.q_len;
            const int pos = (it.k_len - it.q_len) + tok;
            const int32_t *table = p.block_tables + (size_t)it.b * p.MBS;
            const int k_len = it.k_len;
            float m = -INFINITY, l = 0.f;
            uint32_t vmax = 0;  // f16 magnitudes of the converted V rows, max per half
            // boxes of a tile that the producer loads (block ids in [0, NB)); lanes 0-7
            // read the entries a tile ahead
            auto table_entry = [&](int j) -> int {
                const int key0 = (j0 + j) * kWKeys + lane * kBox;
                return (lane < kBoxes && j < all && key0 < k_len) ? __ldg(table + key0 / p.bs) : -1;
            };
            auto loaded = [&](int blk) { return __ballot_sync(FULL, blk >= 0 && blk < p.NB) & 0xffu; };
            // This group's half (64 keys) of V tile j: bf16 -> f16 in place, rows past
            // k_len or of unloaded boxes zeroed (their weight is 0, and 0 * NaN would be
            // NaN).  Both groups take part in every V tile of the item, in order.
            auto convert_v = [&](int j, uint32_t boxes) -> bool {
                const int gv = g0 + j, s = gv % kWVStages, kb = (j0 + j) * kWKeys + 64 * tq;
                if (!__all_sync(FULL, mbar_wait(&v_full[s], (gv / kWVStages) & 1)))
                    return false;
                uint4 *vt = reinterpret_cast<uint4 *>(sV + (size_t)s * kTile + tq * (kTile / 2));
                const uint32_t mine = (boxes >> (4 * tq)) & 0xfu;
                const bool clear = mine != 0xfu || kb + 64 > k_len;
                constexpr int NCH = HALVES * 64 * 8 / 128;  // 16-byte chunks per thread
                uint4 w[NCH];
#pragma unroll
                for (int u = 0; u < NCH; u++)
                    w[u] = vt[r + 128 * u];
#pragma unroll
                for (int u = 0; u < NCH; u++) {
                    w[u].x = bf16x2_to_f16x2_sat(w[u].x);
                    w[u].y = bf16x2_to_f16x2_sat(w[u].y);
                    w[u].z = bf16x2_to_f16x2_sat(w[u].z);
                    w[u].w = bf16x2_to_f16x2_sat(w[u].w);
                }
                if (clear) {
#pragma unroll
                    for (int u = 0; u < NCH; u++) {
                        const int ci = r + 128 * u;
                        const int kr = p.tile_copies ? (ci / 8) % 64
                                                     : (ci / (8 * kBox * HALVES)) * kBox + (ci / 8) % kBox;
                        if (kb + kr >= k_len || !((mine >> (kr / kBox)) & 1u))
                            w[u] = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
#pragma unroll
                for (int u = 0; u < NCH; u++) {
                    vmax = f16x2_absmax(vmax, f16x2_absmax(f16x2_absmax(w[u].x, w[u].y),
                                                           f16x2_absmax(w[u].z, w[u].w)));
                    vt[r + 128 * u] = w[u];
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&v_conv[s]);
                return true;
            };
            uint32_t boxes = loaded(table_entry(0));
            int blk_next = table_entry(1);
            if (!(ok = convert_v(0, boxes)))
                break;
            for (int j = 0; j < nkt; j++) {
                const int gt = gq + j;
                const uint32_t boxes_next = loaded(blk_next);
                blk_next = table_entry(j + 2);
                ok = __all_sync(FULL, mbar_wait(&s_full[tq], gt & 1));
                if (!ok)
                    break;
                tc::fence_after();
                // S_t(j) has completed: its K tile, and after the item's last one its
                // Q, is read
                if ((warp & 3) == 0 && lane == 0) {
                    mbar_arrive(&k_empty[(g0 + j) % kWKStages]);
                    if (j == nkt - 1)
                        mbar_arrive(&q_empty[tq]);
                }
                const int key_base = (j0 + j) * kWKeys;
                // masked keys: past this row's position (the diagonal tiles) or in an
                // unloaded box; most tiles have none in the whole warp
                const bool any_masked = __any_sync(FULL, boxes != 0xffu || key_base + kWKeys - 1 > pos);
                const int lim = pos - key_base;  // keys i > lim are in the future
                float x[64];
                auto load = [&](int half) {
                    uint32_t a[32], b[32];
                    tc::ld32(tS + 64 * half, a);
                    tc::ld32(tS + 64 * half + 32, b);
                    tc::wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; i++) {
                        x[i] = __uint_as_float(a[i]);
                        x[32 + i] = __uint_as_float(b[i]);
                    }
                    if (any_masked) {
                        const uint32_t hb = boxes >> (4 * half);
#pragma unroll
                        for (int i = 0; i < 64; i++)
                            x[i] = (64 * half + i > lim || !((hb >> (i / kBox)) & 1u)) ? -INFINITY : x[i];
                    }
                };
                auto top = [&]() {
                    float t8[8];
#pragma unroll
                    for (int i = 0; i < 8; i++)
                        t8[i] = x[i];
#pragma unroll
                    for (int i = 8; i < 64; i++)
                        t8[i & 7] = fmaxf(t8[i & 7], x[i]);
                    return fmaxf(fmaxf(fmaxf(t8[0], t8[1]), fmaxf(t8[2], t8[3])),
                                 fmaxf(fmaxf(t8[4], t8[5]), fmaxf(t8[6], t8[7])));
                };
                load(0);
                float mraw = top();
                load(1);
                mraw = fmaxf(mraw, top());
                const float mx = mraw == -INFINITY ? -INFINITY : mraw * sl;
                if (__any_sync(FULL, mx > m + kLazy)) {
                    const float mn = fmaxf(m, mx);
                    const float alpha = mn == -INFINITY ? 1.f : fast_exp2(m - mn);
                    if (j > 0) {
                        // O holds P_0..P_{j-1} V: S_t(j) was issued after P.V_t(j - 1)
                        // completed, and the next P.V waits for this group's P
#pragma unroll 1
                        for (int cc = 0; cc < D / 32; cc++) {
                            uint32_t ro[32];
                            tc::ld32(tO + 32 * cc, ro);
                            tc::wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; i++)
                                ro[i] = __float_as_uint(__uint_as_float(ro[i]) * alpha);
                            tc::st32(tO + 32 * cc, ro);
                        }
                        tc::wait_st();
                    }
                    l *= alpha;
                    m = mn;
                }
                const float nmu = m == -INFINITY ? 0.f : -m;
                const float2 nm2 = make_float2(nmu, nmu);
                float2 ls0 = make_float2(0.f, 0.f), ls1 = ls0;
                auto exponentiate = [&](uint32_t to) {
                    uint32_t pk[32];
                    if (!any_masked) {
#pragma unroll
                        for (int i = 0; i < 32; i++) {
                            const float2 a = ffma2(make_float2(x[2 * i], x[2 * i + 1]), sl2, nm2);
                            const float2 e = make_float2(fast_exp2(a.x), fast_exp2(a.y));
                            if (i & 1)
                                ls1 = fadd2(ls1, e);
                            else
                                ls0 = fadd2(ls0, e);
                            pk[i] = pack_f16x2(e.x, e.y);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; i++) {
                            float2 a = ffma2(make_float2(x[2 * i], x[2 * i + 1]), sl2, nm2);
                            // exact zeros for masked keys (also when the scale is 0)
                            a.x = x[2 * i] == -INFINITY ? -INFINITY : a.x;
                            a.y = x[2 * i + 1] == -INFINITY ? -INFINITY : a.y;
                            const float2 e = make_float2(fast_exp2(a.x), fast_exp2(a.y));
                            if (i & 1)
                                ls1 = fadd2(ls1, e);
                            else
                                ls0 = fadd2(ls0, e);
                            pk[i] = pack_f16x2(e.x, e.y);
                        }
                    }
                    tc::st32(to, pk);
                };
                auto hand_over = [&](int half) {
                    tc::wait_st();
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&pv_ready[2 * half + tq]);
                };
                exponentiate(tS + 96);  // keys 64..127, over score columns read above
                hand_over(1);
                load(0);                // keys 0..63 again
                exponentiate(tS);
                l += (ls0.x + ls0.y) + (ls1.x + ls1.y);
                hand_over(0);
                // off the chain: V tile j + 1 while P.V_t(j) and S_t(j + 1) run
                if (j + 1 < all && !(ok = convert_v(j + 1, boxes_next)))
                    break;
                boxes = boxes_next;
            }
            if (!ok)
                break;
            // V tiles that only the other query tile reads
            for (int jv = max(nkt, 1) + (nkt > 0 ? 1 : 0); ok && jv < all; jv++) {
                const uint32_t bx = loaded(table_entry(jv));
                ok = convert_v(jv, bx);
            }
            if (!ok)
                break;
            // a converted V value was clamped to +-65504 (beyond f16's range): bf16
            // values at or below 65280 convert exactly, so only a clamp gives 0x7bff
            if ((vmax & 0x7fffu) >= 0x7bffu || ((vmax >> 16) & 0x7fffu) >= 0x7bffu)
                flag_error(p.err_flag, kFlagVRange);
            // a split that only the other query tile has keys in
            const bool piece = SPLIT && item.split >= 0;
            if (piece && nkt == 0 && valid)
                p.part_lse[(size_t)item.split * p.Tq * p.Hq +
                           ((size_t)it.kvh * p.Tq + it.cq0 + tok) * G + g] = -INFINITY;
            if (nkt > 0) {
                const int gl = gq + nkt - 1;
                ok = __all_sync(FULL, mbar_wait(&pv_done[tq], gl & 1));
                if (!ok)
                    break;
                tc::fence_after();
                const float inv = l > 0.f ? 1.f / l : 0.f;
                const size_t row = (size_t)it.cq0 + tok;
                const size_t lse_at = ((size_t)it.kvh * p.Tq + row) * G + g;
                if (piece) {
                    // this split's output in fp32, and its log-sum-exp (-inf: no key)
                    if (valid)
                        p.part_lse[(size_t)item.split * p.Tq * p.Hq + lse_at] =
                            l == 0.f ? -INFINITY : m + log2f(l);
                    float4 *dst = reinterpret_cast<float4 *>(
                        p.part_out + (((size_t)item.split * p.Tq + row) * p.Hq + it.kvh * G + g) * D);
#pragma unroll 1
                    for (int cc = 0; cc < D / 32; cc++) {
                        uint32_t ro[32];
                        tc::ld32(tO + 32 * cc, ro);
                        tc::wait_ld();
                        if (valid) {
#pragma unroll
                            for (int i = 0; i < 8; i++)
                                dst[8 * cc + i] = make_float4(__uint_as_float(ro[4 * i]) * inv,
                                                              __uint_as_float(ro[4 * i + 1]) * inv,
                                                              __uint_as_float(ro[4 * i + 2]) * inv,
                                                              __uint_as_float(ro[4 * i + 3]) * inv);
                        }
                    }
                } else {
                    // for the attention weights; +inf (weight 0) for a row that could
                    // read no key
                    if (valid) {
                        p.lse[lse_at] = l == 0.f ? INFINITY : m + log2f(l);
                        if (SPLIT)
                            p.part_lse[lse_at] = INFINITY;  // nothing to join
                    }
                    // 64 columns (eight 16-byte pieces) of a row at a time; eight lanes
                    // trade their rows' pieces (three butterfly steps), so that a store
                    // instruction writes whole 128-byte lines of four rows, not 16 bytes
                    // in each of 32 lines
#pragma unroll 1
                    for (int hf = 0; hf < HALVES; hf++) {
                        uint32_t ra[32], rb[32], v[32];
                        tc::ld32(tO + 64 * hf, ra);
                        tc::ld32(tO + 64 * hf + 32, rb);
                        tc::wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; i++) {
                            v[i] = pack_bf16x2(__uint_as_float(ra[2 * i]) * inv, __uint_as_float(ra[2 * i + 1]) * inv);
                            v[16 + i] = pack_bf16x2(__uint_as_float(rb[2 * i]) * inv,
                                                    __uint_as_float(rb[2 * i + 1]) * inv);
                        }
#pragma unroll
                        for (int s = 1; s < 8; s *= 2) {
                            const bool up = (lane & s) != 0;
#pragma unroll
                            for (int k = 0; k < 8; k++) {
                                if (k & s)
                                    continue;
#pragma unroll
                                for (int w = 0; w < 4; w++) {  // piece k of the upper lane for k + s of the lower
                                    const uint32_t give = up ? v[4 * k + w] : v[4 * (k + s) + w];
                                    const uint32_t got = __shfl_xor_sync(FULL, give, s);
                                    v[4 * k + w] = up ? got : v[4 * k + w];
                                    v[4 * (k + s) + w] = up ? v[4 * (k + s) + w] : got;
                                }
                            }
                        }
                        // this lane now has piece lane % 8 of the rows 8 (lane / 8) + k
#pragma unroll
                        for (int k = 0; k < 8; k++) {
                            const int rr = 32 * (warp & 3) + (lane & 24) + k;
                            const int tk = it.tok0 + tq * TPC + rr / G;
                            if (tk < it.q_len)
                                *reinterpret_cast<uint4 *>(
                                    p.out + (((size_t)it.cq0 + tk) * p.Hq + it.kvh * G + rr % G) * D + 64 * hf +
                                    8 * (lane & 7)) =
                                    make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
                        }
                    }
                }
                tc::fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&o_free[tq]);  // the tile's next first P.V may overwrite O
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&item_free[n & 1]);
            g0 += all;
            gq += nkt;
        }
        if (!ok && lane == 0)
            flag_error(p.err_flag, 0x8 /* PKV_FLAG_TIMEOUT */);
    }
    tc::fence_before();
    __syncthreads();
    if (warp == kTcMmaWarp) {
        tc::fence_after();
        tc::dealloc(tmem, kTcCols);
    }
}

template <int D>
inline cudaError_t launch_prefill_wide_d(int G, const CUtensorMap *tmq, const CUtensorMap *tmk,
                                         const CUtensorMap *tmv, const PrefillParams &p, dim3 grid,
                                         size_t smem, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kTcThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    switch (G) {
    case 1:
        return p.splits > 1 ? cudaLaunchKernelEx(&cfg, paged_prefill_wide_kernel<D, 1, true>, *tmq, *tmk, *tmv, p)
                            : cudaLaunchKernelEx(&cfg, paged_prefill_wide_kernel<D, 1, false>, *tmq, *tmk, *tmv, p);
    case 2:
        return p.splits > 1 ? cudaLaunchKernelEx(&cfg, paged_prefill_wide_kernel<D, 2, true>, *tmq, *tmk, *tmv, p)
                            : cudaLaunchKernelEx(&cfg, paged_prefill_wide_kernel<D, 2, false>, *tmq, *tmk, *tmv, p);
    case 4:
        return p.splits > 1 ? cudaLaunchKernelEx(&cfg, paged_prefill_wide_kernel<D, 4, true>, *tmq, *tmk, *tmv, p)
                            : cudaLaunchKernelEx(&cfg, paged_prefill_wide_kernel<D, 4, false>, *tmq, *tmk, *tmv, p);
    case 8:
        return p.splits > 1 ? cudaLaunchKernelEx(&cfg, paged_prefill_wide_kernel<D, 8, true>, *tmq, *tmk, *tmv, p)
                            : cudaLaunchKernelEx(&cfg, paged_prefill_wide_kernel<D, 8, false>, *tmq, *tmk, *tmv, p);
    default: return cudaErrorInvalidValue;
    }
}

template <int D> inline const void *prefill_wide_kernel_d(int G, bool split)
{
    switch (G) {
    case 1:
        return split ? reinterpret_cast<const void *>(&paged_prefill_wide_kernel<D, 1, true>)
                     : reinterpret_cast<const void *>(&paged_prefill_wide_kernel<D, 1, false>);
    case 2:
        return split ? reinterpret_cast<const void *>(&paged_prefill_wide_kernel<D, 2, true>)
                     : reinterpret_cast<const void *>(&paged_prefill_wide_kernel<D, 2, false>);
    case 4:
        return split ? reinterpret_cast<const void *>(&paged_prefill_wide_kernel<D, 4, true>)
                     : reinterpret_cast<const void *>(&paged_prefill_wide_kernel<D, 4, false>);
    case 8:
        return split ? reinterpret_cast<const void *>(&paged_prefill_wide_kernel<D, 8, true>)
                     : reinterpret_cast<const void *>(&paged_prefill_wide_kernel<D, 8, false>);
    default: return nullptr;
    }
}

} // namespace pkv
