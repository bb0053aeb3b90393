// Attention weights of a prefill step, added to the cache's weight table, on
// the 5th-generation tensor cores.
//
// The prefill kernel left every (new token, query head)'s log-sum-exp lse of
// its scores (log2 units).  The weight that token t of a sequence received
// from the recorded queries is
//     w[t] = sum over recorded new tokens i that see t, and over the G heads
//            of the group, of 2^(s[i, g, t] - lse[i, g]),
// which needs the final lse of every row, so the scores are made again here.
// It is added to weights[block, kv head, offset].  The slots of the step's new
// tokens, which may hold what an earlier owner left, were cleared by the prefill
// kernel: a block that is new to one sequence of the step may be another one's
// prefix, so that all additions to it have to come after that.
//
// The scores are made transposed, S^T = K Q^T with the cached tokens as the
// MMA's rows, so that a thread owns one token (a TMEM lane) and the sum over
// queries runs along its own columns: no reduction over threads, one addition
// to memory per token and KV head, and the same result in every run.  An item is
// 256 tokens (two MMA tiles A and B) of one sequence and KV head; the (new
// token, head) rows that see any of them pass by in tiles of 128.  Two token
// tiles per query tile halve the query rows read from L2 (32 KB per 128 x 128
// scores, 8 TB/s with one): 16k step 473 -> 446 us a call.
// Where there are fewer units of 256 tokens than SMs, their query tiles are
// split over several items; each leaves its tokens' partial sums in the
// workspace, and the last one to arrive adds them up in the order of the splits
// (the same result whoever is last).
// A persistent CTA per SM takes items by ticket (sequences in order, early
// tokens first, which are the long items of a causal chunk); the sum does not
// depend on who takes what.  Warps:
//   0..15 four groups of 128 threads, one per token tile and half of a query
//         tile's columns: load 64 scores per token from TMEM, exponentiate
//         against the tile's lse (shared memory, read as broadcasts), add up.
//         Partial sums per tile, then per item: no long sequential fp32 sum.
//         At the item's end the second half's sums go to the first's
//   16    producer: ticket, item, TMA of the K tiles (a ring of three, so that
//         the next item's are on their way) and of the query tiles (three)
//   17, 18 MMA, one warp per token tile (one thread cannot issue for both
//         without leaving the pipe idle): per query tile D / 16 steps of M = 128
//         (tokens), N = 128 (queries) into one of two TMEM buffers
//   19    the query tiles' log-sum-exps into a ring of four (by the softmax warps
//         themselves they cost 500 cycles per tile)
// Work per pair of 128 x 128 tiles and SM: 1024 cycles of 2^x (32 per cycle) and
// as many of MMA; it takes some 2000, the softmax groups' loads, exponentials and
// waits one after the other.  Measured: 144 us where every query of a 16k-token
// step records (148 GFLOP: 1028 TFLOP/s; tensor pipe and 2^x 54% each), 28 us
// where the last 32 of 32 ragged prompts do (72 MB read, 2.5 TB/s: items of one
// query tile, bound by their way through the warps).
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "pkv_kernels.h"
#include "pkv_prefill.h"
#include "pkv_ptx.cuh"
#include "pkv_tc.cuh"

namespace pkv {

constexpr int kPwTokens = 128;  // cached tokens per token tile (MMA M); two per item
constexpr int kPwRows = 128;    // (new token, head) rows per query tile (MMA N)
constexpr int kPwKStages = 3;
constexpr int kPwQStages = 3;
constexpr int kPwItems = 4;     // published items
constexpr int kPwSoftWarps = 16;
constexpr int kPwLseStages = 4;
constexpr int kPwThreads = (kPwSoftWarps + 4) * 32;
constexpr int kPwProducerWarp = kPwSoftWarps;
constexpr int kPwMmaWarp = kPwSoftWarps + 1;  // and the next, for token tile B
constexpr int kPwLseWarp = kPwSoftWarps + 3;

// 256 tokens of one sequence and KV head, and the query tiles that see them
struct PwItem {
    int b, kvh, t0;     // b < 0: no more work
    int cq0, q_len, k_len;
    int i0;             // first recorded new token that sees a token of the item
    int tiles;          // query tiles from i0 on
    int first1;         // the first of them that sees token tile B (tiles: none does)
    // where units (256 tokens of a sequence and KV head) are split over the queries:
    // this item is split `split` of `splits` of unit `unit`
    int unit, split, splits;
};

struct PwSmem {
    size_t q, k, lse, part, bars, items, slot, total;
};

constexpr int kPwBars = 2 * kPwKStages + 2 * kPwQStages + 8 + 2 * kPwItems + 32 + 2 * kPwLseStages + 1;

__host__ __device__ inline PwSmem pw_smem_layout(int D)
{
    PwSmem L;
    size_t o = 0;
    L.q = o;  // stages of [D/64 halves][128 rows][128 B]
    o += (size_t)kPwQStages * (D / 64) * kPwRows * 128;
    L.k = o;  // stages alike
    o += (size_t)kPwKStages * (D / 64) * kPwTokens * 128;
    L.lse = o;  // stages of [128] negated log-sum-exps of a query tile
    o += kPwLseStages * kPwRows * sizeof(float);
    L.part = o;  // [token tile][2][128] the second half's sums on their way to the first
    o += 2 * 2 * kPwTokens * sizeof(float);
    L.bars = o;
    o += 8 * kPwBars;
    L.items = align_up(o, 16);
    o = L.items + kPwItems * sizeof(PwItem);
    L.slot = o;
    o += 16;
    L.total = align_up(o, 16) + 1024;
    // more than half an SM's shared memory: one CTA, which holds all of the
    // SM's TMEM columns, per SM
    if (L.total < kSmemPerSm / 2 + 4 * 1024)
        L.total = kSmemPerSm / 2 + 4 * 1024;
    return L;
}

struct PwParams {
    PrefillParams f;   // the prefill call's (q, lengths, tables, lse, scale)
    int window;        // 0: every new token records
};

// SPLIT: units may be split over the queries (p.pw_count is there).  Of its own:
// with it the others are some 10 us of the 16k step slower (registers).
template <int D, int G, bool SPLIT>
__global__ void __launch_bounds__(kPwThreads, 1)
    prompt_weights_kernel(const __grid_constant__ CUtensorMap tmq,
                          const __grid_constant__ CUtensorMap tmk, const PwParams P)
{
    constexpr int HALVES = D / 64;
    constexpr int TPC = kPwRows / G;                  // new tokens per query tile
    constexpr uint32_t kHalf = kPwRows * 128;         // 128 rows of 64 columns
    constexpr uint32_t kTile = HALVES * kHalf;
    constexpr unsigned FULL = 0xffffffffu;
    static_assert(kPwRows == kPwTokens, "Q and K tiles share their layout");

    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const PwSmem L = pw_smem_layout(D);
    uint64_t *k_full = reinterpret_cast<uint64_t *>(smem + L.bars);
    uint64_t *k_empty = k_full + kPwKStages;   // the item's MMAs of the token tile completed
    uint64_t *q_full = k_empty + kPwKStages;
    uint64_t *q_empty = q_full + kPwQStages;   // both token tiles' MMAs with the query tile completed
    uint64_t *s_full = q_empty + kPwQStages;   // [token tile][2 buffers]
    uint64_t *s_empty = s_full + 4;            // the scores are in registers (8 warps)
    uint64_t *item_ready = s_empty + 4;
    uint64_t *item_free = item_ready + kPwItems;  // the softmax, MMA and lse warps
    uint64_t *part_full = item_free + kPwItems;   // [2][token tile][4] a warp's part written ...
    uint64_t *part_empty = part_full + 16;        // ... and taken over by its partner
    uint64_t *lse_full = part_empty + 16;         // a query tile's log-sum-exps are there
    uint64_t *lse_empty = lse_full + kPwLseStages;  // ... read by every softmax warp
    uint64_t *mma_done = lse_empty + kPwLseStages;
    PwItem *items = reinterpret_cast<PwItem *>(smem + L.items);
    uint32_t *slot = reinterpret_cast<uint32_t *>(smem + L.slot);
    uint8_t *sQ = smem + L.q, *sK = smem + L.k;
    const PrefillParams &p = P.f;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    grid_launch_dependents();
    if (warp == kPwProducerWarp && lane == 0) {
        for (int s = 0; s < kPwKStages; s++) {
            mbar_init(&k_full[s], 1);
            mbar_init(&k_empty[s], 1);
        }
        for (int s = 0; s < kPwQStages; s++) {
            mbar_init(&q_full[s], 1);
            mbar_init(&q_empty[s], 2);
        }
        for (int s = 0; s < 4; s++) {
            mbar_init(&s_full[s], 1);
            mbar_init(&s_empty[s], 8);
        }
        for (int s = 0; s < kPwItems; s++) {
            mbar_init(&item_ready[s], 1);
            mbar_init(&item_free[s], kPwSoftWarps + 3);
        }
        for (int s = 0; s < kPwLseStages; s++) {
            mbar_init(&lse_full[s], 1);
            mbar_init(&lse_empty[s], kPwSoftWarps);
        }
        for (int s = 0; s < 16; s++) {
            mbar_init(&part_full[s], 1);
            mbar_init(&part_empty[s], 1);
        }
        mbar_init(mma_done, 2);
        fence_mbarrier_init();
    } else if (warp == kPwMmaWarp) {
        tc::alloc(smem_u32(slot), 512);
        tc::relinquish();
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = *slot;

    if (warp == kPwProducerWarp) {
        // ------------------------------------------------------------ producer
        if (lane == 0) {
            prefetch_tensormap(&tmq);
            prefetch_tensormap(&tmk);
        }
        grid_dependency_wait();  // lse, caches and the cleared ticket
        bool ok = true;
        int n = 0, gq = 0, nk = 0;  // items published, Q tiles and K tiles issued
        // cursor over the sequences: lane l looks at sequence b0 + l, `before`
        // items lie in the sequences before b0
        int b0 = 0;
        long long before = 0;
        int cq0 = 0, q_len = 0, k_len = 0;  // of sequence b0 + lane
        long long mine = 0, incl = 0;       // its items, and those up to it in this group of 32
        auto look = [&]() {
            cq0 = q_len = k_len = 0;
            const int b = b0 + lane;
            if (b < p.B) {
                const int a0 = __ldg(p.cu_q + b), a1 = __ldg(p.cu_q + b + 1);
                const int c0 = __ldg(p.cu_k + b), c1 = __ldg(p.cu_k + b + 1);
                const int ql = a1 - a0, kl = c1 - c0;
                // the sequences that the attention takes (it reports the others)
                if (a0 >= 0 && ql > 0 && (long long)a1 <= p.Tq && kl >= ql && kl <= p.MBS * p.bs &&
                    ql <= p.max_q) {
                    cq0 = a0;
                    q_len = ql;
                    k_len = kl;
                }
            }
            mine = (((long long)k_len + 2 * kPwTokens - 1) / (2 * kPwTokens)) * p.Hkv;
            incl = mine;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const long long y = __shfl_up_sync(FULL, incl, off);
                if (lane >= off)
                    incl += y;
            }
        };
        // splits per unit: enough items for every SM twice, where there are few units
        int splits = 1;
        if constexpr (SPLIT) {
            long long units = 0;
            int most = 0;  // recorded new tokens of a sequence at most
            for (b0 = 0; b0 < p.B; b0 += 32) {
                look();
                units += __shfl_sync(FULL, incl, 31);
                most = max(most, __reduce_max_sync(FULL, P.window > 0 ? min(q_len, P.window) : q_len));
            }
            b0 = 0;
            if (units > 0 && units < kPwFewUnits)
                splits = min(pw_max_splits(most, G), (int)((2 * kPwFewUnits + units - 1) / units));
        }
        look();
        int ticket = 0;
        if (lane == 0)
            ticket = atomicAdd(p.ticket, 1);
        for (;;) {
            // ---- the ticket's item
            PwItem it{-1, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 1};
            for (bool again = ok; again;) {
                again = false;
                const long long at = __shfl_sync(FULL, ticket, 0), pos = SPLIT ? at / splits : at;
                while (b0 < p.B && pos - before >= __shfl_sync(FULL, incl, 31)) {
                    before += __shfl_sync(FULL, incl, 31);
                    b0 += 32;
                    if (b0 < p.B)
                        look();
                }
                if (b0 < p.B) {
                    const long long r = pos - before;
                    const unsigned in = __ballot_sync(FULL, r >= incl - mine && r < incl);
                    const int src = __ffs(in) - 1;
                    const int rr = (int)(r - __shfl_sync(FULL, incl - mine, src));
                    it.b = b0 + src;
                    it.kvh = rr % p.Hkv;
                    it.t0 = rr / p.Hkv * (2 * kPwTokens);
                    it.cq0 = __shfl_sync(FULL, cq0, src);
                    it.q_len = __shfl_sync(FULL, q_len, src);
                    it.k_len = __shfl_sync(FULL, k_len, src);
                    it.i0 = max(0, it.t0 - (it.k_len - it.q_len));
                    if (P.window > 0)
                        it.i0 = max(it.i0, it.q_len - P.window);
                    it.tiles = ((it.q_len - it.i0) + TPC - 1) / TPC;
                    const int t1 = it.t0 + kPwTokens;
                    it.first1 = t1 < it.k_len
                                    ? max(0, t1 - (it.k_len - it.q_len) - it.i0) / TPC
                                    : it.tiles;
                    if (SPLIT && splits > 1) {
                        const int chunk = max(kPwMinSplit, (it.tiles + splits - 1) / splits);
                        it.unit = (int)pos;
                        it.split = (int)(at - pos * splits);
                        it.splits = (it.tiles + chunk - 1) / chunk;
                        const int skip = it.split * chunk;
                        it.i0 += skip * TPC;
                        it.tiles = min(it.tiles - skip, chunk);
                        it.first1 = min(max(it.first1 - skip, 0), max(it.tiles, 0));
                        if (it.tiles <= 0) {  // the unit has fewer splits: the next ticket
                            it.b = -1;
                            again = true;
                            if (lane == 0)
                                ticket = atomicAdd(p.ticket, 1);
                        }
                    }
                }
            }
            // the next ticket, on its way while this item is copied
            if (it.b >= 0 && lane == 0)
                ticket = atomicAdd(p.ticket, 1);
            const int sl = n % kPwItems;
            if (n >= kPwItems &&
                !(ok = ok && __all_sync(FULL, mbar_wait(&item_free[sl], ((n / kPwItems) & 1) ^ 1))))
                break;  // the other warps time out on item_ready and stop
            if (lane == 0) {
                items[sl] = it;
                mbar_arrive(&item_ready[sl]);
            }
            __syncwarp();
            if (it.b < 0)
                break;
            // ---- K tiles: lanes 0..7 resolve one 16-token box each; where blocks
            // hold whole 64-token runs one copy per run and half, else per box
            for (int kt = 0; kt < 2 && ok; kt++) {
                if (kt == 1 && it.first1 >= it.tiles)
                    break;
                const int t = it.t0 + kt * kPwTokens + lane * kBox;
                int row = -1;
                if (lane < kPwTokens / kBox && t < it.k_len) {
                    const int blk = __ldg(p.block_tables + (size_t)it.b * p.MBS + t / p.bs);
                    if (blk >= 0 && blk < p.NB)
                        row = blk * p.bs + t % p.bs;
                }
                const int per = p.tile_copies ? kPrefillKeys : kBox;  // tokens per copy
                const bool copies = row >= 0 && (lane * kBox) % per == 0;
                const int s = nk % kPwKStages;
                if (!(ok = __all_sync(FULL, mbar_wait(&k_empty[s], ((nk / kPwKStages) & 1) ^ 1))))
                    break;
                const uint32_t bytes = (uint32_t)__popc(__ballot_sync(FULL, copies)) * per * D * 2;
                if (lane == 0)
                    mbar_arrive_expect_tx(&k_full[s], bytes);
                __syncwarp();
                if (copies) {
#pragma unroll
                    for (int hf = 0; hf < HALVES; hf++)
                        tma_load_4d(sK + (size_t)s * kTile + hf * kHalf + lane * kBox * 128, &tmk, 0, hf,
                                    it.kvh, row, &k_full[s]);
                }
                nk++;
            }
            if (!ok)
                break;
            // ---- query tiles
            for (int j = 0; j < it.tiles && ok; j++) {
                const int s = gq % kPwQStages;
                if (!(ok = __all_sync(FULL, mbar_wait(&q_empty[s], ((gq / kPwQStages) & 1) ^ 1))))
                    break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&q_full[s], kTile);
#pragma unroll
                    for (int hf = 0; hf < HALVES; hf++)
                        tma_load_4d(sQ + (size_t)s * kTile + hf * kHalf, &tmq, 0, hf, it.kvh * G,
                                    it.cq0 + it.i0 + j * TPC, &q_full[s]);
                }
                gq++;
            }
            if (!ok)
                break;
            n++;
        }
        if (lane == 0) {
            if (!ok)
                flag_error(p.err_flag, 0x8 /* PKV_FLAG_TIMEOUT */);
            // copies still in flight land before the CTA may exit
            for (int g = max(0, nk - kPwKStages); g < nk; g++)
                mbar_wait(&k_full[g % kPwKStages], (g / kPwKStages) & 1);
            for (int g = max(0, gq - kPwQStages); g < gq; g++)
                mbar_wait(&q_full[g % kPwQStages], (g / kPwQStages) & 1);
        }
        __syncwarp();
    } else if (warp == kPwLseWarp) {
        // ------------------------------------------------------- log-sum-exps
        // Query tile by query tile into a ring, negated, -inf (weight 0) past the
        // sequence; loaded one tile ahead of its stage.
        float *ring = reinterpret_cast<float *>(smem + L.lse);
        grid_dependency_wait();
        bool ok = true;
        int gq = 0;
        for (int n = 0; ok; n++) {
            ok = __all_sync(FULL, mbar_wait(&item_ready[n % kPwItems], (n / kPwItems) & 1));
            if (!ok)
                break;
            const PwItem it = items[n % kPwItems];
            if (it.b < 0)
                break;
            const float *lse = p.lse + ((size_t)it.kvh * p.Tq + it.cq0) * G;
            float ahead[4];
            auto load = [&](int j) {
                const int i_first = it.i0 + j * TPC;
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const int c = lane + 32 * i;
                    ahead[i] = j < it.tiles && i_first + c / G < it.q_len
                                   ? -__ldg(lse + (size_t)i_first * G + c)
                                   : -INFINITY;
                }
            };
            load(0);
            for (int j = 0; j < it.tiles; j++, gq++) {
                const int s = gq % kPwLseStages;
                ok = __all_sync(FULL, mbar_wait(&lse_empty[s], ((gq / kPwLseStages) & 1) ^ 1));
                if (!ok)
                    break;
#pragma unroll
                for (int i = 0; i < 4; i++)
                    ring[s * kPwRows + lane + 32 * i] = ahead[i];
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&lse_full[s]);
                load(j + 1);
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&item_free[n % kPwItems]);
        }
        if (!ok && lane == 0)
            flag_error(p.err_flag, 0x8 /* PKV_FLAG_TIMEOUT */);
    } else if (warp >= kPwMmaWarp) {
        // ----------------------------------------------------------------- MMA
        bool ok = true;
        // A = K (negated for a negative scale: bit 13), B = Q, both K-major
        const uint32_t idS = tc::idesc_bf16(kPwTokens, kPwRows, false) | (p.neg_scale ? 1u << 13 : 0u);
        const int kt = warp - kPwMmaWarp;  // token tile
        // elect.sync, not lane == 0: the compiler then knows that a single thread
        // issues, and an MMA costs the thread 45 cycles instead of 75
        if (tc::elect_one()) {
            int gq = 0, nk = 0;  // query and K tiles so far
            int used = 0;        // query tiles that this token tile took part in
            for (int n = 0; ok; n++) {
                if (!(ok = mbar_wait(&item_ready[n % kPwItems], (n / kPwItems) & 1)))
                    break;
                const PwItem it = items[n % kPwItems];
                if (it.b < 0)
                    break;
                const int kts = it.first1 < it.tiles ? 2 : 1;
                const int first = kt == 0 ? 0 : it.first1;
                const int ks = (nk + kt) % kPwKStages;
                const uint32_t ka = smem_u32(sK + (size_t)ks * kTile);
                if (first < it.tiles && !(ok = mbar_wait(&k_full[ks], ((nk + kt) / kPwKStages) & 1)))
                    break;
                for (int j = 0; j < it.tiles; j++, gq++) {
                    const int s = gq % kPwQStages;
                    if (!(ok = mbar_wait(&q_full[s], (gq / kPwQStages) & 1)))
                        break;
                    if (j >= first) {
                        const int buf = 2 * kt + (used & 1);
                        if (!(ok = mbar_wait(&s_empty[buf], ((used >> 1) & 1) ^ 1)))
                            break;
                        used++;
                        tc::fence_after();
                        const uint32_t qb = smem_u32(sQ + (size_t)s * kTile);
#pragma unroll
                        for (int kq = 0; kq < D / 16; kq++) {
                            const uint32_t off = (uint32_t)(kq >> 2) * kHalf + (uint32_t)(kq & 3) * 32;
                            tc::mma_ss(tmem + 128u * buf, tc::smem_desc(ka + off, 16, 1024),
                                       tc::smem_desc(qb + off, 16, 1024), idS, kq > 0);
                        }
                        tc::commit(smem_u32(&s_full[buf]));
                        tc::commit(smem_u32(&q_empty[s]));
                        if (j == it.tiles - 1)
                            tc::commit(smem_u32(&k_empty[ks]));
                    } else {
                        mbar_arrive(&q_empty[s]);  // a query tile that does not see the token tile
                    }
                }
                if (!ok)
                    break;
                nk += kts;
                mbar_arrive(&item_free[n % kPwItems]);
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
        const int kt = warp >> 3, half = (warp >> 2) & 1;  // token tile, half of the columns
        constexpr int kCols = kPwRows / 2;
        const int r = threadIdx.x & 127;  // token of the tile = TMEM lane
        const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + 256u * kt + kCols * half;
        const float *ring = reinterpret_cast<const float *>(smem + L.lse) + kCols * half;
        float *part = reinterpret_cast<float *>(smem + L.part) + kt * 2 * kPwTokens;
        const float sl = p.scale_log2;
        const float2 sl2 = make_float2(sl, sl);
        grid_dependency_wait();
        bool ok = true;
        int gq = 0;     // query tiles before this item
        int used = 0;   // query tiles of this token tile so far
        int parts = 0;  // sums handed over so far
        for (int n = 0; ok; n++) {
            ok = __all_sync(FULL, mbar_wait(&item_ready[n % kPwItems], (n / kPwItems) & 1));
            if (!ok)
                break;
            const PwItem it = items[n % kPwItems];
            if (it.b < 0)
                break;
            const int first = kt == 0 ? 0 : it.first1;
            // query tiles that do not see this token tile: their log-sum-exps are not
            // needed, but the ring counts every warp
            for (int j = 0; j < first && ok; j++) {
                const int ls = (gq + j) % kPwLseStages;
                ok = __all_sync(FULL, mbar_wait(&lse_full[ls], ((gq + j) / kPwLseStages) & 1));
                if (ok && lane == 0)
                    mbar_arrive(&lse_empty[ls]);
            }
            if (!ok)
                break;
            const int t = it.t0 + kt * kPwTokens + r;
            const int base = it.k_len - it.q_len;
            int blk = -1;
            if (half == 0 && t < it.k_len)
                blk = __ldg(p.block_tables + (size_t)it.b * p.MBS + t / p.bs);
            float sum = 0.f;
            if (first < it.tiles) {
                for (int j = first; j < it.tiles; j++, used++) {
                    const int buf = 2 * kt + (used & 1);
                    const int i_first = it.i0 + j * TPC;
                    const int ls = (gq + j) % kPwLseStages;
                    const float *nl = ring + ls * kPwRows;
                    ok = __all_sync(FULL, mbar_wait(&lse_full[ls], ((gq + j) / kPwLseStages) & 1) &&
                                              mbar_wait(&s_full[buf], (used >> 1) & 1));
                    if (!ok)
                        break;
                    tc::fence_after();
                    uint32_t x[2][32];
                    const uint32_t at = tl + 128u * (used & 1);
                    tc::ld32(at, x[0]);
                    tc::ld32(at + 32, x[1]);
                    tc::wait_ld();
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&s_empty[buf]);  // the scores are in registers
                    // columns c0 <= c < c1 of this half are queries that see this token (a
                    // token far before them is seen by all: times G, 2^28 tokens pass 32 bits)
                    const int c0 = max(t - base - i_first, 0) * G - kCols * half;
                    const int c1 = min(it.q_len - i_first, TPC) * G - kCols * half;
                    float2 a0 = make_float2(0.f, 0.f), a1 = a0;
                    auto add = [&](auto masked_c) {
                        constexpr bool kMasked = decltype(masked_c)::value;
#pragma unroll
                        for (int i = 0; i < kCols / 4; i++) {
                            const uint32_t *y = &x[i >> 3][4 * (i & 7)];
                            const float4 m = *reinterpret_cast<const float4 *>(nl + 4 * i);
                            float2 u = ffma2(make_float2(__uint_as_float(y[0]), __uint_as_float(y[1])), sl2,
                                             make_float2(m.x, m.y));
                            float2 v = ffma2(make_float2(__uint_as_float(y[2]), __uint_as_float(y[3])), sl2,
                                             make_float2(m.z, m.w));
                            if constexpr (kMasked) {
                                const int c = 4 * i;
                                u.x = c >= c0 && c < c1 ? u.x : -INFINITY;
                                u.y = c + 1 >= c0 && c + 1 < c1 ? u.y : -INFINITY;
                                v.x = c + 2 >= c0 && c + 2 < c1 ? v.x : -INFINITY;
                                v.y = c + 3 >= c0 && c + 3 < c1 ? v.y : -INFINITY;
                            }
                            a0 = fadd2(a0, make_float2(fast_exp2(u.x), fast_exp2(u.y)));
                            a1 = fadd2(a1, make_float2(fast_exp2(v.x), fast_exp2(v.y)));
                        }
                    };
                    if (__any_sync(FULL, c0 > 0 || c1 < kCols))
                        add(std::true_type());
                    else
                        add(std::false_type());
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&lse_empty[ls]);
                    sum += (a0.x + a0.y) + (a1.x + a1.y);
                }
                if (!ok)
                    break;
                // ---- the second half hands its sums to the first (the warp with the
                // same tokens), which writes
                const int x = (parts & 1) * 8 + kt * 4 + (warp & 3);
                float *pt = part + (parts & 1) * kPwTokens + r;
                ok = __all_sync(FULL, half == 1 ? mbar_wait(&part_empty[x], ((parts >> 1) & 1) ^ 1)
                                                : mbar_wait(&part_full[x], (parts >> 1) & 1));
                if (!ok)
                    break;
                if (half == 1)
                    *pt = sum;
                else
                    sum += *pt;
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(half == 1 ? &part_full[x] : &part_empty[x]);
                parts++;
            }
            if (half == 0) {
                bool write = first < it.tiles;
                if (SPLIT && it.splits > 1 && it.t0 + kt * kPwTokens < it.k_len) {
                    float *mine = p.pw_part + ((size_t)it.unit * kPwMaxSplits) * 2 * kPwTokens + kt * kPwTokens + r;
                    mine[(size_t)it.split * 2 * kPwTokens] = sum;
                    __threadfence();
                    __syncwarp();
                    int seen = 0;
                    if (lane == 0)
                        seen = atomicAdd(p.pw_count + it.unit * 8 + kt * 4 + (warp & 3), 1);
                    write = __shfl_sync(FULL, seen, 0) == it.splits - 1;
                    if (write) {  // every other split of these 32 tokens is there
                        __threadfence();
                        sum = 0.f;
                        for (int i = 0; i < it.splits; i++)
                            sum += __ldcg(mine + (size_t)i * 2 * kPwTokens);
                    }
                }
                // an addition for new tokens too (the attention cleared their slots):
                // another sequence of the call may have them as its prefix
                if (write && blk >= 0 && blk < p.NB)
                    atomicAdd(p.weights + ((size_t)blk * p.Hkv + it.kvh) * p.bs + t % p.bs, sum);
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&item_free[n % kPwItems]);
            gq += it.tiles;
        }
        if (!ok && lane == 0)
            flag_error(p.err_flag, 0x8 /* PKV_FLAG_TIMEOUT */);
    }
    tc::fence_before();
    __syncthreads();
    if (warp == kPwMmaWarp) {
        tc::fence_after();
        tc::dealloc(tmem, 512);
    }
}

template <int D, bool SPLIT>
static const void *prompt_weights_fn(int G)
{
    switch (G) {
    case 1: return reinterpret_cast<const void *>(&prompt_weights_kernel<D, 1, SPLIT>);
    case 2: return reinterpret_cast<const void *>(&prompt_weights_kernel<D, 2, SPLIT>);
    case 4: return reinterpret_cast<const void *>(&prompt_weights_kernel<D, 4, SPLIT>);
    case 8: return reinterpret_cast<const void *>(&prompt_weights_kernel<D, 8, SPLIT>);
    default: return nullptr;
    }
}

const void *prompt_weights_kernel_fn(int D, int G, bool split)
{
    if (split)
        return D == 128 ? prompt_weights_fn<128, true>(G) : prompt_weights_fn<64, true>(G);
    return D == 128 ? prompt_weights_fn<128, false>(G) : prompt_weights_fn<64, false>(G);
}

size_t prompt_weights_smem_bytes(int D) { return pw_smem_layout(D).total; }

cudaError_t launch_prompt_weights(int D, int G, const CUtensorMap *tmq, const CUtensorMap *tmk,
                                  const PrefillParams &p, int window, int sms, cudaStream_t stream)
{
    PwParams P;
    P.f = p;
    P.window = window;
    // no more CTAs than items there can be
    const long long tiles = ((long long)p.MBS * p.bs + 2 * kPwTokens - 1) / (2 * kPwTokens);
    long long most = tiles * p.Hkv * p.B;
    if (p.pw_count)
        most *= pw_max_splits(window > 0 && window < p.max_q ? window : p.max_q, G);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)(most < sms ? most : sms));
    cfg.blockDim = dim3(kPwThreads);
    cfg.dynamicSmemBytes = pw_smem_layout(D).total;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
#define PKV_PW(DD, GG) \
    if (D == DD && G == GG)                                                                          \
        return p.pw_count ? cudaLaunchKernelEx(&cfg, prompt_weights_kernel<DD, GG, true>, *tmq, *tmk, P) \
                          : cudaLaunchKernelEx(&cfg, prompt_weights_kernel<DD, GG, false>, *tmq, *tmk, P);
    PKV_PW(64, 1) PKV_PW(64, 2) PKV_PW(64, 4) PKV_PW(64, 8)
    PKV_PW(128, 1) PKV_PW(128, 2) PKV_PW(128, 4) PKV_PW(128, 8)
#undef PKV_PW
    return cudaErrorInvalidValue;
}

} // namespace pkv
