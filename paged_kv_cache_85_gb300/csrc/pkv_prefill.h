// Paged prefill: kernel parameters and host-side launch entry points
// (internal; the public ABI is pkv.h).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace pkv {

struct PrefillParams {
    const uint16_t *q;            // bf16 [Tq, Hq, D]: the sequences' new tokens, concatenated
    uint16_t *out;                // bf16 [Tq, Hq, D]
    const int32_t *block_tables;  // [B, MBS]
    const int32_t *cu_q;          // [B + 1] boundaries of the new tokens
    const int32_t *cu_k;          // [B + 1] boundaries of the contexts (cached + new)
    int32_t *err_flag;            // nullable
    long long Tq;
    int B, Hq, Hkv, MBS, bs, NB;
    int max_q;                    // the caller's bound on q_len (sizes the work space)
    int X;                        // query tile pairs per sequence at max_q
    int n_items;                  // work items: X tile pairs x Hkv heads x B sequences
    float scale_log2;             // |scale| * log2(e)
    int neg_scale;                // scale < 0: the score MMA negates Q
    int tile_copies;              // bs % 64 == 0: K/V maps copy whole 64-token tiles
    float *lse = nullptr;         // nullable: [Hkv, Tq, G] log-sum-exp of every row (log2 units)
    float *weights = nullptr;     // [NB, Hkv, bs], where lse is: cleared for the new tokens by the
                                  // attention, added to by the weights kernel
    // 128-key kernel, where its items are split over the keys (splits > 1)
    int splits = 1;
    int whole = 0;                // the first (longest) items, which are not split
    int least = 0;                // nor are items of fewer key tiles
    float *part_out = nullptr;    // [splits, Tq, Hq, D] outputs of the splits
    float *part_lse = nullptr;    // [splits, Hkv, Tq, G] their log-sum-exps, -inf: no key; of
                                  // a whole item's rows the first is +inf
    int32_t *ticket = nullptr;    // nullable: work counter of the weights kernel, cleared here
    // nullable, for the weights kernel's splits: arrivals per unit and warp (cleared
    // here) and partial sums [kPwFewUnits][kPwMaxSplits][256]
    int32_t *pw_count = nullptr;
    float *pw_part = nullptr;
};

cudaError_t launch_prefill(int D, int G, bool wide, const CUtensorMap *tmq, const CUtensorMap *tmk,
                           const CUtensorMap *tmv, const PrefillParams &p, dim3 grid, size_t smem,
                           cudaStream_t stream);
constexpr int kPwFewUnits = 152;  // fewer units (256 tokens, one KV head) than this are split
constexpr int kPwMaxSplits = 16;
constexpr int kPwMinSplit = 4;  // query tiles of 128 rows per split at least
// Splits of a unit at most, for so many recorded tokens.
__host__ __device__ inline int pw_max_splits(int tokens, int G)
{
    const long long tiles = ((long long)tokens * G + 127) / 128;
    const long long s = tiles / kPwMinSplit;
    return s < 1 ? 1 : s > kPwMaxSplits ? kPwMaxSplits : (int)s;
}
// Whether a call may have so few units (its new tokens alone make Tq Hkv / 256).
inline bool pw_may_split(int B, long long Tq, int max_q, int G, int Hkv)
{
    return (long long)B * Hkv < kPwFewUnits && Tq * Hkv < 256LL * kPwFewUnits && pw_max_splits(max_q, G) > 1;
}
constexpr size_t kPwCountBytes = (size_t)kPwFewUnits * 8 * sizeof(int32_t);
constexpr size_t kPwPartBytes = (size_t)kPwFewUnits * kPwMaxSplits * 256 * sizeof(float);
cudaError_t launch_prompt_weights(int D, int G, const CUtensorMap *tmq, const CUtensorMap *tmk,
                                  const PrefillParams &p, int window, int sms, cudaStream_t stream);
const void *prompt_weights_kernel_fn(int D, int G, bool split);
size_t prompt_weights_smem_bytes(int D);
const void *prefill_kernel(int D, int G, bool wide, bool split);
size_t prefill_smem_bytes(int D, bool wide);
// Key tiles (of 128) per split of an item of nkt tiles, which is split where it has
// `least`; its splits are ceil(nkt / chunk) <= splits, a single one if nkt <= chunk.
constexpr int kMinSplitTiles = 4;
__host__ __device__ inline int wide_chunk(int nkt, int splits, int least)
{
    if (nkt < least)
        return nkt;
    const int chunk = (nkt + splits - 1) / splits;
    return chunk < kMinSplitTiles ? kMinSplitTiles : chunk;
}
// How a call's items are split, from its sizes: items from `whole` on, where they
// have `least` key tiles, into up to `splits` pieces.
//  * Where there are fewer items than SMs, all of them, into enough pieces for two
//    per SM, none shorter than kMinSplitTiles tiles of the longest context.
//  * Where there are a few rounds of long items, those of the last, incomplete
//    round: 256 items (2048 new tokens of 32 heads on a context of 28672) are two
//    rounds of 152 SMs, in the second of which 48 have nothing to do.  Worth it
//    where the shorter last round saves more than the pieces' ends (some 8000
//    cycles each), their outputs' way through memory (262 KB written and read of a
//    piece, at 3500 bytes a cycle) and the join cost; a key tile is 3200 cycles.
//    Whole call: those 256 items 820 -> 792 us; 168 items (1300 new tokens on 28672)
//    798 -> 545; 192 (three of 512 on 8192) 269 -> 215; 512 (4096 on 16384) 1002 -> 935.
// The host knows the tables' width and the longest chunk, not the contexts, which may be
// far shorter: `least` leaves items whole that the sum above does not split (four chunks
// of 1024 tokens of 16 heads on nothing, tables of 40960: 97 us with every item of the
// last round split, 68 so, 63 with tables as wide as the contexts).
struct WideSplit {
    int whole, splits, least;
};
// With another number of SMs than this the pieces fill the last round less well; the
// results are the same.
constexpr long long kWideSms = 152;
constexpr int kJoinMaxSeqs = 152;  // sequences that the join kernel can look through
inline WideSplit wide_split(long long items, long long max_ctx, int max_q, int B)
{
    const long long tiles = (max_ctx + 127) / 128;
    if (items < 1 || B > kJoinMaxSeqs)
        return {0, 1, 0};
    if (items < kWideSms) {
        long long s = (2 * kWideSms + items - 1) / items;
        if (s > tiles / kMinSplitTiles)
            s = tiles / kMinSplitTiles;
        return {0, s < 1 ? 1 : (int)s, 0};
    }
    const long long rounds = items / kWideSms, left = items % kWideSms;
    if (rounds > 4 || left == 0)  // (the pieces' buffers hold all rows, 400 MB with four)
        return {0, 1, 0};
    // the last round has the shortest items, the start of the longest sequence's new
    // tokens at least (where they vary more, the longest-first order fills the SMs)
    const long long item = (max_ctx - max_q) / 128 * 3200;
    WideSplit best = {0, 1, 0};
    long long cheapest = item + 8000 - (rounds * item) / 20;  // a twentieth of the call at least
    for (int s = 2; s <= 4; s++) {
        const long long pieces = (left * s + kWideSms - 1) / kWideSms;
        const long long cost = pieces * (item / s + 8000) + left * s * 75 + 20000;
        if (cost < cheapest) {
            cheapest = cost;
            // cost < item + 8000 - rounds item / 20, solved for the item's tiles
            const long long gain = 20 * s - s * rounds - 20 * pieces;  // > 0, of 20 s
            const long long ends = (pieces - 1) * 8000 + left * s * 75 + 20000;
            best = {(int)(rounds * kWideSms), s, (int)(20 * s * ends / (gain * 3200)) + 1};
        }
    }
    return best;
}
cudaError_t launch_prefill_join(int D, const PrefillParams &p, cudaStream_t stream);
constexpr int kPrefillRows = 128;  // (token, head) rows per query tile (two tiles per work item)
constexpr int kPrefillKeys = 64;   // keys per K/V tile
constexpr int kPrefillThreads = 11 * 32;

} // namespace pkv
