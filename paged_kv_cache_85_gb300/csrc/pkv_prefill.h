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
    // 128-key kernel, where its items are split over the keys (splits > 1)
    int splits = 1;
    float *part_out = nullptr;    // [splits, Tq, Hq, D] outputs of the splits
    float *part_lse = nullptr;    // [splits, Hkv, Tq, G] their log-sum-exps, -inf: no key
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
                                  const PrefillParams &p, float *weights, int window, int sms,
                                  cudaStream_t stream);
const void *prompt_weights_kernel_fn(int D, int G, bool split);
size_t prompt_weights_smem_bytes(int D);
const void *prefill_kernel(int D, int G, bool wide, bool split);
size_t prefill_smem_bytes(int D, bool wide);
// Key tiles (of 128) per split of an item of nkt tiles; its splits are
// ceil(nkt / chunk) <= splits.
constexpr int kMinSplitTiles = 4;
__host__ __device__ inline int wide_chunk(int nkt, int splits)
{
    const int chunk = (nkt + splits - 1) / splits;
    return chunk < kMinSplitTiles ? kMinSplitTiles : chunk;
}
// Splits of a call: enough to give two items to every SM of a large GPU where
// the query tile pairs alone do not give it one, and none shorter than
// kMinSplitTiles tiles of the longest context.
inline int wide_splits(long long items, long long max_ctx)
{
    constexpr long long kFew = 152, kWant = 304;
    if (items < 1 || items >= kFew)
        return 1;
    const long long tiles = (max_ctx + 127) / 128;
    long long s = (kWant + items - 1) / items;
    if (s > tiles / kMinSplitTiles)
        s = tiles / kMinSplitTiles;
    return s < 1 ? 1 : (int)s;
}
cudaError_t launch_prefill_join(int D, const PrefillParams &p, cudaStream_t stream);
constexpr int kPrefillRows = 128;  // (token, head) rows per query tile (two tiles per work item)
constexpr int kPrefillKeys = 64;   // keys per K/V tile
constexpr int kPrefillThreads = 11 * 32;

} // namespace pkv
