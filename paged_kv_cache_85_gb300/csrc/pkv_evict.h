// Eviction by accumulated attention weight: kernel parameters and host-side
// launch entry points (internal; the public ABI is pkv.h).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace pkv {

struct EvictParams {
    uint4 *k_cache, *v_cache;     // [NB, bs, Hkv, D], D elements = 16 * units bytes
    float *weights;               // [NB, Hkv, bs]
    const int32_t *block_tables;  // [B, MBS]
    const int32_t *context_lens;  // [B]
    int32_t *out_lens;            // [B], may be context_lens
    int32_t *ws_src;              // [B, Hkv, keep] slot that token j of the trimmed context comes from
    int32_t *ws_dst;              // [B, keep] slot of token j
    int2 *ws_moved;               // [B, Hkv] (first, end): tokens j in [first, end) move
    int32_t *err_flag;            // nullable
    int B, Hkv, MBS, bs, NB;
    int units;                    // 16-byte units of one head's row (D * element bytes / 16)
    int budget, recent;
    int keep;                     // min(budget, MBS * bs): tokens of a trimmed context at most
    int slices;                   // CTAs per (sequence, KV head) in the move, each a run of units
};

cudaError_t launch_evict_select(const EvictParams &p, cudaStream_t stream);
cudaError_t launch_evict_move(const EvictParams &p, cudaStream_t stream);

} // namespace pkv
