// Eviction by accumulated attention weight: kernel parameters and host-side
// launch entry points (internal; the public ABI is pkv.h).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace pkv {

// Division of n < 2^31 by a fixed d >= 1 as a multiplication by ceil-like
// 2^32 (2^l - d) / d + 1 and a shift, with 2^l >= d (Granlund and Montgomery's
// round-up method: exact for every 32-bit n; n < 2^31 keeps the sum in range).
struct FastDiv {
    uint32_t mul, shift, d;
};
inline FastDiv fast_div(uint32_t d)
{
    uint32_t l = 0;
    while ((1ull << l) < d)
        l++;
    return {(uint32_t)((((1ull << l) - d) << 32) / d + 1), l, d};
}

struct EvictParams {
    uint4 *k_cache, *v_cache;     // [NB, bs, Hkv, D], D elements = 16 * units bytes
    float *weights;               // [NB, Hkv, bs]
    const int32_t *block_tables;  // [B, MBS]
    const int32_t *context_lens;  // [B]
    int32_t *out_lens;            // [B], may be context_lens
    int32_t *ws_src;              // [B, Hkv, keep] slot that token j of the trimmed context comes from
    int2 *ws_moved;               // [B, Hkv] (first, new length): tokens first .. length - 1 move
    int32_t *err_flag;            // nullable
    int B, Hkv, MBS, bs, NB;
    int units;                    // 16-byte units of one head's row (D * element bytes / 16)
    int budget, recent;
    int keep;                     // min(budget, MBS * bs): tokens of a trimmed context at most
    int slices;                   // CTAs per (sequence, KV head) that move rows, each a run of units
    int move_threads;             // threads of such a CTA: 128 or 256
    int cluster;                  // CTAs per (sequence, KV head) in the selection: 1, 2, 4 or 8
    int cap;                      // keys each of them holds in shared memory (a multiple of 8)
    FastDiv block;                // division by bs
};

constexpr int kSelCapMax = 12288;  // keys per CTA of the selection at most: three CTAs per SM fit
size_t evict_select_smem_bytes(int cap);
const void *evict_select_kernel_fn();
cudaError_t launch_evict_select(const EvictParams &p, cudaStream_t stream);
cudaError_t launch_evict_move(const EvictParams &p, cudaStream_t stream);

} // namespace pkv
