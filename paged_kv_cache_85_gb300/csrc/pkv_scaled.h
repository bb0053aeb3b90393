// The store into an E4M3 cache with a scale per block and KV head, and the copy of
// blocks: kernel parameters and host-side launch entry points (internal; the public
// ABI is pkv.h).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "pkv_evict.h"

namespace pkv {

struct StoreScaledParams {
    const uint8_t *x[2];      // K and V rows, bf16 [N, Hkv, D]
    uint8_t *cache[2];        // E4M3 [NB, bs, Hkv, D]
    float *scales[2];         // [NB, Hkv]
    const int64_t *slots;     // [N]
    int32_t *err_flag;        // nullable
    long long N, n_slots;     // n_slots = NB * bs < 2^31
    int Hkv, bs;
    FastDiv block;            // division by bs
};

cudaError_t launch_store_scaled(int D, const StoreScaledParams &p, cudaStream_t stream);

constexpr int kCopyTensors = 64;  // tensors per launch of the block copy

struct CopyTensor {
    uint8_t *base;
    long long block_bytes;
    int chunks;  // warp-sized pieces per block
    int vec;     // bytes per load: 16, 4 or 1, which divide the address and block_bytes
};

struct CopyParams {
    CopyTensor t[kCopyTensors];
    const int2 *pairs;  // [n] source, destination
    int32_t *err_flag;  // nullable
    int n_tensors, n, NB;
    int chunks;         // of all tensors
};

constexpr int kCopyChunk = 4096;  // bytes per piece (one warp, 16-byte loads)
cudaError_t launch_copy_blocks(const CopyParams &p, int sms, cudaStream_t stream);

} // namespace pkv
