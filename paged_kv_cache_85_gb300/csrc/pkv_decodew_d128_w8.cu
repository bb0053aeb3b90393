// Instantiations of the paged decode kernel that records attention scores:
// head_dim 128, 8 workers per CTA, bf16 caches, G = 1, 2, 4, 8.
#include "pkv_decode.cuh"

namespace pkv {

cudaError_t launch_decodew_d128_w8(int G, const CUtensorMap *tmk, const CUtensorMap *tmv,
                                 const DecodeParams &p, int grid, size_t smem, cudaStream_t stream)
{
    return launch_decode_shape<128, 8, false, kBox, true>(G, tmk, tmv, p, grid, smem, stream);
}

const void *decodew_kernel_d128_w8(int G) { return decode_kernel_shape<128, 8, false, kBox, true>(G); }

} // namespace pkv
