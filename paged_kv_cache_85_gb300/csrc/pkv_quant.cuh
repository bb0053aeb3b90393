// E4M3 conversions shared by the quantising stores.
#pragma once

#include <stdint.h>

#include "pkv_ptx.cuh"

namespace pkv {

// Eight bf16 values (16 B) times inv, in fp32, as E4M3 codes (8 B; nearest even,
// finite saturation, NaN stays NaN).
__device__ __forceinline__ uint2 quantize8(uint4 a, float inv)
{
    const float2 f0 = bf16x2_to_float2(a.x), f1 = bf16x2_to_float2(a.y);
    const float2 f2 = bf16x2_to_float2(a.z), f3 = bf16x2_to_float2(a.w);
    const uint32_t c0 = f32x2_to_e4m3x2(__fmul_rn(f0.x, inv), __fmul_rn(f0.y, inv));
    const uint32_t c1 = f32x2_to_e4m3x2(__fmul_rn(f1.x, inv), __fmul_rn(f1.y, inv));
    const uint32_t c2 = f32x2_to_e4m3x2(__fmul_rn(f2.x, inv), __fmul_rn(f2.y, inv));
    const uint32_t c3 = f32x2_to_e4m3x2(__fmul_rn(f3.x, inv), __fmul_rn(f3.y, inv));
    return make_uint2(c0 | (c1 << 16), c2 | (c3 << 16));
}

// Four bf16 values alike (4 codes).
__device__ __forceinline__ uint32_t quantize4(uint32_t a, uint32_t b, float inv)
{
    const float2 f2 = make_float2(inv, inv);
    const float2 x = fmul2(bf16x2_to_float2(a), f2), y = fmul2(bf16x2_to_float2(b), f2);
    return f32x2_to_e4m3x2(x.x, x.y) | (f32x2_to_e4m3x2(y.x, y.y) << 16);
}

// Four codes as the codes of their values times f.
__device__ __forceinline__ uint32_t recode4(uint32_t w, float f)
{
    uint32_t lo, hi;
    e4m3x4_to_f16x2x2(w, lo, hi);
    const float2 a = f16x2_to_float2(lo), b = f16x2_to_float2(hi);
    return f32x2_to_e4m3x2(__fmul_rn(a.x, f), __fmul_rn(a.y, f)) |
           (f32x2_to_e4m3x2(__fmul_rn(b.x, f), __fmul_rn(b.y, f)) << 16);
}

} // namespace pkv
