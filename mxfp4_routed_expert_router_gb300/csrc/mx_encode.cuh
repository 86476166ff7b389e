// mx_encode.cuh -- values to BF16 and MXFP8 (E4M3 values with one E8M0 byte per 32): what the kernels that write the
// library's 16- and 8-bit rows share.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace moe {

__device__ __forceinline__ uint32_t bf16_pair(float a, float b)
{
    const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&p);
}

__device__ __forceinline__ uint4 bf16x8(const float v[8])
{
    return make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7]));
}

// E8M0 byte of a block whose largest value is amax = 1.m * 2^(E - 127): the
// smallest p with amax <= 448 * 2^p = 1.75 * 2^(p + 8), as p + 127.
__device__ __forceinline__ int mx_scale_byte(float amax)
{
    const uint32_t b = __float_as_uint(amax);
    const int byte = (int)(b >> 23) - 8 + ((b & 0x7FFFFFu) > 0x600000u);
    return byte < 0 ? 0 : byte;  // at most 247
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

}  // namespace moe
