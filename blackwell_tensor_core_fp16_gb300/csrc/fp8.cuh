// E4M3 codes with E8M0 scales: conversions that the operators on an 8-bit cache share.
#pragma once

#include "decode_common.cuh"

namespace decode {

// Two codes as two float16 (exact), and the nearest codes of two fp32 values: of NaN NaN, of a value
// past 448 the largest.
__device__ __forceinline__ uint32_t codes_to_half2(uint32_t two)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
    return r;
}
__device__ __forceinline__ uint32_t codes_of(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// 2^(e - 127) for e in -22 .. 254, where it is a number of fp32, subnormal ones among them.
__device__ __forceinline__ float power_of(int e)
{
    return __uint_as_float(e > 0 ? static_cast<uint32_t>(e) << 23 : 0x400000u >> -e);
}
// What a scale stands for.
__device__ __forceinline__ float scale_of(int e) { return e == 255 ? NAN : power_of(e); }

// What is wrong with a cache's sizes; DECODE_OK if nothing is.
inline int check_cache(int64_t pages, int64_t page_size, int64_t block, int64_t heads, int64_t d)
{
    constexpr int64_t kMost = (int64_t(1) << 31) - 1;
    if (pages < 0 || page_size <= 0 || heads <= 0)
        return fail(DECODE_ERR_INVALID_ARG, "negative size, no head or no page size");
    if (block <= 0 || page_size % block != 0)
        return fail(DECODE_ERR_INVALID_ARG, "pages of %lld tokens in blocks of %lld",
                    (long long)page_size, (long long)block);
    if (d != 64 && d != 128 && d != 256)
        return fail(DECODE_ERR_UNSUPPORTED, "head_dim %lld (64, 128 or 256)", (long long)d);
    if (pages > kMost || page_size > kMost || heads >= (1 << 20))
        return fail(DECODE_ERR_UNSUPPORTED, "problem too large for one call");
    return DECODE_OK;
}

}  // namespace decode
