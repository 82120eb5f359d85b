// cache.cuh — the paged 8-bit key/value cache as the kernels see it, and its number format.
#pragma once

#include "common.cuh"

namespace dspark {

// Checks a caller's cache (sizes, pointers, alignment); `fn` names the entry point.
int check_cache(const char* fn, const dspark_cache* c);

struct Rope;
int launch_append(const dspark_cache& cache, const Rope& rope, const void* k, int64_t ks,
                  const void* v, int64_t vs, const void* q, int64_t qs, void* q_out, int64_t os,
                  int q_heads, int dtype, int rows, int B, const int32_t* row_req,
                  const int32_t* row_pos, const int32_t* lengths, int32_t* status,
                  cudaStream_t stream);

// Four e4m3 codes from fp32, rounded to nearest even, saturating; x[0] in the lowest byte.
__device__ __forceinline__ uint32_t e4m3x4(float x0, float x1, float x2, float x3)
{
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x1), "f"(x0));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(x3), "f"(x2));
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// Four codes as fp32 (exact: every e4m3 value is an fp16 value).
__device__ __forceinline__ void e4m3x4_to_f32(uint32_t c, float* x)
{
    uint32_t a, b;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(a) : "h"(static_cast<uint16_t>(c & 0xffffu)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(b) : "h"(static_cast<uint16_t>(c >> 16)));
    asm("{.reg .b16 l, h; mov.b32 {l, h}, %2; cvt.f32.f16 %0, l; cvt.f32.f16 %1, h;}"
        : "=f"(x[0]), "=f"(x[1]) : "r"(a));
    asm("{.reg .b16 l, h; mov.b32 {l, h}, %2; cvt.f32.f16 %0, l; cvt.f32.f16 %1, h;}"
        : "=f"(x[2]), "=f"(x[3]) : "r"(b));
}

// Exponent e of a block's scale 2^e: the smallest with amax <= 448 * 2^e, at least -64.
// 448 = 1.75 * 2^8, so with amax = f * 2^E, 1 <= f < 2, it is E - 8 where f <= 1.75, else E - 7;
// read off the bits, without a division. amax must be finite; 0 and subnormals give -64.
__device__ __forceinline__ int scale_exponent(float amax)
{
    const uint32_t u = __float_as_uint(amax);
    const int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return e < -64 ? -64 : e;
}
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

}  // namespace dspark
