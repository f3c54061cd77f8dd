// numeric.cuh -- bf16 and e4m3 conversions shared by the expert products and
// the gradient kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

namespace moe {

// bf16 pair (low half = first element) -> two fp32, exactly (bf16 is the high
// half of an fp32).
__device__ __forceinline__ float bf16_pair_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_pair_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ void unpack_bf16x8(const uint4 v, float (&f)[8]) {
    const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        f[2 * k] = bf16_pair_lo(q[k]);
        f[2 * k + 1] = bf16_pair_hi(q[k]);
    }
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);   // round to nearest even
    return (uint32_t)__bfloat16_as_ushort(h.x) | ((uint32_t)__bfloat16_as_ushort(h.y) << 16);
}

__device__ __forceinline__ uint4 pack_bf16x8(const float *f) {
    return make_uint4(bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7]));
}

// The block quantisation of moe_dispatch: amax raised to 2^-119 (the smallest
// power of two with 448 / amax finite in fp32), scale = amax / 448 and
// inv = 448 / amax by IEEE division, q = e4m3(v * inv), saturated to +-448.
__device__ __forceinline__ float quant_amax(float amax) { return fmaxf(amax, 0x1p-119f); }
__device__ __forceinline__ float quant_scale(float amax) { return __fdiv_rn(amax, 448.0f); }
__device__ __forceinline__ float quant_inverse(float amax) { return __fdiv_rn(448.0f, amax); }

// Four values to four e4m3 bytes, the first in the lowest byte.
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
    const uint32_t lo = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

__device__ __forceinline__ float e4m3_to_float(unsigned char b) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)b, __NV_E4M3)));
}

// The logistic function from t = exp(-|v|): 1 / (1 + t), or t / (1 + t) for
// negative v.  The divisor lies in [1, 2], inside the range where the fast
// division keeps its 2 ulp (it returns 0 for divisors past 2^126, which 1 +
// exp(-v) is from v = -87.4 on, where silu times a large factor still counts).
// expf is within 2 ulp as well; an IEEE division took the gated product's tiles
// 10 % longer.  Against 1 / (1 + exp(-v)) it costs the gated prefill layer 1 % in
// long runs (6.81 and 6.75 ms).
__device__ __forceinline__ float sigmoid(float v) {
    const float t = expf(-fabsf(v));
    return __fdividef(v < 0.0f ? t : 1.0f, 1.0f + t);
}

// With __expf: within (1 - s) * (2 + 1.2 |v|) + 2 ulp, a few ulp wherever s is
// not tiny, for the gate's gradient, which waited on the arithmetic of expf (745
// against 663 us) and has no forward values to agree with code by code.  Below
// 2^-126 (v < -87.3) it is 0: the form above took that gradient 711 us.
__device__ __forceinline__ float sigmoid_fast(float v) { return __fdividef(1.0f, 1.0f + __expf(-v)); }

// Pairs of fp32 in one instruction each, rounded as the single operations are.
__device__ __forceinline__ float2 mul_pair(float2 a, float2 b) {
    float2 r;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<unsigned long long &>(r))
        : "l"(reinterpret_cast<const unsigned long long &>(a)), "l"(reinterpret_cast<const unsigned long long &>(b)));
    return r;
}
// acc = f * v + acc
__device__ __forceinline__ void fma_pair(float2 &acc, float2 f, float2 v) {
    asm("fma.rn.f32x2 %0, %1, %2, %0;"
        : "+l"(reinterpret_cast<unsigned long long &>(acc))
        : "l"(reinterpret_cast<const unsigned long long &>(f)), "l"(reinterpret_cast<const unsigned long long &>(v)));
}
__device__ __forceinline__ float2 bf16_pair_floats(uint32_t w) { return make_float2(bf16_pair_lo(w), bf16_pair_hi(w)); }

}  // namespace moe
