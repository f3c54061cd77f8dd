// mx4.cu -- rows of bf16 or fp32 to 4-bit values with a scale per 32 channels,
// and back to bf16, or the bare values to e4m3 (which holds them exactly).
//
// Both are one pass: a thread takes 8 channels, so 4 neighbouring lanes hold a
// block and share its largest magnitude by two shuffles; rows lie one after the
// other, so the whole tensor is one run of blocks.  Bound by HBM: 65536 x 7168 to 4
// bits and back in 343 us (2.4 GB, 1.02 of the measured copy rate).
#include "launch.h"
#include "mx4.cuh"

namespace moe {

constexpr int kMx4Threads = 256;
constexpr int kMx4Chunks = 4;   // of 8 channels a thread, all in flight at once

template <bool kF32>
__global__ void __launch_bounds__(kMx4Threads) quantize_mx4_kernel(const void *x, long long chunks, uint32_t *q,
                                                                   unsigned char *scale) {
    pdl_launch_dependents();
    pdl_wait();
    const long long first = (long long)blockIdx.x * (kMx4Threads * kMx4Chunks) + threadIdx.x;
    uint4 v[kMx4Chunks][kF32 ? 2 : 1];
#pragma unroll
    for (int i = 0; i < kMx4Chunks; ++i) {
        const long long c = first + i * kMx4Threads;
        const unsigned char *from = static_cast<const unsigned char *>(x) + c * (kF32 ? 32 : 16);
#pragma unroll
        for (int h = 0; h < (kF32 ? 2 : 1); ++h)
            v[i][h] = c < chunks ? ld_chained_v4(from + h * 16) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < kMx4Chunks; ++i) {
        const long long c = first + i * kMx4Threads;
        float f[8];
        if constexpr (kF32) {
            const uint4 a = v[i][0], b = v[i][1];
            const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
            for (int k = 0; k < 8; ++k) f[k] = __uint_as_float(w[k]);
        } else {
            unpack_bf16x8(v[i][0], f);
        }
        uint32_t amax = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) amax = max(amax, magnitude_bits(f[k]));
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const uint32_t byte = mx4_scale_byte(amax);
        if (c < chunks) {
            q[c] = pack_e2m1x8(f, mx4_inverse(byte));
            if ((threadIdx.x & 3) == 0) scale[c >> 2] = (unsigned char)byte;
        }
    }
}

// kValues: the codes' values alone, in e4m3.
template <bool kValues>
__global__ void __launch_bounds__(kMx4Threads) dequantize_mx4_kernel(const uint32_t *q, const unsigned char *scale,
                                                                     long long chunks, void *out) {
    pdl_launch_dependents();
    pdl_wait();
    const long long first = (long long)blockIdx.x * (kMx4Threads * kMx4Chunks) + threadIdx.x;
    uint32_t w[kMx4Chunks], s[kMx4Chunks];
#pragma unroll
    for (int i = 0; i < kMx4Chunks; ++i) {
        const long long c = first + i * kMx4Threads;
        w[i] = c < chunks ? (uint32_t)ld_chained(reinterpret_cast<const int32_t *>(q) + c) : 0u;
        s[i] = !kValues && c < chunks ? ld_chained(scale + (c >> 2)) : 0u;
    }
#pragma unroll
    for (int i = 0; i < kMx4Chunks; ++i) {
        const long long c = first + i * kMx4Threads;
        uint32_t h[4];
        unpack_e2m1x8(w[i], h);
        float2 f[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) f[k] = __half22float2(reinterpret_cast<const __half2 &>(h[k]));
        if (c >= chunks) continue;
        if constexpr (kValues) {
            reinterpret_cast<uint2 *>(out)[c] = make_uint2(pack_e4m3x4(f[0].x, f[0].y, f[1].x, f[1].y),
                                                           pack_e4m3x4(f[2].x, f[2].y, f[3].x, f[3].y));
        } else {
            const float t = mx4_scale(s[i]);
            st_v4(static_cast<unsigned char *>(out) + c * 16,
                  make_uint4(bf16_pair(f[0].x * t, f[0].y * t), bf16_pair(f[1].x * t, f[1].y * t),
                             bf16_pair(f[2].x * t, f[2].y * t), bf16_pair(f[3].x * t, f[3].y * t)));
        }
    }
}

static unsigned blocks_of(long long chunks) {
    return (unsigned)((chunks + kMx4Threads * kMx4Chunks - 1) / (kMx4Threads * kMx4Chunks));
}

cudaError_t launch_quantize_mx4(const void *x, bool f32, long long blocks, void *q, void *scale, cudaStream_t stream) {
    const long long chunks = blocks * (kMx4Block / 8);
    return launch_chained(f32 ? quantize_mx4_kernel<true> : quantize_mx4_kernel<false>, blocks_of(chunks), kMx4Threads,
                          0, stream, x, chunks, static_cast<uint32_t *>(q), static_cast<unsigned char *>(scale));
}

cudaError_t launch_dequantize_mx4(const void *q, const void *scale, long long blocks, void *out, cudaStream_t stream) {
    const long long chunks = blocks * (kMx4Block / 8);
    return launch_chained(scale ? dequantize_mx4_kernel<false> : dequantize_mx4_kernel<true>, blocks_of(chunks),
                          kMx4Threads, 0, stream, static_cast<const uint32_t *>(q),
                          static_cast<const unsigned char *>(scale), chunks, out);
}

}  // namespace moe
