// expert_gemm.cu -- the experts' products over the rows a dispatch leaves
// grouped by expert, in e4m3 with fp32 scales per 128 channels of a row and
// per 128 x 128 block of a weight.
//
// Plain tiled form: a block computes 64 rows x 128 columns (for the gated form
// 128 columns of each half) of one expert from tiles of e4m3 values held as
// fp32 in shared memory.  The values of a 128-channel block are summed as they
// are and the block's sum is scaled once, a_scale * w_scale, into the result.
#include "launch.h"
#include "numeric.cuh"

namespace moe {

constexpr int kTileM = 64, kTileN = 128, kTileK = 32;

struct ProductArgs {
    const unsigned char *a, *w;
    const float *a_scale, *w_scale;
    const int32_t *expert_offsets;
    int E, N, C;        // out[rows, N] = a[rows, C] x weight
    long long rows;
    bool transpose;     // weight is [E, C, N] (contraction over its rows) instead of [E, N, C]
    bool out_f32;
    void *out;          // plain form
    unsigned char *q;   // gated form: [rows, N / 2]
    float *q_scale;
    __nv_bfloat16 *h;
};

__device__ __forceinline__ float weight_at(const ProductArgs &p, int e, int n, int c) {
    if (n >= p.N || c >= p.C) return 0.0f;
    return e4m3_to_float(p.w[p.transpose ? ((size_t)e * p.C + c) * p.N + n : ((size_t)e * p.N + n) * p.C + c]);
}

// The scale of the weight block that holds output column n and channel block b.
__device__ __forceinline__ float weight_scale_at(const ProductArgs &p, int e, int n, int b) {
    const int nb = (p.N + 127) / 128, cb = (p.C + 127) / 128;
    return __ldg(p.w_scale + (p.transpose ? ((size_t)e * cb + b) * nb + n / 128 : ((size_t)e * nb + n / 128) * cb + b));
}

template <bool kGated>
__global__ void __launch_bounds__(256) expert_product_kernel(const ProductArgs p) {
    constexpr int kSides = kGated ? 2 : 1;
    __shared__ float s_a[kTileK][kTileM];
    __shared__ float s_w[kSides][kTileK][kTileN];
    __shared__ int s_e, s_row0, s_end;
    if (threadIdx.x == 0) {   // which expert's m-tile blockIdx.y is
        long long t = blockIdx.y;
        s_e = -1;
        for (int e = 0; e < p.E; ++e) {
            const int lo = min(max(p.expert_offsets[e], 0), (int)p.rows), hi = min(max(p.expert_offsets[e + 1], 0), (int)p.rows);
            const int tiles = hi > lo ? (hi - lo + kTileM - 1) / kTileM : 0;
            if (t < tiles) {
                s_e = e;
                s_row0 = lo + (int)t * kTileM;
                s_end = hi;
                break;
            }
            t -= tiles;
        }
    }
    __syncthreads();
    if (s_e < 0) return;
    const int e = s_e, row0 = s_row0, nvalid = min(s_end - row0, kTileM);
    const int n0 = blockIdx.x * kTileN;
    const int cb = (p.C + 127) / 128;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[kSides][4][8] = {}, sum[kSides][4][8] = {};
    for (int c0 = 0; c0 < p.C; c0 += kTileK) {
        for (int i = threadIdx.x; i < kTileM * kTileK; i += 256) {
            const int r = i / kTileK, c = c0 + i % kTileK;
            s_a[i % kTileK][r] = (r < nvalid && c < p.C) ? e4m3_to_float(p.a[(size_t)(row0 + r) * p.C + c]) : 0.0f;
        }
        for (int s = 0; s < kSides; ++s)
            for (int i = threadIdx.x; i < kTileN * kTileK; i += 256) {
                const int n = p.transpose ? i % kTileN : i / kTileK, c = p.transpose ? i / kTileN : i % kTileK;
                s_w[s][c][n] = weight_at(p, e, n0 + n + s * (p.N / 2), c0 + c);
            }
        __syncthreads();
#pragma unroll 4
        for (int c = 0; c < kTileK; ++c)
#pragma unroll
            for (int s = 0; s < kSides; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        sum[s][i][k] = __fmaf_rn(s_a[c][ty * 4 + i], s_w[s][c][tx + 16 * k], sum[s][i][k]);
        __syncthreads();
        if ((c0 + kTileK) % 128 != 0 && c0 + kTileK < p.C) continue;
#pragma unroll
        for (int s = 0; s < kSides; ++s) {   // the end of a block
            const float sw = weight_scale_at(p, e, n0 + s * (p.N / 2), c0 / 128);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = min(ty * 4 + i, nvalid - 1);
                const float f = __ldg(p.a_scale + (size_t)(row0 + r) * cb + c0 / 128) * sw;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    acc[s][i][k] = __fmaf_rn(f, sum[s][i][k], acc[s][i][k]);
                    sum[s][i][k] = 0.0f;
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = ty * 4 + i;
        const size_t row = (size_t)row0 + r;
        if constexpr (kGated) {
            const int I = p.N / 2;
            float v[8], amax = 0.0f;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                v[k] = acc[0][i][k] * sigmoid(acc[0][i][k]) * acc[1][i][k];
                amax = fmaxf(amax, fabsf(v[k]));
            }
#pragma unroll
            for (int off = 8; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
            if (r >= nvalid) continue;
            amax = quant_amax(amax);
            const float inv = quant_inverse(amax);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int n = n0 + tx + 16 * k;
                p.q[row * I + n] = (unsigned char)(pack_e4m3x4(__fmul_rn(v[k], inv), 0.f, 0.f, 0.f) & 0xffu);
                if (p.h) {
                    p.h[row * p.N + n] = __float2bfloat16_rn(acc[0][i][k]);
                    p.h[row * p.N + I + n] = __float2bfloat16_rn(acc[1][i][k]);
                }
            }
            if (tx == 0) p.q_scale[row * (I / 128) + blockIdx.x] = quant_scale(amax);
        } else {
            if (r >= nvalid) continue;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int n = n0 + tx + 16 * k;
                if (n >= p.N) continue;
                if (p.out_f32) static_cast<float *>(p.out)[row * p.N + n] = acc[0][i][k];
                else static_cast<__nv_bfloat16 *>(p.out)[row * p.N + n] = __float2bfloat16_rn(acc[0][i][k]);
            }
        }
    }
}

static cudaError_t launch_product(const ProductArgs &p, bool gated, cudaStream_t stream) {
    const long long mtiles = (p.rows + kTileM - 1) / kTileM + p.E;
    const int ntiles = ((gated ? p.N / 2 : p.N) + kTileN - 1) / kTileN;
    const dim3 grid((unsigned)ntiles, (unsigned)mtiles);
    if (gated) expert_product_kernel<true><<<grid, 256, 0, stream>>>(p);
    else expert_product_kernel<false><<<grid, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_expert_gemm(const void *a, const float *a_scale, const void *w, const float *w_scale,
                               const int32_t *expert_offsets, int E, int N, int C, long long rows, bool transpose,
                               bool out_f32, void *out, cudaStream_t stream) {
    ProductArgs p = {static_cast<const unsigned char *>(a), static_cast<const unsigned char *>(w), a_scale, w_scale,
                     expert_offsets, E, N, C, rows, transpose, out_f32, out, nullptr, nullptr, nullptr};
    return launch_product(p, false, stream);
}

cudaError_t launch_expert_gated_gemm(const void *a, const float *a_scale, const void *w, const float *w_scale,
                                     const int32_t *expert_offsets, int E, int I, int C, long long rows, void *q,
                                     float *q_scale, void *h, cudaStream_t stream) {
    ProductArgs p = {static_cast<const unsigned char *>(a), static_cast<const unsigned char *>(w), a_scale, w_scale,
                     expert_offsets, E, 2 * I, C, rows, false, false, nullptr, static_cast<unsigned char *>(q),
                     q_scale, static_cast<__nv_bfloat16 *>(h)};
    return launch_product(p, true, stream);
}

}  // namespace moe
