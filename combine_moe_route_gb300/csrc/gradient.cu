// gradient.cu -- gradients of the weighted combine, of the dispatch scatter
// and of the experts' gate.
//
// The forward of a layer is, for token g with experts e_j and weights w_j,
//   out[g] = sum_j w_j * y[row(g, j)],   w = softmax of the K selected logits,
//   recv[row(g, j)] = x[g],
// so the gradients are
//   dy[row(g, j)] = w_j * dout[g]
//   dw_j          = <dout[g], y[row(g, j)]>
//   dlogit[e_j]   = w_j * (dw_j - sum_i w_i dw_i), 0 for the other experts
//   dx[g]         = sum_j drows[row(g, j)].
// The last one is the combine with unit weights and runs as that kernel
// (combine.cu).
#include "launch.h"
#include "numeric.cuh"

namespace moe {

// --------------------------------------------------------------------------
// combine backward
// --------------------------------------------------------------------------
// One block per token.  A thread owns 16-byte chunks (8 channels) of the row:
// for each it loads dout once and the chunk of up to kGradBatch rows of y, all
// in flight together, adds the products to one fp32 sum per row and writes
// w_j * dout.  The sums are folded by shuffles and then, in a fixed order,
// across the warps.  FP8: 16 lanes hold a block of 128 channels; its amax is
// |w_j| * max|dout| (rounding is monotone, so this is the amax of the rounded
// products), one shuffle reduction per block for all K copies.
constexpr int kGradThreads = 256;
constexpr int kGradBatch = 8;

template <bool kFp8>
__global__ void __launch_bounds__(kGradThreads) combine_backward_kernel(
    const __nv_bfloat16 *__restrict__ dout, const __nv_bfloat16 *__restrict__ y, const int32_t *__restrict__ tok2row,
    const float *__restrict__ topk_w, const int32_t *__restrict__ topk_idx, int T, int K, int H, long long rows, int E,
    void *__restrict__ dy, float *__restrict__ dy_scale, float *__restrict__ dtopk_w, float *__restrict__ dlogits) {
    extern __shared__ float s_dl[];   // [E] when dlogits is wanted
    __shared__ int32_t s_row[MOE_MAX_TOPK];
    __shared__ float s_w[MOE_MAX_TOPK];
    __shared__ float s_part[kGradThreads / 32][MOE_MAX_TOPK];
    __shared__ float s_dw[MOE_MAX_TOPK];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nchunk = H / 8;
    const int nchunk_warp = (nchunk + 31) & ~31;   // whole warps, so that the shuffles are uniform
    const long long g = blockIdx.x;

    if (threadIdx.x < K) {
        const long long r = tok2row ? (long long)__ldg(tok2row + g * K + threadIdx.x) : g * K + threadIdx.x;
        s_row[threadIdx.x] = (r >= 0 && r < rows) ? (int32_t)r : -1;
        s_w[threadIdx.x] = __ldg(topk_w + g * K + threadIdx.x);
    }
    if (dlogits)
        for (int e = threadIdx.x; e < E; e += kGradThreads) s_dl[e] = 0.0f;
    __syncthreads();

    for (int j0 = 0; j0 < K; j0 += kGradBatch) {
        float acc[kGradBatch];
#pragma unroll
        for (int jj = 0; jj < kGradBatch; ++jj) acc[jj] = 0.0f;
        for (int c = threadIdx.x; c < nchunk_warp; c += kGradThreads) {
            const bool in = c < nchunk;
            uint4 v[kGradBatch];
#pragma unroll
            for (int jj = 0; jj < kGradBatch; ++jj) {
                const int r = (j0 + jj < K) ? s_row[j0 + jj] : -1;
                v[jj] = (in && r >= 0) ? ld_stream_v4(y + (size_t)r * H + (size_t)c * 8) : make_uint4(0u, 0u, 0u, 0u);
            }
            float d[8];
            unpack_bf16x8(in ? *reinterpret_cast<const uint4 *>(dout + (size_t)g * H + (size_t)c * 8)
                             : make_uint4(0u, 0u, 0u, 0u), d);
            float dmax = 0.0f;
            if (kFp8) {
#pragma unroll
                for (int k = 0; k < 8; ++k) dmax = fmaxf(dmax, fabsf(d[k]));
#pragma unroll
                for (int off = 8; off > 0; off >>= 1) dmax = fmaxf(dmax, __shfl_xor_sync(0xffffffffu, dmax, off));
            }
#pragma unroll
            for (int jj = 0; jj < kGradBatch; ++jj) {
                if (j0 + jj >= K) break;
                const int r = s_row[j0 + jj];
                if (r < 0 || !in) continue;
                const float w = s_w[j0 + jj];
                float f[8];
                unpack_bf16x8(v[jj], f);
#pragma unroll
                for (int k = 0; k < 8; ++k) acc[jj] = __fmaf_rn(d[k], f[k], acc[jj]);
#pragma unroll
                for (int k = 0; k < 8; ++k) f[k] = __fmul_rn(w, d[k]);
                if (kFp8) {
                    const float amax = quant_amax(__fmul_rn(fabsf(w), dmax));
                    const float inv = quant_inverse(amax);
#pragma unroll
                    for (int k = 0; k < 8; ++k) f[k] = __fmul_rn(f[k], inv);
                    *reinterpret_cast<uint2 *>(static_cast<unsigned char *>(dy) + (size_t)r * H + (size_t)c * 8) =
                        make_uint2(pack_e4m3x4(f[0], f[1], f[2], f[3]), pack_e4m3x4(f[4], f[5], f[6], f[7]));
                    if ((lane & 15) == 0) dy_scale[(size_t)r * (H / 128) + (c >> 4)] = quant_scale(amax);
                } else {
                    st_v4(static_cast<__nv_bfloat16 *>(dy) + (size_t)r * H + (size_t)c * 8, pack_bf16x8(f));
                }
            }
        }
#pragma unroll
        for (int jj = 0; jj < kGradBatch; ++jj) {
            if (j0 + jj >= K) break;
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) acc[jj] += __shfl_xor_sync(0xffffffffu, acc[jj], off);
            if (lane == 0) s_part[warp][j0 + jj] = acc[jj];
        }
    }
    __syncthreads();
    if (threadIdx.x < K) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < kGradThreads / 32; ++i) s += s_part[i][threadIdx.x];
        s_dw[threadIdx.x] = s;
        dtopk_w[g * K + threadIdx.x] = s;
    }
    if (!dlogits) return;
    __syncthreads();
    if (threadIdx.x < K) {
        float mean = 0.0f;
        for (int i = 0; i < K; ++i) mean = __fmaf_rn(s_w[i], s_dw[i], mean);
        const int e = __ldg(topk_idx + g * K + threadIdx.x);
        if (e >= 0 && e < E) s_dl[e] = s_w[threadIdx.x] * (s_dw[threadIdx.x] - mean);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kGradThreads) dlogits[g * E + e] = s_dl[e];
}

cudaError_t launch_combine_backward(const void *dout, const void *y, const int32_t *tok2row, const float *topk_w,
                                    const int32_t *topk_idx, int T, int K, int H, long long rows, int E, bool fp8,
                                    void *dy, float *dy_scale, float *dtopk_w, float *dlogits, cudaStream_t stream) {
    const size_t smem = dlogits ? (size_t)E * 4 : 0;
    const __nv_bfloat16 *db = static_cast<const __nv_bfloat16 *>(dout), *yb = static_cast<const __nv_bfloat16 *>(y);
    if (fp8)
        combine_backward_kernel<true><<<(unsigned)T, kGradThreads, smem, stream>>>(
            db, yb, tok2row, topk_w, topk_idx, T, K, H, rows, E, dy, dy_scale, dtopk_w, dlogits);
    else
        combine_backward_kernel<false><<<(unsigned)T, kGradThreads, smem, stream>>>(
            db, yb, tok2row, topk_w, topk_idx, T, K, H, rows, E, dy, dy_scale, dtopk_w, dlogits);
    return cudaGetLastError();
}

// --------------------------------------------------------------------------
// gate backward
// --------------------------------------------------------------------------
// v = silu(g) * u with s = sigmoid(g):
//   dg = dv * u * s * (1 + g * (1 - s)),   du = dv * g * s.
// A thread owns 8 channels of a row's gate and up halves; FP8: 16 lanes hold a
// block of 128 channels of each half and fold its amax by shuffles.
constexpr int kGateThreads = 256;

template <bool kFp8>
__global__ void __launch_bounds__(kGateThreads) gated_backward_kernel(const __nv_bfloat16 *__restrict__ h,
                                                                      const __nv_bfloat16 *__restrict__ da,
                                                                      long long rows, int I, void *__restrict__ dh,
                                                                      float *__restrict__ dh_scale) {
    const int nchunk = I / 8;
    const long long item = (long long)blockIdx.x * kGateThreads + threadIdx.x;
    const long long row = item / nchunk;
    const int c = (int)(item - row * nchunk);
    const bool in = row < rows;
    float g[8], u[8], d[8];
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    const __nv_bfloat16 *hr = h + (size_t)row * 2 * I + (size_t)c * 8;
    const uint4 vg = in ? ld_stream_v4(hr) : zero;
    const uint4 vu = in ? ld_stream_v4(hr + I) : zero;
    const uint4 vd = in ? ld_stream_v4(da + (size_t)row * I + (size_t)c * 8) : zero;
    unpack_bf16x8(vg, g);
    unpack_bf16x8(vu, u);
    unpack_bf16x8(vd, d);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float s = sigmoid(g[k]);
        const float ds = d[k] * s;
        const float du = ds * g[k];
        g[k] = ds * u[k] * __fmaf_rn(g[k], 1.0f - s, 1.0f);
        u[k] = du;
    }
    if (kFp8) {
        float ag = 0.0f, au = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            ag = fmaxf(ag, fabsf(g[k]));
            au = fmaxf(au, fabsf(u[k]));
        }
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) {
            ag = fmaxf(ag, __shfl_xor_sync(0xffffffffu, ag, off));
            au = fmaxf(au, __shfl_xor_sync(0xffffffffu, au, off));
        }
        if (!in) return;
        ag = quant_amax(ag);
        au = quant_amax(au);
        const float ig = quant_inverse(ag), iu = quant_inverse(au);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            g[k] = __fmul_rn(g[k], ig);
            u[k] = __fmul_rn(u[k], iu);
        }
        unsigned char *o = static_cast<unsigned char *>(dh) + (size_t)row * 2 * I + (size_t)c * 8;
        *reinterpret_cast<uint2 *>(o) =
            make_uint2(pack_e4m3x4(g[0], g[1], g[2], g[3]), pack_e4m3x4(g[4], g[5], g[6], g[7]));
        *reinterpret_cast<uint2 *>(o + I) =
            make_uint2(pack_e4m3x4(u[0], u[1], u[2], u[3]), pack_e4m3x4(u[4], u[5], u[6], u[7]));
        if ((threadIdx.x & 15) == 0) {
            float *sc = dh_scale + (size_t)row * (2 * I / 128) + (c >> 4);
            sc[0] = quant_scale(ag);
            sc[I / 128] = quant_scale(au);
        }
    } else {
        if (!in) return;
        __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(dh) + (size_t)row * 2 * I + (size_t)c * 8;
        st_v4(o, pack_bf16x8(g));
        st_v4(o + I, pack_bf16x8(u));
    }
}

cudaError_t launch_gated_backward(const void *h, const void *da, long long rows, int I, bool fp8, void *dh,
                                  float *dh_scale, cudaStream_t stream) {
    const long long grid = (rows * (I / 8) + kGateThreads - 1) / kGateThreads;
    const __nv_bfloat16 *hb = static_cast<const __nv_bfloat16 *>(h), *db = static_cast<const __nv_bfloat16 *>(da);
    if (fp8)
        gated_backward_kernel<true><<<(unsigned)grid, kGateThreads, 0, stream>>>(hb, db, rows, I, dh, dh_scale);
    else
        gated_backward_kernel<false><<<(unsigned)grid, kGateThreads, 0, stream>>>(hb, db, rows, I, dh, dh_scale);
    return cudaGetLastError();
}

}  // namespace moe
