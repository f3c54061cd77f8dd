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

// Both kernels here start while the kernel before them in the stream runs out,
// wait for it before they read, and let the kernel after do the same.
template <class... Params, class... Args>
static cudaError_t launch_chained(void (*kernel)(Params...), unsigned grid, int threads, size_t smem,
                                  cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

// --------------------------------------------------------------------------
// combine backward
// --------------------------------------------------------------------------
// One block per token.  A thread owns 16-byte chunks (8 channels) of the row:
// for each it loads dout once and the chunk of up to kGradBatch rows of y, all
// in flight together, adds the products to one fp32 sum per row and writes
// w_j * dout.  The sums are folded by shuffles and then, in a fixed order,
// across the warps.  FP8: 16 lanes hold a block of 128 channels; its amax is
// |w_j| * max|dout| (rounding is monotone, so this is the amax of the rounded
// products), one shuffle reduction per block for all K copies.  The 16 lanes
// also share the divisions: for the eight copies under way, eight lanes form
// 448 / amax, the other eight amax / 448 (each lane dividing for itself took a
// third of the kernel's instructions).
//
// Bound by HBM: 32768 tokens, top-8, H = 7168 to FP8 rows and logits move 6.2 GB
// in 929 us (6.68 TB/s, 0.99 of the measured copy rate), to bf16 rows 8.0 GB in
// 1198 us.  Small blocks, many to an SM, keep loads in flight while others
// divide and store: 256 threads x 3 blocks took 1038 us, 128 x 6 950, 128 x 8
// 960; 1003 tokens take 31.0 us, and 37.4 us with 6 blocks, whose last wave is
// nearly empty there.
constexpr int kGradThreads = 128;   // at most
constexpr int kGradBlocks = 7;      // resident blocks the registers are held to (72 a thread)
constexpr int kGradBatch = 8;       // copies whose rows are in flight at once

template <bool kFp8>
__global__ void __launch_bounds__(kGradThreads, kGradBlocks) combine_backward_kernel(
    const __nv_bfloat16 *dout, const __nv_bfloat16 *y, const int32_t *tok2row,
    const float *topk_w, const int32_t *topk_idx, int T, int K, int H, long long rows, int E,
    void *dy, float *dy_scale, float *dtopk_w, float *dlogits) {
    extern __shared__ float s_dl[];   // [E] when dlogits is wanted
    __shared__ int32_t s_row[MOE_MAX_TOPK];
    __shared__ float s_w[MOE_MAX_TOPK];
    __shared__ float s_part[kGradThreads / 32][MOE_MAX_TOPK];
    __shared__ float s_dw[MOE_MAX_TOPK];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nchunk = H / 8;
    const int nchunk_warp = (nchunk + 31) & ~31;   // whole warps, so that the shuffles are uniform
    const long long g = blockIdx.x;
    pdl_launch_dependents();
    pdl_wait();

    if (threadIdx.x < K) {
        const long long r = tok2row ? (long long)ld_chained(tok2row + g * K + threadIdx.x) : g * K + threadIdx.x;
        s_row[threadIdx.x] = (r >= 0 && r < rows) ? (int32_t)r : -1;
        s_w[threadIdx.x] = ld_chained(topk_w + g * K + threadIdx.x);
    }
    if (dlogits)
        for (int e = threadIdx.x; e < E; e += blockDim.x) s_dl[e] = 0.0f;
    __syncthreads();

    for (int j0 = 0; j0 < K; j0 += kGradBatch) {
        float2 acc[kGradBatch];   // even and odd channels
#pragma unroll
        for (int jj = 0; jj < kGradBatch; ++jj) acc[jj] = make_float2(0.0f, 0.0f);
        for (int c = threadIdx.x; c < nchunk_warp; c += blockDim.x) {
            const bool in = c < nchunk;
            uint4 v[kGradBatch];
#pragma unroll
            for (int jj = 0; jj < kGradBatch; ++jj) {
                const int r = (j0 + jj < K) ? s_row[j0 + jj] : -1;
                v[jj] = (in && r >= 0) ? ld_chained_v4(y + (size_t)r * H + (size_t)c * 8) : make_uint4(0u, 0u, 0u, 0u);
            }
            const uint4 dv = in ? ld_chained_v4(dout + (size_t)g * H + (size_t)c * 8)
                                : make_uint4(0u, 0u, 0u, 0u);
            const float2 d[4] = {bf16_pair_floats(dv.x), bf16_pair_floats(dv.y), bf16_pair_floats(dv.z),
                                 bf16_pair_floats(dv.w)};
            float share = 0.0f;   // FP8: 448 / amax of copy lane % 8, or in the upper lanes amax / 448
            if (kFp8) {
                float dmax = 0.0f;
#pragma unroll
                for (int k = 0; k < 4; ++k) dmax = fmaxf(dmax, fmaxf(fabsf(d[k].x), fabsf(d[k].y)));
#pragma unroll
                for (int off = 8; off > 0; off >>= 1) dmax = fmaxf(dmax, __shfl_xor_sync(0xffffffffu, dmax, off));
                const int j = j0 + (lane & 7);
                const float amax = quant_amax(__fmul_rn(j < K ? fabsf(s_w[j]) : 0.0f, dmax));
                share = (lane & 8) ? quant_scale(amax) : quant_inverse(amax);
                const int r = (j < K) ? s_row[j] : -1;
                if ((lane & 8) && in && r >= 0) dy_scale[(size_t)r * (H / 128) + (c >> 4)] = share;
            }
#pragma unroll
            for (int jj = 0; jj < kGradBatch; ++jj) {
                if (j0 + jj >= K) break;
                const float inv = kFp8 ? __shfl_sync(0xffffffffu, share, (lane & 16) + jj) : 0.0f;
                const int r = s_row[j0 + jj];
                if (r < 0 || !in) continue;
                const float w = s_w[j0 + jj];
                const uint32_t q[4] = {v[jj].x, v[jj].y, v[jj].z, v[jj].w};
                float2 f[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    fma_pair(acc[jj], d[k], bf16_pair_floats(q[k]));
                    f[k] = mul_pair(make_float2(w, w), d[k]);
                    if (kFp8) f[k] = mul_pair(f[k], make_float2(inv, inv));
                }
                if (kFp8)
                    *reinterpret_cast<uint2 *>(static_cast<unsigned char *>(dy) + (size_t)r * H + (size_t)c * 8) =
                        make_uint2(pack_e4m3x4(f[0].x, f[0].y, f[1].x, f[1].y),
                                   pack_e4m3x4(f[2].x, f[2].y, f[3].x, f[3].y));
                else
                    st_v4(static_cast<__nv_bfloat16 *>(dy) + (size_t)r * H + (size_t)c * 8,
                          make_uint4(bf16_pair(f[0].x, f[0].y), bf16_pair(f[1].x, f[1].y),
                                     bf16_pair(f[2].x, f[2].y), bf16_pair(f[3].x, f[3].y)));
            }
        }
#pragma unroll
        for (int jj = 0; jj < kGradBatch; ++jj) {
            if (j0 + jj >= K) break;
            float sum = acc[jj].x + acc[jj].y;
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            if (lane == 0) s_part[warp][j0 + jj] = sum;
        }
    }
    __syncthreads();
    if (threadIdx.x < K) {
        float s = 0.0f;
        for (int i = 0; i < (int)blockDim.x / 32; ++i) s += s_part[i][threadIdx.x];
        s_dw[threadIdx.x] = s;
        dtopk_w[g * K + threadIdx.x] = s;
    }
    if (!dlogits) return;
    __syncthreads();
    if (threadIdx.x < K) {
        float mean = 0.0f;
        for (int i = 0; i < K; ++i) mean = __fmaf_rn(s_w[i], s_dw[i], mean);
        const int e = ld_chained(topk_idx + g * K + threadIdx.x);
        if (e >= 0 && e < E) s_dl[e] = s_w[threadIdx.x] * (s_dw[threadIdx.x] - mean);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) dlogits[g * E + e] = s_dl[e];
}

cudaError_t launch_combine_backward(const void *dout, const void *y, const int32_t *tok2row, const float *topk_w,
                                    const int32_t *topk_idx, int T, int K, int H, long long rows, int E, bool fp8,
                                    void *dy, float *dy_scale, float *dtopk_w, float *dlogits, cudaStream_t stream) {
    const size_t smem = dlogits ? (size_t)E * 4 : 0;
    // as many whole warps as share the row's chunks evenly (H = 7168: 128 threads, 7 chunks each)
    const int nchunk = H / 8, rounds = (nchunk + kGradThreads - 1) / kGradThreads;
    const int threads = ((nchunk + rounds - 1) / rounds + 31) / 32 * 32;
    const __nv_bfloat16 *db = static_cast<const __nv_bfloat16 *>(dout), *yb = static_cast<const __nv_bfloat16 *>(y);
    return launch_chained(fp8 ? combine_backward_kernel<true> : combine_backward_kernel<false>, (unsigned)T, threads,
                          smem, stream, db, yb, tok2row, topk_w, topk_idx, T, K, H, rows, E, dy, dy_scale, dtopk_w,
                          dlogits);
}

// --------------------------------------------------------------------------
// gate backward
// --------------------------------------------------------------------------
// v = silu(g) * u with s = sigmoid(g):
//   dg = dv * u * s * (1 + g * (1 - s)),   du = dv * g * s.
// A thread owns chunks of 8 channels of a row's gate and up halves; FP8: 16
// lanes hold a block of 128 channels of each half and fold its amax by
// shuffles.
//
// Bound by HBM: 262144 rows of I = 2048 move 4.33 GB to FP8 in 665 us (6.51
// TB/s, 0.96 of the measured copy rate) and 5.37 GB to bf16 in 755 us (1.05).
// With one chunk a thread the FP8 form took 729 us (the arithmetic of a block
// left too few loads in flight); 256 threads with two chunks 699 us; with expf
// and an IEEE division per channel 807 us.
constexpr int kGateThreads = 128;
constexpr int kGateChunks = 2;   // per thread, all loaded before the first is used
static_assert(kGatedBackwardMost == ((1ll << 31) - 1) * kGateThreads * kGateChunks * 8, "the channels of a grid");

template <bool kFp8>
__global__ void __launch_bounds__(kGateThreads) gated_backward_kernel(const __nv_bfloat16 *h,
                                                                      const __nv_bfloat16 *da,
                                                                      long long rows, int I, void *dh,
                                                                      float *dh_scale) {
    pdl_launch_dependents();
    pdl_wait();
    const uint32_t nchunk = I / 8;
    const int lane = threadIdx.x & 31;
    // this block's first chunk of 8 channels, by one 64-bit division of the block
    const unsigned long long first = (unsigned long long)blockIdx.x * (kGateThreads * kGateChunks);
    const unsigned long long row0 = first / nchunk;
    uint4 vg[kGateChunks], vu[kGateChunks], vd[kGateChunks];
    size_t at[kGateChunks];   // of the gate's chunk in h and dh
    int chunk[kGateChunks];
    bool in[kGateChunks];
#pragma unroll
    for (int i = 0; i < kGateChunks; ++i) {   // every load before the first use
        const uint32_t n = (uint32_t)(first - row0 * nchunk) + i * kGateThreads + threadIdx.x;
        const long long row = (long long)(row0 + n / nchunk);
        chunk[i] = (int)(n % nchunk);
        in[i] = row < rows;
        at[i] = (size_t)row * 2 * I + (size_t)chunk[i] * 8;
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        vg[i] = in[i] ? ld_chained_v4(h + at[i]) : zero;
        vu[i] = in[i] ? ld_chained_v4(h + at[i] + I) : zero;
        vd[i] = in[i] ? ld_chained_v4(da + (size_t)row * I + (size_t)chunk[i] * 8) : zero;
    }
#pragma unroll
    for (int i = 0; i < kGateChunks; ++i) {
        float g[8], u[8], d[8];
        unpack_bf16x8(vg[i], g);
        unpack_bf16x8(vu[i], u);
        unpack_bf16x8(vd[i], d);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float s = sigmoid_fast(g[k]);
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
            // of 16 lanes with the same maxima, each divides once: 448 / ag, ag / 448, and so for au
            const float amax = quant_amax((lane & 2) ? au : ag);
            const float share = (lane & 1) ? quant_scale(amax) : quant_inverse(amax);
            const float ig = __shfl_sync(0xffffffffu, share, lane & 16);
            const float iu = __shfl_sync(0xffffffffu, share, (lane & 16) + 2);
            if (!in[i]) continue;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                g[k] = __fmul_rn(g[k], ig);
                u[k] = __fmul_rn(u[k], iu);
            }
            unsigned char *o = static_cast<unsigned char *>(dh) + at[i];
            *reinterpret_cast<uint2 *>(o) =
                make_uint2(pack_e4m3x4(g[0], g[1], g[2], g[3]), pack_e4m3x4(g[4], g[5], g[6], g[7]));
            *reinterpret_cast<uint2 *>(o + I) =
                make_uint2(pack_e4m3x4(u[0], u[1], u[2], u[3]), pack_e4m3x4(u[4], u[5], u[6], u[7]));
            if ((lane & 13) == 1)   // at[i] / 128 is the gate's block
                dh_scale[(at[i] >> 7) + ((lane & 2) ? I / 128 : 0)] = share;
        } else if (in[i]) {
            __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(dh) + at[i];
            st_v4(o, pack_bf16x8(g));
            st_v4(o + I, pack_bf16x8(u));
        }
    }
}

cudaError_t launch_gated_backward(const void *h, const void *da, long long rows, int I, bool fp8, void *dh,
                                  float *dh_scale, cudaStream_t stream) {
    const long long per = kGateThreads * kGateChunks, grid = (rows * (I / 8) + per - 1) / per;
    const __nv_bfloat16 *hb = static_cast<const __nv_bfloat16 *>(h), *db = static_cast<const __nv_bfloat16 *>(da);
    return launch_chained(fp8 ? gated_backward_kernel<true> : gated_backward_kernel<false>, (unsigned)grid,
                          kGateThreads, 0, stream, hb, db, rows, I, dh, dh_scale);
}

}  // namespace moe
