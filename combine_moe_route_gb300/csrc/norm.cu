// norm.cu -- the root-mean-square norm in front of a layer, with the residual's
// addition and, where wanted, e4m3 rows beside the bf16 ones; and its gradient.
//
//   s = x + residual,   r = 1 / sqrt(mean(s^2) + eps),   y = s * r * weight
//
// and for dy = dL/dy, with h = s and g = dy * weight,
//
//   dx = r * (g - h * r * mean(g * h) * r) + dh,   dweight = sum over rows of dy * h * r,
//
// where dh is the gradient that reaches s past the norm.  All sums are fp32.
//
// A team of 32, 128 or 256 threads holds a row in registers, 8 channels a chunk,
// so that it is read once; 16 neighbouring lanes hold a block of 128 channels.
#include "launch.h"
#include "numeric.cuh"

namespace moe {

// The sum over a team's threads, in an order that does not change.  `part`: a
// slot for each of the team's warps.
template <int kTeam, int kSums>
__device__ __forceinline__ void team_sums(float (&v)[kSums], float (*part)[kSums]) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
#pragma unroll
        for (int i = 0; i < kSums; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], off);
    if constexpr (kTeam > 32) {
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int i = 0; i < kSums; ++i) part[threadIdx.x >> 5][i] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kSums; ++i) {
            v[i] = 0.0f;
#pragma unroll
            for (int w = 0; w < kTeam / 32; ++w) v[i] += part[w][i];
        }
    }
}

template <int kTeam>
__host__ __device__ constexpr int norm_threads() {
    return kTeam < 128 ? 128 : kTeam;   // small teams share a block
}

template <int kTeam, int kChunks, bool kFp8>
__global__ void __launch_bounds__(norm_threads<kTeam>()) rms_norm_kernel(const __nv_bfloat16 *x,
                                                                         const __nv_bfloat16 *residual,
                                                                         const __nv_bfloat16 *weight, long long T, int H,
                                                                         float eps, __nv_bfloat16 *y, __nv_bfloat16 *h,
                                                                         unsigned char *q, float *q_scale) {
    constexpr int kTeams = norm_threads<kTeam>() / kTeam;
    __shared__ float s_part[norm_threads<kTeam>() / 32][1];
    const int nchunk = H / 8, at = threadIdx.x % kTeam;
    const long long row = (long long)blockIdx.x * kTeams + threadIdx.x / kTeam;
    pdl_launch_dependents();
    pdl_wait();
    if (row >= T) return;   // whole warps: a block of several teams has teams of one warp
    const size_t from = (size_t)row * H;
    uint4 v[kChunks], w[kChunks];
    float f[kChunks][8];
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        const int c = at + i * kTeam;
        v[i] = c < nchunk ? ld_chained_v4(x + from + c * 8) : make_uint4(0u, 0u, 0u, 0u);
    }
    if (residual) {
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            const int c = at + i * kTeam;
            w[i] = c < nchunk ? ld_chained_v4(residual + from + c * 8) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            const int c = at + i * kTeam;
            float a[8];
            unpack_bf16x8(v[i], f[i]);
            unpack_bf16x8(w[i], a);
#pragma unroll
            for (int k = 0; k < 8; ++k) f[i][k] += a[k];
            if (c < nchunk) st_v4(h + from + c * 8, pack_bf16x8(f[i]));
        }
    } else {
#pragma unroll
        for (int i = 0; i < kChunks; ++i) unpack_bf16x8(v[i], f[i]);
    }
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {   // in flight over the sum
        const int c = at + i * kTeam;
        w[i] = c < nchunk ? ld_cached_v4(weight + c * 8) : make_uint4(0u, 0u, 0u, 0u);
    }
    float sum[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) sum[0] = fmaf(f[i][k], f[i][k], sum[0]);
    team_sums<kTeam, 1>(sum, s_part);
    const float r = rsqrtf(sum[0] / (float)H + eps);
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        const int c = at + i * kTeam;
        float g[8];
        unpack_bf16x8(w[i], g);
#pragma unroll
        for (int k = 0; k < 8; ++k) g[k] *= f[i][k] * r;
        if (c < nchunk) st_v4(y + from + c * 8, pack_bf16x8(g));
        if constexpr (kFp8) {
            // H is a multiple of 128 here: 16 lanes are all inside the row or all outside
            float amax = 0.0f;
#pragma unroll
            for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fabsf(g[k]));
#pragma unroll
            for (int off = 8; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
            amax = quant_amax(amax);
            const float inv = quant_inverse(amax);
            if (c < nchunk) {
                *reinterpret_cast<uint2 *>(q + from + c * 8) =
                    make_uint2(pack_e4m3x4(g[0] * inv, g[1] * inv, g[2] * inv, g[3] * inv),
                               pack_e4m3x4(g[4] * inv, g[5] * inv, g[6] * inv, g[7] * inv));
                if ((at & 15) == 0) q_scale[(size_t)row * (H / 128) + (c >> 4)] = quant_scale(amax);
            }
        }
    }
}

template <int kTeam, int kChunks>
static cudaError_t launch_norm(const void *x, const void *residual, const void *weight, long long T, int H, float eps,
                               void *y, void *h, void *q, float *q_scale, cudaStream_t stream) {
    constexpr int kThreads = norm_threads<kTeam>();
    const unsigned grid = (unsigned)((T + kThreads / kTeam - 1) / (kThreads / kTeam));
    return launch_chained(q ? rms_norm_kernel<kTeam, kChunks, true> : rms_norm_kernel<kTeam, kChunks, false>, grid,
                          kThreads, 0, stream, static_cast<const __nv_bfloat16 *>(x),
                          static_cast<const __nv_bfloat16 *>(residual), static_cast<const __nv_bfloat16 *>(weight), T,
                          H, eps, static_cast<__nv_bfloat16 *>(y), static_cast<__nv_bfloat16 *>(h),
                          static_cast<unsigned char *>(q), q_scale);
}

cudaError_t launch_rms_norm(const void *x, const void *residual, const void *weight, long long T, int H, float eps,
                            void *y, void *h, void *q, float *q_scale, cudaStream_t stream) {
    const int nchunk = H / 8;
#define MOE_NORM(team, chunks) \
    if (nchunk <= team * chunks) \
        return launch_norm<team, chunks>(x, residual, weight, T, H, eps, y, h, q, q_scale, stream)
    MOE_NORM(32, 1);
    MOE_NORM(32, 2);
    MOE_NORM(32, 4);
    MOE_NORM(128, 2);
    MOE_NORM(128, 3);
    MOE_NORM(128, 4);
    MOE_NORM(128, 5);
    MOE_NORM(128, 6);
    MOE_NORM(128, 7);
    MOE_NORM(128, 8);
    MOE_NORM(256, 6);
    MOE_NORM(256, 8);
#undef MOE_NORM
    return cudaErrorInvalidValue;
}

// --------------------------------------------------------------------------
// gradient
// --------------------------------------------------------------------------
// Teams walk the rows; each keeps its sums of dweight in registers and leaves
// them as a row of the workspace, which a second kernel adds up in order.
constexpr int kNormGrid = 456;   // blocks at most: three on each of 152 SMs

template <int kTeam, int kChunks>
__global__ void __launch_bounds__(norm_threads<kTeam>(), 2) rms_norm_backward_kernel(
    const __nv_bfloat16 *dy, const __nv_bfloat16 *h, const __nv_bfloat16 *weight, const __nv_bfloat16 *dh, long long T,
    int H, float eps, __nv_bfloat16 *dx, float *partial) {
    constexpr int kTeams = norm_threads<kTeam>() / kTeam;
    __shared__ float s_part[2][norm_threads<kTeam>() / 32][2];
    const int nchunk = H / 8, at = threadIdx.x % kTeam;
    const long long team = (long long)blockIdx.x * kTeams + threadIdx.x / kTeam;
    pdl_launch_dependents();
    pdl_wait();
    float acc[kChunks][8];
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[i][k] = 0.0f;
    int turn = 0;   // the sums' slots alternate, so that one barrier a row is enough
    for (long long row = team; row < T; row += (long long)gridDim.x * kTeams, turn ^= 1) {
        const size_t from = (size_t)row * H;
        uint4 hv[kChunks], gv[kChunks];
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            const int c = at + i * kTeam;
            hv[i] = c < nchunk ? ld_chained_v4(h + from + c * 8) : make_uint4(0u, 0u, 0u, 0u);
            gv[i] = c < nchunk ? ld_chained_v4(dy + from + c * 8) : make_uint4(0u, 0u, 0u, 0u);
        }
        float sum[2] = {0.0f, 0.0f};   // of h^2 and of g * h
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            const int c = at + i * kTeam;
            float a[8], d[8], w[8];
            unpack_bf16x8(hv[i], a);
            unpack_bf16x8(gv[i], d);
            unpack_bf16x8(c < nchunk ? ld_cached_v4(weight + c * 8) : make_uint4(0u, 0u, 0u, 0u), w);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                sum[0] = fmaf(a[k], a[k], sum[0]);
                sum[1] = fmaf(d[k] * w[k], a[k], sum[1]);
            }
        }
        team_sums<kTeam, 2>(sum, s_part[turn]);
        const float r = rsqrtf(sum[0] / (float)H + eps);
        const float m = sum[1] / (float)H * r * r;   // mean(g n) r: of h * r taken from g
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            const int c = at + i * kTeam;
            if (c >= nchunk) break;
            float a[8], d[8], w[8], o[8];
            if (dh) unpack_bf16x8(ld_chained_v4(dh + from + c * 8), o);
            unpack_bf16x8(hv[i], a);
            unpack_bf16x8(gv[i], d);
            unpack_bf16x8(ld_cached_v4(weight + c * 8), w);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                acc[i][k] = fmaf(d[k], a[k] * r, acc[i][k]);
                const float t = r * (d[k] * w[k] - a[k] * m);
                o[k] = dh ? t + o[k] : t;
            }
            st_v4(dx + from + c * 8, pack_bf16x8(o));
        }
    }
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        const int c = at + i * kTeam;
        if (c >= nchunk) break;
        float4 *to = reinterpret_cast<float4 *>(partial + (size_t)team * H + c * 8);
        to[0] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
        to[1] = make_float4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
    }
}

// Columns of the partial rows: 32 a block, its 8 warps a run of rows each.
__global__ void __launch_bounds__(256) norm_columns_kernel(const float *partial, int parts, int H, float *dweight) {
    __shared__ float s_sum[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    pdl_launch_dependents();
    pdl_wait();
    float sum = 0.0f;
    if (c < H)
        for (int i = warp; i < parts; i += 8) sum += ld_chained(partial + (size_t)i * H + c);
    s_sum[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && c < H) {
#pragma unroll
        for (int w = 1; w < 8; ++w) sum += s_sum[w][lane];
        dweight[c] = sum;
    }
}

static int team_of(int H) { return H <= 32 * 4 * 8 ? 32 : H <= 128 * 8 * 8 ? 128 : 256; }
static int teams_a_block(int H) { return team_of(H) == 32 ? 4 : 1; }
static int norm_grid(long long T, int H) {
    const int teams = teams_a_block(H);
    const long long blocks = (T + teams - 1) / teams;
    return (int)(blocks < kNormGrid ? blocks : kNormGrid);
}

size_t norm_workspace_bytes(long long T, int H) {
    return (size_t)norm_grid(T, H) * teams_a_block(H) * H * sizeof(float);
}

template <int kTeam, int kChunks>
static cudaError_t launch_norm_backward(const void *dy, const void *h, const void *weight, const void *dh, long long T,
                                        int H, float eps, void *dx, float *partial, cudaStream_t stream) {
    return launch_chained(rms_norm_backward_kernel<kTeam, kChunks>, (unsigned)norm_grid(T, H), norm_threads<kTeam>(), 0,
                          stream, static_cast<const __nv_bfloat16 *>(dy), static_cast<const __nv_bfloat16 *>(h),
                          static_cast<const __nv_bfloat16 *>(weight), static_cast<const __nv_bfloat16 *>(dh), T, H, eps,
                          static_cast<__nv_bfloat16 *>(dx), partial);
}

static cudaError_t launch_rows_backward(const void *dy, const void *h, const void *weight, const void *dh, long long T,
                                        int H, float eps, void *dx, float *partial, cudaStream_t stream) {
    const int nchunk = H / 8;
#define MOE_NORM(team, chunks) \
    if (nchunk <= team * chunks) \
        return launch_norm_backward<team, chunks>(dy, h, weight, dh, T, H, eps, dx, partial, stream)
    MOE_NORM(32, 1);
    MOE_NORM(32, 2);
    MOE_NORM(32, 4);
    MOE_NORM(128, 2);
    MOE_NORM(128, 3);
    MOE_NORM(128, 4);
    MOE_NORM(128, 5);
    MOE_NORM(128, 6);
    MOE_NORM(128, 7);
    MOE_NORM(128, 8);
    MOE_NORM(256, 6);
    MOE_NORM(256, 8);
#undef MOE_NORM
    return cudaErrorInvalidValue;
}

cudaError_t launch_rms_norm_backward(const void *dy, const void *h, const void *weight, const void *dh, long long T,
                                     int H, float eps, void *dx, float *dweight, void *workspace, cudaStream_t stream) {
    if (T == 0) return cudaMemsetAsync(dweight, 0, (size_t)H * sizeof(float), stream);
    float *partial = static_cast<float *>(workspace);
    const cudaError_t e = launch_rows_backward(dy, h, weight, dh, T, H, eps, dx, partial, stream);
    if (e != cudaSuccess) return e;
    return launch_chained(norm_columns_kernel, (unsigned)((H + 31) / 32), 256, 0, stream,
                          static_cast<const float *>(partial), norm_grid(T, H) * teams_a_block(H), H, dweight);
}

}  // namespace moe
