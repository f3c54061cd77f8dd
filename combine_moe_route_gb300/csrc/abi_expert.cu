// abi_expert.cu -- the extern "C" entry points of the expert products, the 4-bit
// rows, the norm and the gradients (declared and documented in include/moe_route.h): host-side
// argument validation and the kernel launches.  As in abi.cu, nothing here
// allocates or synchronises, and validation runs before the first CUDA call.
#include <cuda_runtime.h>
#include <stdint.h>

#include "launch.h"
#include "moe_route.h"

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// A failure is reported here and nowhere else: left as the thread's last error, it would be the
// next launch's.
moe_status cuda_status(cudaError_t e) {
    if (e == cudaSuccess) return MOE_OK;
    (void)cudaGetLastError();
    return MOE_ERR_CUDA;
}

bool expert_dim_ok(int d, int multiple) { return d >= multiple && d <= MOE_MAX_EXPERT_DIM && d % multiple == 0; }

bool hidden_ok(int H) { return H >= 8 && H <= MOE_MAX_HIDDEN && H % 8 == 0; }

}  // namespace

extern "C" {

moe_status moe_expert_gemm(const void *a, const float *a_scale, const void *w, const float *w_scale,
                           const int32_t *expert_offsets, int E, int N, int C, int rows, int transpose,
                           moe_dtype out_dtype, void *out, moe_stream_t stream) {
    if (E < 1 || E > MOE_MAX_EXPERTS || rows < 0) return MOE_ERR_INVALID_ARG;
    if (!expert_dim_ok(N, 16) || !expert_dim_ok(C, 16)) return MOE_ERR_INVALID_ARG;
    if (out_dtype != MOE_DTYPE_BF16 && out_dtype != MOE_DTYPE_FP32) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if (!a || !a_scale || !w || !w_scale || !expert_offsets || !out) return MOE_ERR_INVALID_ARG;
    if (!aligned16(a) || !aligned16(w) || !aligned16(out)) return MOE_ERR_UNSUPPORTED;
    return cuda_status(moe::launch_expert_gemm(a, a_scale, w, w_scale, expert_offsets, E, N, C, rows, transpose != 0,
                                               out_dtype == MOE_DTYPE_FP32, out, (cudaStream_t)stream));
}

moe_status moe_expert_gated_gemm(const void *a, const float *a_scale, const void *w, const float *w_scale,
                                 const int32_t *expert_offsets, int E, int I, int C, int rows, void *q, float *q_scale,
                                 void *h, moe_stream_t stream) {
    if (E < 1 || E > MOE_MAX_EXPERTS || rows < 0) return MOE_ERR_INVALID_ARG;
    if (I < 128 || I > MOE_MAX_EXPERT_DIM / 2 || I % 128 != 0 || !expert_dim_ok(C, 16)) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if (!a || !a_scale || !w || !w_scale || !expert_offsets || !q || !q_scale) return MOE_ERR_INVALID_ARG;
    if (!aligned16(a) || !aligned16(w) || !aligned16(q) || !aligned16(h)) return MOE_ERR_UNSUPPORTED;
    return cuda_status(moe::launch_expert_gated_gemm(a, a_scale, w, w_scale, expert_offsets, E, I, C, rows, q, q_scale,
                                                     h, (cudaStream_t)stream));
}

moe_status moe_quantize_mx4(const void *x, moe_dtype x_dtype, int64_t rows, int C, void *q, void *scale,
                            moe_stream_t stream) {
    if (rows < 0 || C < 32 || C % 32 != 0) return MOE_ERR_INVALID_ARG;
    if (x_dtype != MOE_DTYPE_BF16 && x_dtype != MOE_DTYPE_FP32) return MOE_ERR_INVALID_ARG;
    if (rows > moe::kMx4Most / (C / 32)) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if (!x || !q || !scale) return MOE_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(q)) return MOE_ERR_UNSUPPORTED;
    return cuda_status(moe::launch_quantize_mx4(x, x_dtype == MOE_DTYPE_FP32, rows * (C / 32), q, scale,
                                                (cudaStream_t)stream));
}

moe_status moe_dequantize_mx4(const void *q, const void *scale, int64_t rows, int C, moe_dtype out_dtype, void *out,
                              moe_stream_t stream) {
    if (rows < 0 || C < 32 || C % 32 != 0) return MOE_ERR_INVALID_ARG;
    if (out_dtype != MOE_DTYPE_BF16 && out_dtype != MOE_DTYPE_FP8_E4M3) return MOE_ERR_INVALID_ARG;
    if (rows > moe::kMx4Most / (C / 32)) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if ((out_dtype == MOE_DTYPE_FP8_E4M3) != (scale == nullptr)) return MOE_ERR_INVALID_ARG;
    if (!q || !out) return MOE_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(out)) return MOE_ERR_UNSUPPORTED;
    return cuda_status(moe::launch_dequantize_mx4(q, scale, rows * (C / 32), out, (cudaStream_t)stream));
}

moe_status moe_expert_gemm_mx4(const void *a, const void *a_scale, const void *w, const void *w_scale,
                               const int32_t *expert_offsets, int E, int N, int C, int rows, moe_dtype out_dtype,
                               void *out, moe_stream_t stream) {
    if (E < 1 || E > MOE_MAX_EXPERTS || rows < 0) return MOE_ERR_INVALID_ARG;
    if (!expert_dim_ok(N, 16) || !expert_dim_ok(C, 32)) return MOE_ERR_INVALID_ARG;
    if (out_dtype != MOE_DTYPE_BF16 && out_dtype != MOE_DTYPE_FP32) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if (!a || !a_scale || !w || !w_scale || !expert_offsets || !out) return MOE_ERR_INVALID_ARG;
    if (!aligned16(a) || !aligned16(w) || !aligned16(out)) return MOE_ERR_UNSUPPORTED;
    return cuda_status(moe::launch_expert_gemm_mx4(a, a_scale, w, w_scale, expert_offsets, E, N, C, rows,
                                                   out_dtype == MOE_DTYPE_FP32, out, (cudaStream_t)stream));
}

moe_status moe_expert_gated_gemm_mx4(const void *a, const void *a_scale, const void *w, const void *w_scale,
                                     const int32_t *expert_offsets, int E, int I, int C, int rows, void *q,
                                     void *q_scale, moe_stream_t stream) {
    if (E < 1 || E > MOE_MAX_EXPERTS || rows < 0) return MOE_ERR_INVALID_ARG;
    if (I < 32 || I > MOE_MAX_EXPERT_DIM / 2 || I % 32 != 0 || !expert_dim_ok(C, 32)) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if (!a || !a_scale || !w || !w_scale || !expert_offsets || !q || !q_scale) return MOE_ERR_INVALID_ARG;
    if (!aligned16(a) || !aligned16(w) || !aligned16(q)) return MOE_ERR_UNSUPPORTED;
    return cuda_status(moe::launch_expert_gated_gemm_mx4(a, a_scale, w, w_scale, expert_offsets, E, I, C, rows, q,
                                                         q_scale, (cudaStream_t)stream));
}

moe_status moe_rms_norm(const void *x, const void *residual, const void *weight, int T, int H, float eps, void *y,
                        void *h, void *q, float *q_scale, moe_stream_t stream) {
    if (T < 0 || !hidden_ok(H) || !(eps >= 0.0f)) return MOE_ERR_INVALID_ARG;
    if (q && H % 128 != 0) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    if (!x || !weight || !y || (residual != nullptr) != (h != nullptr) || (q && !q_scale)) return MOE_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(residual) || !aligned16(weight) || !aligned16(y) || !aligned16(h) || !aligned16(q))
        return MOE_ERR_UNSUPPORTED;
    return cuda_status(moe::launch_rms_norm(x, residual, weight, T, H, eps, y, h, q, q_scale, (cudaStream_t)stream));
}

size_t moe_rms_norm_workspace_bytes(int T, int H) {
    return T > 0 && hidden_ok(H) ? moe::norm_workspace_bytes(T, H) : 0;
}

moe_status moe_rms_norm_backward(const void *dy, const void *h, const void *weight, const void *dh, int T, int H,
                                 float eps, void *dx, float *dweight, void *workspace, size_t workspace_bytes,
                                 moe_stream_t stream) {
    if (T < 0 || !hidden_ok(H) || !(eps >= 0.0f) || !dweight) return MOE_ERR_INVALID_ARG;
    if (T > 0 && (!dy || !h || !weight || !dx)) return MOE_ERR_INVALID_ARG;
    const size_t need = moe_rms_norm_workspace_bytes(T, H);
    if (need > 0 && (!workspace || workspace_bytes < need)) return MOE_ERR_WORKSPACE;
    if (!aligned16(dy) || !aligned16(h) || !aligned16(weight) || !aligned16(dh) || !aligned16(dx) ||
        !aligned16(workspace))
        return MOE_ERR_UNSUPPORTED;
    return cuda_status(moe::launch_rms_norm_backward(dy, h, weight, dh, T, H, eps, dx, dweight, workspace,
                                                     (cudaStream_t)stream));
}

moe_status moe_get_expert_error(int32_t *host_code, moe_stream_t stream) {
    if (!host_code) return MOE_ERR_INVALID_ARG;
    const moe_status read = cuda_status(moe::read_product_error(host_code, (cudaStream_t)stream));
    return *host_code ? MOE_ERR_TIMEOUT : read;
}

moe_status moe_expert_gated_backward(const void *h, const void *dv, int rows, int I, moe_dtype dh_dtype, void *dh,
                                     float *dh_scale, moe_stream_t stream) {
    if (rows < 0 || I < 8 || I > MOE_MAX_EXPERT_DIM / 2 || I % 8 != 0) return MOE_ERR_INVALID_ARG;
    if ((long long)rows * I > moe::kGatedBackwardMost) return MOE_ERR_INVALID_ARG;
    if (dh_dtype != MOE_DTYPE_BF16 && dh_dtype != MOE_DTYPE_FP8_E4M3) return MOE_ERR_INVALID_ARG;
    const bool fp8 = dh_dtype == MOE_DTYPE_FP8_E4M3;
    if (fp8 && I % 128 != 0) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if (!h || !dv || !dh || (fp8 && !dh_scale)) return MOE_ERR_INVALID_ARG;
    if (!aligned16(h) || !aligned16(dv) || !aligned16(dh)) return MOE_ERR_UNSUPPORTED;
    return cuda_status(moe::launch_gated_backward(h, dv, rows, I, fp8, dh, dh_scale, (cudaStream_t)stream));
}

moe_status moe_combine_backward(const void *dout, const void *y, const int32_t *tok2row, const float *topk_w,
                                const int32_t *topk_idx, int T, int K, int H, int64_t rows, int E, moe_dtype dy_dtype,
                                void *dy, float *dy_scale, float *dtopk_w, float *dlogits, moe_stream_t stream) {
    if (T < 0 || K < 1 || K > MOE_MAX_TOPK || !hidden_ok(H)) return MOE_ERR_INVALID_ARG;
    if ((long long)T * K >= (1ll << 31) || rows < 0 || rows >= (1ll << 31)) return MOE_ERR_INVALID_ARG;
    if (dy_dtype != MOE_DTYPE_BF16 && dy_dtype != MOE_DTYPE_FP8_E4M3) return MOE_ERR_INVALID_ARG;
    const bool fp8 = dy_dtype == MOE_DTYPE_FP8_E4M3;
    if (fp8 && H % 128 != 0) return MOE_ERR_INVALID_ARG;
    if (dlogits && (E < 1 || E > MOE_MAX_EXPERTS)) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    if (!dout || !topk_w || !dtopk_w || (dlogits && !topk_idx)) return MOE_ERR_INVALID_ARG;
    if (rows > 0 && (!y || !dy || (fp8 && !dy_scale))) return MOE_ERR_INVALID_ARG;
    if (!aligned16(dout) || !aligned16(y) || !aligned16(dy)) return MOE_ERR_UNSUPPORTED;
    return cuda_status(moe::launch_combine_backward(dout, y, tok2row, topk_w, topk_idx, T, K, H, rows, E, fp8, dy,
                                                    dy_scale, dtopk_w, dlogits, (cudaStream_t)stream));
}

moe_status moe_dispatch_backward(const void *drows, const int32_t *tok2row, int T, int K, int H, int64_t rows,
                                 moe_dtype out_dtype, void *dx, moe_stream_t stream) {
    if (T < 0 || K < 1 || K > MOE_MAX_TOPK || !hidden_ok(H)) return MOE_ERR_INVALID_ARG;
    if ((long long)T * K >= (1ll << 31) || rows < 0 || rows >= (1ll << 31)) return MOE_ERR_INVALID_ARG;
    if (out_dtype != MOE_DTYPE_BF16 && out_dtype != MOE_DTYPE_FP32) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    if (!tok2row || !dx || (rows > 0 && !drows)) return MOE_ERR_INVALID_ARG;
    if (!aligned16(drows) || !aligned16(dx)) return MOE_ERR_UNSUPPORTED;
    return cuda_status(moe::launch_dispatch_backward(drows, tok2row, T, K, H, rows, out_dtype == MOE_DTYPE_FP32, dx,
                                                     (cudaStream_t)stream));
}

}  // extern "C"
