// product.cuh -- what the experts' products in e4m3 and in 4 bits share: where an
// expert's rows lie, rings of stages, the output's way to memory, and the host's
// tensor maps.
#pragma once

#include <atomic>

#include "numeric.cuh"
#include "tcgen05.cuh"

namespace moe {

constexpr int kProductThreads = 384;
constexpr int kRowTile = 128;     // rows of a tile: the M of one product
constexpr int kFewRows = 32;      // rows of the small load of A
constexpr int kStagingWarp = 32 * 64;       // output staging of a warp: 32 rows x 64 bytes
constexpr int kTmemColumns = 512;

// Position in a ring of n slots and the parity of its current pass.
struct Ring {
    int slot = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void advance(int n) {
        if (++slot == n) {
            slot = 0;
            parity ^= 1u;
        }
    }
};

// Expert e's first row and number of rows, inside [0, rows] whatever the offsets hold.
template <class Args>
__device__ __forceinline__ int2 expert_rows(const Args &p, int e) {
    const int lo = min(max(ld_chained(p.expert_offsets + e), 0), p.rows);
    const int hi = min(max(ld_chained(p.expert_offsets + e + 1), 0), p.rows);
    return make_int2(lo, max(hi - lo, 0));
}

// Bytes that a row tile's load of A brings.
__device__ __forceinline__ uint32_t row_load_bytes(int valid) {
    return valid > kFewRows ? kRowTile * 128 : valid > 0 ? kFewRows * 128 : 0;
}

// 64 bytes of each of a warp's 32 rows (a lane holds its row's) to global
// memory, four lanes per row, through the warp's staging, which is swizzled
// against bank conflicts.  (Each lane writing its own row took three times as
// long: 32 lines a store.)  `dst` is the address in the warp's row 0, rows lie
// `pitch` bytes apart.  `keep`: which rows to write, a bit each (kMask) or the first
// so many (a mask's bits cost a product's tiles 2 %); bytes at or past `limit`
// are not written.
template <bool kMask>
__device__ __forceinline__ void store_rows64(const uint4 (&v)[4], uint32_t stage, unsigned char *dst, size_t pitch,
                                             uint32_t keep, int limit, int lane) {
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 4; ++c) st_shared_v4(stage + lane * 64 + ((c ^ ((lane >> 1) & 3)) * 16), v[c]);
    __syncwarp();
    const int c = lane & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = i * 8 + (lane >> 2);
        const uint4 x = ld_shared_v4(stage + r * 64 + ((c ^ ((r >> 1) & 3)) * 16));
        const bool kept = kMask ? (keep >> r & 1u) != 0 : r < (int)keep;
        if (kept && c * 16 < limit) st_v4(dst + (size_t)r * pitch + c * 16, x);
    }
}

// 64 fp32 values of a row, as bf16.
template <bool kMask>
__device__ __forceinline__ void store_bf16x64(const float2 *acc, uint32_t stage, unsigned char *dst, size_t pitch,
                                              uint32_t keep, int limit, int lane) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        uint4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 *a = acc + c * 16 + i * 4;
            v[i] = make_uint4(bf16_pair(a[0].x, a[0].y), bf16_pair(a[1].x, a[1].y), bf16_pair(a[2].x, a[2].y),
                              bf16_pair(a[3].x, a[3].y));
        }
        store_rows64<kMask>(v, stage, dst + c * 64, pitch, keep, limit - c * 64, lane);
    }
}

// ------------------------------------------------------------------- host

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiled encode_tiled() {
    static std::atomic<EncodeTiled> fn{nullptr};
    EncodeTiled f = fn.load(std::memory_order_acquire);
    if (!f) {
        void *sym = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &sym, 12000, cudaEnableDefault, &found) !=
                cudaSuccess || found != cudaDriverEntryPointSuccess)
            return nullptr;
        f = reinterpret_cast<EncodeTiled>(sym);
        fn.store(f, std::memory_order_release);
    }
    return f;
}

// Byte tensor of up to 3 dimensions (x innermost, dense), boxes of 128 x ny (x 1), 128-byte swizzle.
inline bool encode_bytes(CUtensorMap *map, const void *base, uint64_t x, uint64_t y, uint64_t z, int ny) {
    const EncodeTiled f = encode_tiled();
    if (!f) return false;
    const int rank = z ? 3 : 2;
    const cuuint64_t dims[3] = {x, y, z};
    const cuuint64_t strides[2] = {x, x * y};
    const cuuint32_t box[3] = {128, (cuuint32_t)ny, 1}, elem[3] = {1, 1, 1};
    return f(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, const_cast<void *>(base), dims, strides, box, elem,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// bf16 matrix of y rows of x (dense), boxes of nx x ny, 64 or 128 bytes wide and swizzled as wide.
inline bool encode_bf16(CUtensorMap *map, void *base, uint64_t x, uint64_t y, int nx, int ny) {
    const EncodeTiled f = encode_tiled();
    if (!f) return false;
    const cuuint64_t dims[2] = {x, y}, strides[1] = {2 * x};
    const cuuint32_t box[2] = {(cuuint32_t)nx, (cuuint32_t)ny}, elem[2] = {1, 1};
    return f(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
             nx == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Raises the kernel's limit of shared memory, once per device (`ready`: those done).
inline cudaError_t raise_shared_limit(const void *kernel, int bytes, std::atomic<uint64_t> &ready) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (dev >= 64 || !(ready.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_release);
    }
    return cudaSuccess;
}

}  // namespace moe
