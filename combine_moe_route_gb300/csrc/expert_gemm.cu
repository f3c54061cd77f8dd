// expert_gemm.cu -- the experts' products over the rows a dispatch leaves
// grouped by expert, in e4m3 with fp32 scales per 128 channels of a row and
// per 128 x 128 block of a weight.
//
//   p[r, n] = sum_b a_scale[r, b] * w_scale[e, n/128, b] * sum_{c in b} a[r, c] * w[e, n, c]
//
// The scales are general fp32 values, so they cannot ride in the tensor
// cores' own block scaling (powers of two): the inner sum over a block of 128
// channels runs on the tensor cores into a fresh fp32 accumulator, and the
// outer sum adds that accumulator, times the two scales, to registers.
//
// A persistent block per SM walks output tiles of 128 rows of one expert x kBN
// columns.  Its warps have fixed jobs:
//   warp 8      loads the e4m3 tiles of both operands, 128 channels a stage,
//               with tiled bulk tensor copies into a ring of stages;
//   warp 9      issues the products of a stage (4 x K = 32) into one of the
//               tensor memory's accumulators, which alternate stage by stage;
//   warps 0-7   (two warpgroups) read a finished accumulator, one row per
//               thread and kBN / 2 columns per warpgroup, scale it into
//               registers, and after the last stage write the tile.
// A row tile is one load of 128 rows, or of 32 where it has no more: a block's
// loads take about 165 cycles each to issue, so a stage has as few of them as
// its operands allow.  Rows past a tile's own are the next expert's, or hold
// leftovers; nothing reads them (a row of the result depends on its own row of
// A alone).
//
// The forward weight [E, N, C] is a K-major operand.  The transposed product
// reads the same weight, [E, C, N] in its terms, as an MN-major operand, so
// no transposed copy is made.
//
// The gated form takes 128 columns of the gate and the 128 of the up
// projection as one tile of 256: each warpgroup holds 64 of both, forms
// silu(g) * u in fp32, and the two exchange their maxima of a row to quantise
// its block of 128.
#include <atomic>

#include "launch.h"
#include "numeric.cuh"
#include "tcgen05.cuh"

namespace moe {

constexpr int kProductThreads = 384;
// Registers of a thread of the loading and issuing warpgroup and of the two
// others, out of the 168 that a block of 384 threads starts with:
// 88 + 2 * 208 = 3 * 168.
constexpr int kIssueRegisters = 88, kSumRegisters = 208;
constexpr int kRowTile = 128;     // rows of a tile: the M of one product
constexpr int kFewRows = 32;      // rows of the small load of A
constexpr int kBlockK = 128;      // channels per stage: one scale block, 128 bytes
constexpr int kStageA = kRowTile * kBlockK;
constexpr int kTmemColumns = 512;
constexpr int kChunk = 16;                  // accumulator columns read at a time
constexpr int kStagingWarp = 16 * 128;      // output staging of a warp: 16 rows x 128 bytes

// Set when a bounded wait of a product kernel ran out (never in a sound run).
__device__ int32_t g_product_error;

struct ProductArgs {
    const float *a_scale, *w_scale;
    const int32_t *expert_offsets;
    int E, N, C;
    int rows;
    int ntiles;         // column tiles
    bool out_f32;
    void *out;          // plain form: [rows, N]
    unsigned char *q;   // gated form: [rows, N / 2]
    float *q_scale;
    __nv_bfloat16 *h;   // gated form: [rows, N] or null
};

// kCtas blocks work on one tile of kCtas * 128 rows x kBN columns.
template <int kCtas, int kBN>
struct ProductLayout {
    static constexpr int kStageBytes = kStageA + kBN / kCtas * kBlockK;
    static constexpr int kStages = 192 * 1024 / kStageBytes;
    static constexpr int kBuffers = kTmemColumns / kBN;
    static constexpr int kStaging = kStages * kStageBytes;
    static constexpr int kBytes = kStaging + 8 * kStagingWarp + 1024;   // + alignment of the swizzled tiles
};

// Columns of one load of the weight.  A block's share of a stage is one load,
// or two of 128: an MN-major row is 128 bytes (the swizzle's span), and the
// gate's and the up projection's columns lie apart.
template <int kCtas, int kBN, bool kTransposed, bool kGated>
constexpr int weight_box() {
    return (kTransposed || kGated) ? 128 : kBN / kCtas;
}

// Bytes that a row tile's load of A brings.
__device__ __forceinline__ uint32_t row_load_bytes(int valid) {
    return valid > kFewRows ? kRowTile * kBlockK : valid > 0 ? kFewRows * kBlockK : 0;
}

template <int kCtas, int kBN>
struct ProductShared {
    uint64_t full[ProductLayout<kCtas, kBN>::kStages], empty[ProductLayout<kCtas, kBN>::kStages];
    uint64_t acc_full[ProductLayout<kCtas, kBN>::kBuffers], acc_empty[ProductLayout<kCtas, kBN>::kBuffers];
    uint64_t pair[4];                      // gated: the two warps that share a quarter of the rows
    uint64_t drain;
    uint32_t tmem;
    volatile int32_t stop;                 // a wait ran out: every role leaves
    int32_t warp_tiles[kProductThreads / 32];
    int32_t tiles[MOE_MAX_EXPERTS + 1];    // row tiles before expert e
    float amax[2][2][kRowTile];            // gated: by tile parity, each warpgroup's maximum of a row's block
};

// Wait for a barrier's phase; false once any wait of the block has run out.
// The clock is read once per kPolls polls only: reading %globaltimer on every
// wait that did not succeed at once cost more than the rest of a stage.
constexpr uint32_t kPolls = 256;
template <class Shared>
__device__ __forceinline__ bool wait_or_stop(Shared &s, uint64_t *bar, uint32_t parity) {
    uint64_t t0 = 0;
    for (uint32_t i = 1; !mbar_try_wait(bar, parity); ++i) {
        if (i % kPolls != 0) continue;
        if (s.stop) return false;
        const uint64_t now = global_timer_ns();
        if (t0 == 0) t0 = now;
        if (now - t0 > kWaitLimitNs) {
            s.stop = 1;
            atomicOr(&g_product_error, MOE_DEVERR_COPY_TIMEOUT);
            return false;
        }
    }
    return true;
}

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

struct Tile {
    int e, row0, valid, n;   // expert, this block's first row and rows, column tile
    int pair_valid;          // rows of the blocks together
};

// Expert e's first row and number of rows, inside [0, rows] whatever the offsets hold.
__device__ __forceinline__ int2 expert_rows(const ProductArgs &p, int e) {
    const int lo = min(max(__ldg(p.expert_offsets + e), 0), p.rows);
    const int hi = min(max(__ldg(p.expert_offsets + e + 1), 0), p.rows);
    return make_int2(lo, max(hi - lo, 0));
}

// Tile t: experts in order; within an expert the row tiles of one column tile
// come first, so that blocks working at the same time share the weight.
template <int kCtas, class Shared>
__device__ __forceinline__ Tile tile_at(const Shared &s, const ProductArgs &p, long long t, int rank) {
    const int e = upper_bound_minus_one(s.tiles, p.E, (int)(t / p.ntiles));
    const int mt = s.tiles[e + 1] - s.tiles[e];
    const int i = (int)(t - (long long)s.tiles[e] * p.ntiles);
    const int m = i % mt;
    const int2 r = expert_rows(p, e);
    const int valid = min(r.y - m * (kCtas * kRowTile), kCtas * kRowTile);
    return {e, r.x + (m * kCtas + rank) * kRowTile, max(min(valid - rank * kRowTile, kRowTile), 0), i / mt, valid};
}

// Writes the 16-byte chunks a lane holds of its row (32 rows of a warp, kChunks
// each) to global memory in whole rows: 16 rows at a time through the warp's
// staging, swizzled against bank conflicts, then kChunks lanes per row.  `dst`
// is the address in the warp's row 0, rows lie `pitch` bytes apart; rows at or
// past nrows and bytes at or past `limit` are not written.
template <int kChunks>
__device__ __forceinline__ void store_rows(const uint4 (&v)[kChunks], unsigned char *stage, unsigned char *dst,
                                           size_t pitch, int nrows, int limit, int lane) {
    constexpr int kRows = 32 / kChunks;   // rows per store instruction
    const int c = lane % kChunks;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        __syncwarp();
        if ((lane >> 4) == half) {
#pragma unroll
            for (int k = 0; k < kChunks; ++k)
                *reinterpret_cast<uint4 *>(stage + (lane & 15) * 128 + ((k ^ (lane & 7)) * 16)) = v[k];
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 16 / kRows; ++i) {
            const int r = i * kRows + lane / kChunks;
            const uint4 x = *reinterpret_cast<const uint4 *>(stage + r * 128 + ((c ^ (r & 7)) * 16));
            if (half * 16 + r < nrows && c * 16 < limit) st_v4(dst + (size_t)(half * 16 + r) * pitch + c * 16, x);
        }
    }
}

// 64 fp32 values of a row, as bf16.
__device__ __forceinline__ void store_bf16x64(const float2 *acc, unsigned char *stage, unsigned char *dst, size_t pitch,
                                              int nrows, int limit, int lane) {
    uint4 v[8];
#pragma unroll
    for (int c = 0; c < 8; ++c)
        v[c] = make_uint4(bf16_pair(acc[4 * c].x, acc[4 * c].y), bf16_pair(acc[4 * c + 1].x, acc[4 * c + 1].y),
                          bf16_pair(acc[4 * c + 2].x, acc[4 * c + 2].y), bf16_pair(acc[4 * c + 3].x, acc[4 * c + 3].y));
    store_rows<8>(v, stage, dst, pitch, nrows, limit, lane);
}

// Columns of a product at the right edge, where `left` are left.  Both blocks of
// a pair bring half of them, and half a tile's columns have to be a multiple of 16
// for the loads of an MN-major weight (columns past N read as zeros).
template <int kCtas, int kBN>
__device__ __forceinline__ int tile_columns(int left) {
    const int cols = min(kBN, left);
    return kCtas == 2 ? (cols + 31) & ~31 : cols;
}

// The accumulator column of a warpgroup's i-th column.
template <int kCols, bool kGated>
__device__ __forceinline__ int chunk_column(int wg, int i) {
    return kGated ? (i < 64 ? wg * 64 + i : 128 + wg * 64 + (i - 64)) : wg * kCols + i;
}

template <int kCtas, int kBN, bool kTransposed, bool kGated>
__global__ void __launch_bounds__(kProductThreads, 1)
    expert_product_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_few,
                          const __grid_constant__ CUtensorMap map_w, const ProductArgs p) {
    using Layout = ProductLayout<kCtas, kBN>;
    extern __shared__ unsigned char s_raw[];
    __shared__ ProductShared<kCtas, kBN> s;
    unsigned char *tiles = s_raw + ((1024u - (smem_u32(s_raw) & 1023u)) & 1023u);   // swizzled tiles: 1024-byte aligned
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = kCtas == 2 ? (int)cluster_rank() : 0;
    const int nkb = (p.C + kBlockK - 1) / kBlockK;

    // prologue: barriers, tensor memory, and the experts' row tiles
    if (threadIdx.x == 0) {
        for (int i = 0; i < Layout::kStages; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < Layout::kBuffers; ++i) {
            mbar_init(&s.acc_full[i], 1);
            mbar_init(&s.acc_empty[i], 8 * kCtas);
        }
        for (int i = 0; i < 4; ++i) mbar_init(&s.pair[i], 2);
        mbar_init(&s.drain, 1);
        s.stop = 0;
        fence_mbarrier_init();
        prefetch_tensor_map(&map_a);
        prefetch_tensor_map(&map_few);
        prefetch_tensor_map(&map_w);
    }
    if (warp == 9) tmem_alloc<kCtas, kTmemColumns>(&s.tmem);
    {
        constexpr int kPer = (MOE_MAX_EXPERTS + kProductThreads - 1) / kProductThreads;
        int mine = 0, mt[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = threadIdx.x * kPer + i;
            mt[i] = 0;
            if (e < p.E) mt[i] = (expert_rows(p, e).y + kCtas * kRowTile - 1) / (kCtas * kRowTile);
            mine += mt[i];
        }
        int sum = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, sum, off);
            if (lane >= off) sum += v;
        }
        if (lane == 31) s.warp_tiles[warp] = sum;
        __syncthreads();
        // 64 bits and a cap: offsets that overlap may not make the prefix wrap
        long long before = sum - mine;
        for (int w = 0; w < warp; ++w) before += s.warp_tiles[w];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = threadIdx.x * kPer + i;
            if (e < p.E) s.tiles[e] = (int)min(before, 1ll << 30);
            before += mt[i];
            if (e == p.E - 1) s.tiles[p.E] = (int)min(before, 1ll << 30);
        }
    }
    tcgen05_fence_before();
    if (kCtas == 2) cluster_barrier();   // the pair's barriers are ready
    else __syncthreads();
    tcgen05_fence_after();
    const long long total = (long long)s.tiles[p.E] * p.ntiles;
    const uint32_t tmem = s.tmem;

    if (warp >= 8) {
        registers_decrease<kIssueRegisters>();
        if (warp == 8 && lane == 0) {
            // ---------------------------------------------------- loads
            Ring r;
            long long issued = 0;
            bool go = true;
            for (long long t = blockIdx.x / kCtas; go && t < total; t += gridDim.x / kCtas) {
                const Tile tile = tile_at<kCtas>(s, p, t, rank);
                const int n0 = tile.n * (kGated ? kBN / 2 : kBN);
                const int cols = kGated ? kBN : tile_columns<kCtas, kBN>(p.N - n0);
                // a pair splits the columns: each block brings half of them
                constexpr int kBox = weight_box<kCtas, kBN, kTransposed, kGated>(), kBoxBytes = kBox * kBlockK;
                const int boxes = kCtas == 2 ? 1 : kGated ? 2 : (cols + kBox - 1) / kBox;
                const int first = kGated ? n0 + rank * (p.N / 2) : n0 + rank * (cols / 2);
                const CUtensorMap *rows = tile.valid > kFewRows ? &map_a : &map_few;
                const uint32_t bytes =
                    kCtas * boxes * kBoxBytes +
                    (kCtas == 2 ? row_load_bytes(min(tile.pair_valid, kRowTile)) +
                                      row_load_bytes(tile.pair_valid - kRowTile)
                                : row_load_bytes(tile.valid));
                for (int kb = 0; kb < nkb; ++kb) {
                    if (!(go = wait_or_stop(s, &s.empty[r.slot], r.parity ^ 1u))) break;
                    unsigned char *a = tiles + r.slot * Layout::kStageBytes, *w = a + kStageA;
                    uint64_t *bar = &s.full[r.slot];
                    if (rank == 0) mbar_arrive_expect_tx(bar, bytes);
                    if (tile.valid > 0) tensor_load_2d<kCtas>(a, rows, kb * kBlockK, tile.row0, bar);
                    for (int i = 0; i < boxes; ++i) {
                        const int n = first + i * (kGated ? p.N / 2 : kBox);
                        if (kTransposed)
                            tensor_load_3d<kCtas>(w + i * kBoxBytes, &map_w, n, kb * kBlockK, tile.e, bar);
                        else tensor_load_3d<kCtas>(w + i * kBoxBytes, &map_w, kb * kBlockK, n, tile.e, bar);
                    }
                    r.advance(Layout::kStages);
                    ++issued;
                }
            }
            // nothing in flight when the block ends: the products have read every stage, or (after
            // a wait ran out) at least its loads have landed
            const int last = (int)(issued < Layout::kStages ? issued : Layout::kStages);
            for (int i = 0; i < last; ++i) {
                r.slot = (r.slot == 0 ? Layout::kStages : r.slot) - 1;
                if (r.slot == Layout::kStages - 1) r.parity ^= 1u;
                if (!wait_or_stop(s, &s.empty[r.slot], r.parity) && rank == 0)
                    mbar_wait_bounded(&s.full[r.slot], r.parity);   // a pair's barrier counts both blocks' loads
            }
        } else if (warp == 9 && lane == 0 && rank == 0) {
            // ------------------------------------------------- products
            Ring r, b;
            bool go = true;
            for (long long t = blockIdx.x / kCtas; go && t < total; t += gridDim.x / kCtas) {
                const Tile tile = tile_at<kCtas>(s, p, t, rank);
                const int cols = kGated ? kBN : tile_columns<kCtas, kBN>(p.N - tile.n * kBN);
                const uint32_t instruction = f8_instruction(kCtas * kRowTile, cols, kTransposed);
                for (int kb = 0; kb < nkb; ++kb) {
                    if (!(go = wait_or_stop(s, &s.acc_empty[b.slot], b.parity ^ 1u))) break;
                    if (!(go = wait_or_stop(s, &s.full[r.slot], r.parity))) break;
                    tcgen05_fence_after();
                    const uint32_t a = smem_u32(tiles) + r.slot * Layout::kStageBytes, w = a + kStageA;
#pragma unroll
                    for (int k = 0; k < kBlockK / 32; ++k) {
                        // 32 channels on: 32 bytes along a K-major row, 32 rows of 128 bytes MN-major
                        const uint64_t da = smem_descriptor(a + k * 32, 16, 1024);
                        const uint64_t dw = kTransposed ? smem_descriptor(w + k * 32 * 128, 128 * kBlockK, 1024)
                                                        : smem_descriptor(w + k * 32, 16, 1024);
                        mma_f8<kCtas>(tmem + b.slot * kBN, da, dw, instruction, k > 0);
                    }
                    mma_commit<kCtas>(&s.empty[r.slot]);
                    mma_commit<kCtas>(&s.acc_full[b.slot]);
                    r.advance(Layout::kStages);
                    b.advance(Layout::kBuffers);
                }
            }
            if (!go) {   // leave no product running
                mma_commit<kCtas>(&s.drain);
                mbar_wait_bounded(&s.drain, 0);
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------- scaled sums and the output
        registers_increase<kSumRegisters>();
        constexpr int kCols = kBN / 2;            // columns of a warpgroup
        const int wg = warp >> 2, quarter = warp & 3;
        unsigned char *stage = tiles + Layout::kStaging + warp * kStagingWarp;
        const int nb = (p.N + 127) / 128;         // scale blocks along the columns
        const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
        Ring b;
        uint32_t pair_parity = 0;
        bool go = true;
        for (long long t = blockIdx.x / kCtas; go && t < total; t += gridDim.x / kCtas) {
            const Tile tile = tile_at<kCtas>(s, p, t, rank);
            const int nrows = min(tile.valid - quarter * 32, 32);   // rows of this warp
            const int n0 = kGated ? tile.n * 128 : tile.n * kBN + wg * kCols;
            const bool active = nrows > 0 && (kGated || n0 < p.N);
            const size_t row = (size_t)tile.row0 + quarter * 32 + min(lane, max(nrows, 1) - 1);
            const float *sa = p.a_scale + (active ? row : 0) * nkb;
            // the weight scales of block b: sw[b * step] (and su for the up projection's block)
            const size_t step = kTransposed ? nb : 1;
            const int cblock = active ? n0 / 128 : 0;
            const float *sw = p.w_scale + (kTransposed ? (size_t)tile.e * nkb * nb + cblock
                                                       : ((size_t)tile.e * nb + cblock) * nkb);
            const float *su = kGated ? sw + (size_t)(nb / 2) * nkb : nullptr;

            float2 acc[kCols / 2];
#pragma unroll
            for (int i = 0; i < kCols / 2; ++i) acc[i] = make_float2(0.0f, 0.0f);
            // scales are fetched a group of four blocks ahead
            float fa[4], fw[4], fu[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                fa[i] = i < nkb ? __ldg(sa + i) : 0.0f;
                fw[i] = i < nkb ? __ldg(sw + i * step) : 0.0f;
                if (kGated) fu[i] = i < nkb ? __ldg(su + i) : 0.0f;
            }
            for (int kb0 = 0; go && kb0 < nkb; kb0 += 4) {
                float f[4], g[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f[i] = fa[i] * fw[i];
                    if (kGated) g[i] = fa[i] * fu[i];
                    const int kb = kb0 + 4 + i;
                    if (kb < nkb) {
                        fa[i] = __ldg(sa + kb);
                        fw[i] = __ldg(sw + kb * step);
                        if (kGated) fu[i] = __ldg(su + kb);
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (kb0 + i >= nkb) break;
                    go = __all_sync(0xffffffffu, wait_or_stop(s, &s.acc_full[b.slot], b.parity));
                    if (!go) break;
                    tcgen05_fence_after();
                    if (active) {
                        // the next columns are on their way while these are added
                        uint32_t v[2][kChunk];
                        const uint32_t at = lanes + b.slot * kBN;
                        tmem_load(at + chunk_column<kCols, kGated>(wg, 0), v[0]);
#pragma unroll
                        for (int c = 0; c < kCols / kChunk; ++c) {
                            tmem_wait_load();
                            if (c + 1 < kCols / kChunk)
                                tmem_load(at + chunk_column<kCols, kGated>(wg, (c + 1) * kChunk), v[(c + 1) & 1]);
                            const float fc = (kGated && c * kChunk >= 64) ? g[i] : f[i];
#pragma unroll
                            for (int k = 0; k < kChunk / 2; ++k)
                                fma_pair(acc[c * (kChunk / 2) + k], make_float2(fc, fc),
                                         make_float2(__uint_as_float(v[c & 1][2 * k]),
                                                     __uint_as_float(v[c & 1][2 * k + 1])));
                        }
                    }
                    tcgen05_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (kCtas == 2) mbar_arrive_first(&s.acc_empty[b.slot]);
                        else mbar_arrive(&s.acc_empty[b.slot]);
                    }
                    b.advance(Layout::kBuffers);
                }
            }
            if (!go) break;
            const size_t warp_row = (size_t)tile.row0 + quarter * 32;
            if constexpr (kGated) {
                const int I = p.N / 2, i0 = n0 + wg * 64;
                if (p.h && active) {
                    unsigned char *h = reinterpret_cast<unsigned char *>(p.h + warp_row * p.N + i0);
                    store_bf16x64(acc, stage, h, (size_t)p.N * 2, nrows, 128, lane);
                    store_bf16x64(acc + 32, stage, h + (size_t)I * 2, (size_t)p.N * 2, nrows, 128, lane);
                }
                float amax = 0.0f;
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    acc[k].x = acc[k].x * sigmoid(acc[k].x) * acc[32 + k].x;
                    acc[k].y = acc[k].y * sigmoid(acc[k].y) * acc[32 + k].y;
                    amax = fmaxf(amax, fmaxf(fabsf(acc[k].x), fabsf(acc[k].y)));
                }
                // the two warps that hold a row swap their maxima; a warp writes a parity's slot
                // again only after the other has arrived for the tile in between, so after its read
                s.amax[pair_parity][wg][quarter * 32 + lane] = amax;
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.pair[quarter]);
                go = __all_sync(0xffffffffu, wait_or_stop(s, &s.pair[quarter], pair_parity));
                if (!go) break;
                amax = quant_amax(fmaxf(amax, s.amax[pair_parity][wg ^ 1][quarter * 32 + lane]));
                pair_parity ^= 1u;
                if (active) {
                    const float inv = quant_inverse(amax);
                    uint4 v[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t w[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float2 v0 = acc[c * 8 + 2 * k], v1 = acc[c * 8 + 2 * k + 1];
                            w[k] = pack_e4m3x4(__fmul_rn(v0.x, inv), __fmul_rn(v0.y, inv), __fmul_rn(v1.x, inv),
                                               __fmul_rn(v1.y, inv));
                        }
                        v[c] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    store_rows<4>(v, stage, p.q + warp_row * I + i0, I, nrows, 64, lane);
                    if (wg == 0 && lane < nrows)
                        p.q_scale[(warp_row + lane) * (I / 128) + tile.n] = quant_scale(amax);
                }
            } else if (active) {
                if (p.out_f32) {
#pragma unroll
                    for (int c = 0; c < kCols / 32; ++c) {
                        uint4 v[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const float2 v0 = acc[c * 16 + 2 * k], v1 = acc[c * 16 + 2 * k + 1];
                            v[k] = make_uint4(__float_as_uint(v0.x), __float_as_uint(v0.y), __float_as_uint(v1.x),
                                              __float_as_uint(v1.y));
                        }
                        const int n = n0 + c * 32;
                        if (n < p.N)
                            store_rows<8>(v, stage, static_cast<unsigned char *>(p.out) + (warp_row * p.N + n) * 4,
                                          (size_t)p.N * 4, nrows, (p.N - n) * 4, lane);
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < kCols / 64; ++c) {
                        const int n = n0 + c * 64;
                        if (n < p.N)
                            store_bf16x64(acc + c * 32, stage,
                                          static_cast<unsigned char *>(p.out) + (warp_row * p.N + n) * 2,
                                          (size_t)p.N * 2, nrows, (p.N - n) * 2, lane);
                    }
                }
            }
        }
    }
    tcgen05_fence_before();
    if (kCtas == 2) cluster_barrier();   // nothing of the other block's reaches this one any more
    else __syncthreads();
    tcgen05_fence_after();
    if (warp == 9) tmem_free<kCtas, kTmemColumns>(tmem);
}

// ------------------------------------------------------------------- host

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeTiled encode_tiled() {
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
static bool encode_bytes(CUtensorMap *map, const void *base, uint64_t x, uint64_t y, uint64_t z, int ny) {
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

template <int kCtas, int kBN, bool kTransposed, bool kGated>
static cudaError_t launch_tiles(const void *a, const void *w, ProductArgs p, cudaStream_t stream) {
    CUtensorMap map_a, map_few, map_w;
    if (!encode_bytes(&map_a, a, p.C, p.rows, 0, kRowTile) || !encode_bytes(&map_few, a, p.C, p.rows, 0, kFewRows) ||
        !encode_bytes(&map_w, w, kTransposed ? p.N : p.C, kTransposed ? p.C : p.N, p.E,
                      kTransposed ? kBlockK : weight_box<kCtas, kBN, kTransposed, kGated>()))
        return cudaErrorInvalidValue;
    auto kernel = expert_product_kernel<kCtas, kBN, kTransposed, kGated>;
    constexpr int smem = ProductLayout<kCtas, kBN>::kBytes;
    static std::atomic<uint64_t> ready{0};   // devices whose limit is raised
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (dev >= 64 || !(ready.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_release);
    }
    const int cols = kGated ? kBN / 2 : kBN;
    p.ntiles = ((kGated ? p.N / 2 : p.N) + cols - 1) / cols;
    // no more tiles than this exist; the blocks walk them
    const long long most = ((long long)p.rows / (kCtas * kRowTile) + (p.rows < p.E ? p.rows : p.E)) * p.ntiles;
    const int groups = device_sm_count() / kCtas;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(kCtas * (most < groups ? (most > 0 ? most : 1) : groups)));
    cfg.blockDim = dim3(kProductThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kCtas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, map_a, map_few, map_w, p);
}

template <bool kTransposed, bool kGated>
static cudaError_t launch_product(const void *a, const void *w, const ProductArgs &p, cudaStream_t stream) {
    const bool pairs = p.rows >= (long long)p.E * 192;
    if (pairs) return launch_tiles<2, 256, kTransposed, kGated>(a, w, p, stream);
    if constexpr (kGated) return launch_tiles<1, 256, kTransposed, kGated>(a, w, p, stream);
    else return launch_tiles<1, 128, kTransposed, kGated>(a, w, p, stream);
}

cudaError_t launch_expert_gemm(const void *a, const float *a_scale, const void *w, const float *w_scale,
                               const int32_t *expert_offsets, int E, int N, int C, long long rows, bool transpose,
                               bool out_f32, void *out, cudaStream_t stream) {
    ProductArgs p = {};
    p.a_scale = a_scale, p.w_scale = w_scale, p.expert_offsets = expert_offsets;
    p.E = E, p.N = N, p.C = C, p.rows = (int)rows;
    p.out_f32 = out_f32, p.out = out;
    return transpose ? launch_product<true, false>(a, w, p, stream) : launch_product<false, false>(a, w, p, stream);
}

cudaError_t launch_expert_gated_gemm(const void *a, const float *a_scale, const void *w, const float *w_scale,
                                     const int32_t *expert_offsets, int E, int I, int C, long long rows, void *q,
                                     float *q_scale, void *h, cudaStream_t stream) {
    ProductArgs p = {};
    p.a_scale = a_scale, p.w_scale = w_scale, p.expert_offsets = expert_offsets;
    p.E = E, p.N = 2 * I, p.C = C, p.rows = (int)rows;
    p.q = static_cast<unsigned char *>(q), p.q_scale = q_scale, p.h = static_cast<__nv_bfloat16 *>(h);
    return launch_product<false, true>(a, w, p, stream);
}

cudaError_t read_product_error(int32_t *host_code, cudaStream_t stream) {
    int32_t v = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_product_error, sizeof(v), 0, cudaMemcpyDeviceToHost, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (e != cudaSuccess) return e;
    *host_code = v;
    if (v) {
        const int32_t zero = 0;
        e = cudaMemcpyToSymbolAsync(g_product_error, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, stream);
        if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    }
    return e;
}

}  // namespace moe
