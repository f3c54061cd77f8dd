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
// columns; for experts of many rows a pair of blocks walks tiles of 256 rows,
// each holding half of the rows and loading half of the weight's columns (32 KB
// a stage and block instead of 48).  The warps of a block have fixed jobs:
//   warp 8      loads the e4m3 tiles of both operands, 128 channels a stage,
//               with tiled bulk tensor copies into a ring of stages;
//   warps 9, 10 take turns at issuing the products of a stage (4 x K = 32) into
//               the tensor memory's accumulators, which alternate (two of 256
//               columns, four of 128);
//   warp 11     forms the products of the two scales, one per row, channel block
//               and 128 columns, some blocks ahead, in a ring of its own (reading
//               them where they are used stalled the sums on L2), and tells the
//               sums where their tile is;
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
//
// Where the tiles are too few to occupy the card, the blocks of a cluster share
// a tile's channels (split_parts) and add up through each other's shared memory.
//
// What bounds it: few rows, the weight's bytes (256 experts x 32 rows, 7168 x
// 2048: 3.9 GB in 567 us, 0.99 of the measured copy rate).  Many rows, a stage
// takes about 650 cycles of which its products are 512 (the sums alone would take
// about 600), and a tile's output about 3000 more, which nothing overlaps: the
// tensor cores are active 75 % of the cycles over 7168 channels (8 experts x 1024
// rows, 4096 x 7168, in 157 us, 3.1 PFLOP/s) and 58 % over 2048 (7168 x 2048, 95 us,
// 2.5 PFLOP/s).  64 such experts of 7168 channels, for seconds, run at the card's
// power limit: 2.7 to 2.8 PFLOP/s with the SM clock at 1.5 GHz.
#include <pthread.h>

#include <atomic>

#include "launch.h"
#include "product.cuh"

namespace moe {

// Registers of a thread of the loading and issuing warpgroup and of the two
// others, out of the 168 that a block of 384 threads starts with:
// 40 + 2 * 232 = 3 * 168.
constexpr int kIssueRegisters = 40, kSumRegisters = 232;
constexpr int kBlockK = 128;      // channels per stage: one scale block, 128 bytes
constexpr int kStageA = kRowTile * kBlockK;
constexpr int kScaleSlots = 4;             // of the ring of scales

// Set when a bounded wait of a product kernel ran out (never in a sound run), and
// what the last read took out of it.
__device__ int32_t g_product_error, g_product_error_taken;

struct ProductArgs {
    const float *a_scale, *w_scale;
    const int32_t *expert_offsets;
    int E, N, C;
    int rows;
    int ntiles;         // column tiles
    int split;          // blocks that share a tile's channels (split launches)
    bool tails;         // single blocks: only what the pairs' launch before leaves (see below)
    bool out_f32;
    void *out;          // plain form: [rows, N]
    unsigned char *q;   // gated form: [rows, N / 2]
    float *q_scale;
    __nv_bfloat16 *h;   // gated form: [rows, N] or null
};

// kCtas blocks work on one tile of kCtas * 128 rows x kBN columns; every stage's
// product goes to the next of kGroup accumulators.
template <int kCtas, int kBN>
struct ProductLayout {
    static constexpr int kStageBytes = kStageA + kBN / kCtas * kBlockK;
    static constexpr int kStages = 192 * 1024 / kStageBytes;
    static constexpr int kGroup = kTmemColumns / kBN;
    static constexpr int kHalves = kBN / 128;   // 64-column groups of a warpgroup
    static constexpr int kStaging = kStages * kStageBytes;
    static constexpr int kBytes = kStaging + 8 * kStagingWarp + 1024;   // + alignment of the swizzled tiles
};

// Columns of one load of the weight.  A block's share of a stage is one load,
// or two: an MN-major row is 128 bytes (the swizzle's span), and the gate's and
// the up projection's columns lie apart.
template <int kCtas, int kBN, bool kTransposed, bool kGated>
constexpr int weight_box() {
    return (kTransposed || kGated) ? 128 : kBN / kCtas;
}

template <int kCtas, int kBN>
struct ProductShared {
    uint64_t full[ProductLayout<kCtas, kBN>::kStages], empty[ProductLayout<kCtas, kBN>::kStages];
    uint64_t acc_full[ProductLayout<kCtas, kBN>::kGroup], acc_empty[ProductLayout<kCtas, kBN>::kGroup];
    uint64_t pair[4];                      // gated: the two warps that share a quarter of the rows
    uint64_t scale_full[kScaleSlots], scale_empty[kScaleSlots];
    uint64_t drain[2];
    uint32_t tmem;
    int32_t warp_tiles[kProductThreads / 32];
    int32_t tiles[MOE_MAX_EXPERTS + 1];    // row tiles before expert e
    float scales[kScaleSlots][4][kRowTile];   // a_scale * w_scale: a group's stages, kHalves each
    int4 tile[kScaleSlots];                // of the group in a slot: first row, rows, first column
    float amax[2][2][kRowTile];            // gated: by tile parity, each warpgroup's maximum of a row's block
};

struct Tile {
    int e, row0, valid, n;   // expert, this block's first row and rows, column tile
    int pair_valid;          // rows of the blocks together
};

// Row tiles of an expert with n rows.  Pairs take its whole 256 rows and a rest
// of more than 128; a rest of up to 128 rows, half of a pair's tile, is a tile
// of the single blocks' launch that follows (`tails`).  Without pairs single
// blocks take every 128 rows.
template <int kCtas>
__device__ __forceinline__ int row_tiles(const ProductArgs &p, int n) {
    constexpr int kPair = 2 * kRowTile;
    if (kCtas == 2) return n / kPair + (n % kPair > kRowTile);
    if (p.tails) return n % kPair > 0 && n % kPair <= kRowTile;
    return (n + kRowTile - 1) / kRowTile;
}

// Tile t: experts in order; within an expert the row tiles of one column tile
// come first, so that blocks working at the same time share the weight.
template <int kCtas, class Shared>
__device__ __forceinline__ Tile tile_at(const Shared &s, const ProductArgs &p, long long t, int rank) {
    const int e = upper_bound_minus_one(s.tiles, p.E, (int)(t / p.ntiles));
    const int mt = s.tiles[e + 1] - s.tiles[e];
    const int i = (int)(t - (long long)s.tiles[e] * p.ntiles);
    const int2 r = expert_rows(p, e);
    const int m = kCtas == 1 && p.tails ? r.y / (2 * kRowTile) * 2 : i % mt * kCtas;   // in units of 128 rows
    const int valid = min(r.y - m * kRowTile, kCtas * kRowTile);
    return {e, r.x + (m + rank) * kRowTile, max(min(valid - rank * kRowTile, kRowTile), 0), i / mt, valid};
}

// kSplit: the blocks of a cluster share one tile, each taking a run of its
// channels, and then add up: a row's sums go to the block that owns the row,
// through the shared memory of its ring, which is free by then.
template <int kCtas, int kBN, bool kTransposed, bool kGated, bool kSplit>
__global__ void __launch_bounds__(kProductThreads, 1)
    expert_product_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_few,
                          const __grid_constant__ CUtensorMap map_w, const ProductArgs p) {
    using Layout = ProductLayout<kCtas, kBN>;
    extern __shared__ unsigned char s_raw[];
    __shared__ ProductShared<kCtas, kBN> s;
    unsigned char *tiles = s_raw + ((1024u - (smem_u32(s_raw) & 1023u)) & 1023u);   // swizzled tiles: 1024-byte aligned
    // broadcast, so that the compiler knows it to be the same in a warp
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const bool issue = lane == 0;
    const int rank = kCtas == 2 ? (int)cluster_rank() : 0;
    const int nkb = (p.C + kBlockK - 1) / kBlockK;
    const int parts = kSplit ? p.split : 1, part = kSplit ? (int)cluster_rank() : 0;
    const int kb_first = kSplit ? nkb * part / parts : 0;                     // this block's channels
    const int nk = kSplit ? nkb * (part + 1) / parts - kb_first : nkb;

    // prologue: barriers, tensor memory, and the experts' row tiles
    if (threadIdx.x == 0) {
        for (int i = 0; i < Layout::kStages; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < Layout::kGroup; ++i) {
            mbar_init(&s.acc_full[i], 1);
            mbar_init(&s.acc_empty[i], 8 * kCtas);
        }
        for (int i = 0; i < 4; ++i) mbar_init(&s.pair[i], 2);
        for (int i = 0; i < kScaleSlots; ++i) {
            mbar_init(&s.scale_full[i], 1);
            mbar_init(&s.scale_empty[i], 8);
        }
        mbar_init(&s.drain[0], 1);
        mbar_init(&s.drain[1], 1);
        fence_mbarrier_init();
        prefetch_tensor_map(&map_a);
        prefetch_tensor_map(&map_few);
        prefetch_tensor_map(&map_w);
    }
    if (warp == 9) tmem_alloc<kCtas, kTmemColumns>(&s.tmem);
    // Up to here nothing is read: this block may have started while the kernel before ran out, and
    // lets the kernel after do the same.  Only this wait makes what earlier kernels wrote visible,
    // so it stands before the first read in the tails' launch as well, although what that reads
    // was written before the pairs' launch: that the pairs waited for it orders their own reads,
    // not those of a grid that starts beside them.
    pdl_launch_dependents();
    pdl_wait();
    {
        constexpr int kPer = (MOE_MAX_EXPERTS + kProductThreads - 1) / kProductThreads;
        int mine = 0, mt[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = threadIdx.x * kPer + i;
            mt[i] = 0;
            if (e < p.E) mt[i] = row_tiles<kCtas>(p, expert_rows(p, e).y);
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

    // Every wait below has a limit and runs out on its own if its partner has left; a role whose
    // wait ran out leaves its loop.  `go` is looked at after the work that a wait released is
    // issued: that work is harmless on stale data, and the look is then off the critical path.
    const auto at = [](const uint64_t *bar) { return smem_u32(bar); };
    const uint32_t tiles_at = smem_u32(tiles);
    bool go = true;
    if (warp >= 8) {
        registers_decrease<kIssueRegisters>();
        if (warp == 8) {
            // ---------------------------------------------------- loads
            Ring r;
            long long issued = 0;
            for (long long t = blockIdx.x / (kCtas * parts); go && t < total; t += kSplit ? total : gridDim.x / kCtas) {
                const Tile tile = tile_at<kCtas>(s, p, t, rank);
                const int n0 = tile.n * (kGated ? kBN / 2 : kBN);
                // a pair splits the columns: each block brings half of them
                constexpr int kBox = weight_box<kCtas, kBN, kTransposed, kGated>(), kBoxBytes = kBox * kBlockK;
                constexpr int kBoxes = kBN / kCtas / kBox;
                const int first = n0 + rank * (kGated ? p.N / 2 : 128);
                const CUtensorMap *rows = tile.valid > kFewRows ? &map_a : &map_few;
                const uint32_t bytes =
                    kCtas * kBoxes * kBoxBytes +
                    (kCtas == 2 ? row_load_bytes(min(tile.pair_valid, kRowTile)) +
                                      row_load_bytes(tile.pair_valid - kRowTile)
                                : row_load_bytes(tile.valid));
                for (int kb = kb_first; kb < kb_first + nk; ++kb) {
                    go = __all_sync(0xffffffffu, mbar_wait_polls(at(&s.empty[r.slot]), r.parity ^ 1u));
                    if (!go) break;
                    const uint32_t a = tiles_at + r.slot * Layout::kStageBytes, w = a + kStageA;
                    const uint32_t bar = at(&s.full[r.slot]);
#ifdef MOE_TEST_WITHHOLD_PRODUCT_STAGE
                    // Test builds only: the loads of this stage never happen, so the waits run out.
                    const bool load = issue && issued != MOE_TEST_WITHHOLD_PRODUCT_STAGE;
#else
                    const bool load = issue;
#endif
                    mbar_expect(bar, bytes, load && rank == 0);
                    tensor_load_2d<kCtas>(a, rows, kb * kBlockK, tile.row0, bar, load && tile.valid > 0);
#pragma unroll
                    for (int i = 0; i < kBoxes; ++i) {
                        const int n = first + i * (kGated ? p.N / 2 : kBox);
                        if (kTransposed)
                            tensor_load_3d<kCtas>(w + i * kBoxBytes, &map_w, n, kb * kBlockK, tile.e, bar, load);
                        else tensor_load_3d<kCtas>(w + i * kBoxBytes, &map_w, kb * kBlockK, n, tile.e, bar, load);
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
                go = go && __all_sync(0xffffffffu, mbar_wait_polls(at(&s.empty[r.slot]), r.parity));
                if (!go && rank == 0)   // a pair's barrier counts both blocks' loads
                    mbar_wait_polls(at(&s.full[r.slot]), r.parity);
            }
        } else if (warp < 11) {
            // ------------------------------------------------- products
            // two warps take turns: a thread issues about as fast as its products run, so one
            // alone would leave the tensor cores idle while it waits on barriers
            if (rank == 0) {
                const int turn = warp - 9;
                constexpr uint32_t instruction = f8_instruction(kCtas * kRowTile, kBN, kTransposed);
                // 32 channels on: 32 bytes along a K-major row, 32 rows of 128 bytes MN-major
                constexpr int kStepW = (kTransposed ? 32 * 128 : 32) >> 4, kStepA = 32 >> 4;
                const uint64_t a0 = smem_descriptor(tiles_at, 16, 1024);
                const uint64_t w0 = smem_descriptor(tiles_at + kStageA, kTransposed ? 128 * kBlockK : 16, 1024);
                Ring r;
                uint32_t parities = 0;   // of the accumulators' passes
                for (long long t = blockIdx.x / (kCtas * parts); go && t < total; t += kSplit ? total : gridDim.x / kCtas) {
                    for (int kb = 0; kb < nk; ++kb) {
                        if ((kb & 1) == turn) {
                            const int slot = kb % Layout::kGroup;
                            const bool free_now =
                                mbar_wait_polls(at(&s.acc_empty[slot]), ((parities >> slot) & 1u) ^ 1u);
                            const bool full_now = mbar_wait_polls(at(&s.full[r.slot]), r.parity);
                            tcgen05_fence_after();
                            const uint64_t da = a0 + (uint32_t)r.slot * (Layout::kStageBytes >> 4);
                            const uint64_t dw = w0 + (uint32_t)r.slot * (Layout::kStageBytes >> 4);
#pragma unroll
                            for (int k = 0; k < kBlockK / 32; ++k)
                                mma_f8<kCtas>(tmem + slot * kBN, da + k * kStepA, dw + k * kStepW, instruction, k > 0,
                                              issue);
                            mma_commit<kCtas>(at(&s.acc_full[slot]), issue);
                            mma_commit<kCtas>(at(&s.empty[r.slot]), issue);
                            parities ^= 1u << slot;
                            go = __all_sync(0xffffffffu, free_now && full_now);
                            if (!go) break;
                        }
                        r.advance(Layout::kStages);
                    }
                }
                if (!go) {   // leave no product running
                    mma_commit<kCtas>(at(&s.drain[turn]), issue);
                    mbar_wait_polls(at(&s.drain[turn]), 0);
                }
            }
        } else if (warp == 11) {
            // --------------------------------------------------- scales
            const int nb = (p.N + 127) / 128;           // scale blocks along the columns
            const size_t step = kTransposed ? nb : 1;   // from one block of channels to the next
            Ring c;
            for (long long t = blockIdx.x / (kCtas * parts); go && t < total; t += kSplit ? total : gridDim.x / kCtas) {
                const Tile tile = tile_at<kCtas>(s, p, t, rank);
                const float *sw[Layout::kHalves];
#pragma unroll
                for (int h = 0; h < Layout::kHalves; ++h) {
                    // h: the gate's and the up projection's block, or the warpgroup's
                    const int block = kGated ? h * (nb / 2) + tile.n : min(tile.n * Layout::kHalves + h, nb - 1);
                    sw[h] = p.w_scale + (size_t)tile.e * nkb * nb + (kTransposed ? (size_t)block : (size_t)block * nkb);
                }
                for (int kb0 = 0; kb0 < nk; kb0 += Layout::kGroup) {
                    float fa[4][Layout::kGroup], fw[Layout::kHalves][Layout::kGroup];
#pragma unroll
                    for (int i = 0; i < Layout::kGroup; ++i) {
                        const int kb = kb_first + min(kb0 + i, nk - 1);
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const int r = q * 32 + lane;
                            fa[q][i] = r < tile.valid ? ld_chained(p.a_scale + ((size_t)tile.row0 + r) * nkb + kb) : 0.0f;
                        }
#pragma unroll
                        for (int h = 0; h < Layout::kHalves; ++h) fw[h][i] = ld_chained(sw[h] + kb * step);
                    }
                    go = __all_sync(0xffffffffu, mbar_wait_polls(at(&s.scale_empty[c.slot]), c.parity ^ 1u));
                    if (!go) break;
#pragma unroll
                    for (int i = 0; i < Layout::kGroup; ++i)
#pragma unroll
                        for (int h = 0; h < Layout::kHalves; ++h)
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                s.scales[c.slot][i * Layout::kHalves + h][q * 32 + lane] = fa[q][i] * fw[h][i];
                    if (issue) s.tile[c.slot] = make_int4(tile.row0, tile.valid, tile.n * (kGated ? 128 : kBN), 0);
                    __syncwarp();
                    mbar_arrive(at(&s.scale_full[c.slot]), issue);
                    c.advance(kScaleSlots);
                }
            }
        }
        if (kSplit) {   // the sums' exchange below
            cluster_barrier();
            cluster_barrier();
        }
    } else {
        // ------------------------------------- scaled sums and the output
        registers_increase<kSumRegisters>();
        // a warpgroup takes half of the columns, in groups of 64: of the gate's and of the up
        // projection's (h = 0, 1), or side by side
        constexpr int kHalves = Layout::kHalves, kGroup = Layout::kGroup;
        constexpr int kApart = kGated ? 128 : 64;                    // from one group to the next
        constexpr int kFirst = kGated || kHalves == 1 ? 64 : 128;    // from one warpgroup's first to the other's
        const int wg = warp >> 2, quarter = warp & 3;
        const uint32_t stage = tiles_at + Layout::kStaging + warp * kStagingWarp;
        const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16) + wg * kFirst;
        const uint32_t first_empty = kCtas == 2 ? first_block_address(at(&s.acc_empty[0])) : 0;   // 8 bytes each
        Ring c;
        uint32_t parities = 0, pair_parity = 0;
        for (long long t = blockIdx.x / (kCtas * parts); go && t < total; t += kSplit ? total : gridDim.x / kCtas) {
            int4 tile;
            float2 acc[kHalves * 32];
#pragma unroll
            for (int i = 0; i < kHalves * 32; ++i) acc[i] = make_float2(0.0f, 0.0f);
            bool ok = true;
            for (int kb0 = 0; kb0 < nk; kb0 += kGroup) {
                ok = mbar_wait_polls(at(&s.scale_full[c.slot]), c.parity) && ok;
                const float *f0 = &s.scales[c.slot][0][quarter * 32 + lane];
                if (kb0 == 0) tile = s.tile[c.slot];
#pragma unroll
                for (int i = 0; i < kGroup; ++i) {
                    if (i > 0 && kb0 + i >= nk) break;
                    float f[kHalves];   // read here: a read after the wait would wait in its turn
#pragma unroll
                    for (int h = 0; h < kHalves; ++h)
                        f[h] = f0[(i * kHalves + (kGated ? h : kHalves == 1 ? 0 : wg)) * kRowTile];
                    ok = mbar_wait_polls(at(&s.acc_full[i]), (parities >> i) & 1u) && ok;
                    tcgen05_fence_after();
                    // every warp adds, rows past its own included: a branch would cost more
#pragma unroll
                    for (int k = 0; k < kHalves * 4; ++k) {
                        const int h = k / 4;
                        uint32_t r[16];
                        tmem_load(lanes + i * kBN + h * kApart + (k & 3) * 16, r);
                        tmem_wait_load(r);
                        if (k == kHalves * 4 - 1) {   // all read: the accumulator is free
                            tcgen05_fence_before();
                            if (kCtas == 2) mbar_arrive_cluster(first_empty + i * 8, issue);
                            else mbar_arrive(at(&s.acc_empty[i]), issue);
                        }
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            fma_pair(acc[k * 8 + j], make_float2(f[h], f[h]),
                                     make_float2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1])));
                    }
                    parities ^= 1u << i;
                }
                __syncwarp();
                mbar_arrive(at(&s.scale_empty[c.slot]), issue);
                c.advance(kScaleSlots);
                if (!ok) break;   // the lanes of a warp poll together and see the same
            }
            go = __all_sync(0xffffffffu, ok);
            uint32_t keep;   // rows of this warp that are this block's to write: a mask (kSplit) or how many
            if constexpr (kSplit) {
                const int row = quarter * 32 + lane, owner = row % parts;
                const bool valid = go && row < tile.y;
                constexpr int kRowBytes = kBN * 4 + 16;   // no bank conflicts between rows
                // part q's sums of the owner's rows, one after the other
                const auto room = [&](int q) {
                    return tiles_at + (q * (kRowTile / parts) + row / parts) * kRowBytes + wg * kBN * 2;
                };
                cluster_barrier();   // every block's products are done with its ring
                if (valid && owner != part) {
                    const uint32_t to = block_address(room(part), owner);
#pragma unroll
                    for (int i = 0; i < kHalves * 16; ++i)
                        st_cluster_v4(to + i * 16, make_float4(acc[2 * i].x, acc[2 * i].y, acc[2 * i + 1].x,
                                                               acc[2 * i + 1].y));
                }
                cluster_barrier();
                if (valid && owner == part) {
                    for (int q = 0; q < parts; ++q) {   // ascending, after the own: an order that never changes
                        if (q == part) continue;
                        const uint32_t from = room(q);
#pragma unroll
                        for (int i = 0; i < kHalves * 16; ++i) {
                            const uint4 v = ld_shared_v4(from + i * 16);
                            acc[2 * i].x += __uint_as_float(v.x);
                            acc[2 * i].y += __uint_as_float(v.y);
                            acc[2 * i + 1].x += __uint_as_float(v.z);
                            acc[2 * i + 1].y += __uint_as_float(v.w);
                        }
                    }
                }
                keep = __ballot_sync(0xffffffffu, valid && owner == part);
            } else {
                keep = (uint32_t)max(min(tile.y - quarter * 32, 32), 0);
            }
            if (!go) break;
            const int n0 = tile.z + wg * kFirst;                // first column
            const bool mine = keep != 0 && n0 < p.N;
            const size_t warp_row = (size_t)tile.x + quarter * 32;
            if constexpr (kGated) {
                const int I = p.N / 2;
                if (p.h && mine) {
                    unsigned char *h = reinterpret_cast<unsigned char *>(p.h + warp_row * p.N + n0);
                    store_bf16x64<kSplit>(acc, stage, h, (size_t)p.N * 2, keep, 128, lane);
                    store_bf16x64<kSplit>(acc + 32, stage, h + (size_t)I * 2, (size_t)p.N * 2, keep, 128, lane);
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
                mbar_arrive(at(&s.pair[quarter]), issue);
                go = __all_sync(0xffffffffu, mbar_wait_polls(at(&s.pair[quarter]), pair_parity));
                if (!go) break;
                amax = quant_amax(fmaxf(amax, s.amax[pair_parity][wg ^ 1][quarter * 32 + lane]));
                pair_parity ^= 1u;
                if (mine) {
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
                    store_rows64<kSplit>(v, stage, p.q + warp_row * I + n0, I, keep, 64, lane);
                    if (wg == 0 && (kSplit ? (keep >> lane & 1u) != 0 : lane < (int)keep))
                        p.q_scale[(warp_row + lane) * (I / 128) + n0 / 128] = quant_scale(amax);
                }
            } else if (mine) {
#pragma unroll
                for (int h = 0; h < kHalves; ++h) {
                    const int n = n0 + h * 64;
                    if (!p.out_f32) {
                        store_bf16x64<kSplit>(acc + h * 32, stage,
                                      static_cast<unsigned char *>(p.out) + (warp_row * p.N + n) * 2, (size_t)p.N * 2,
                                      keep, (p.N - n) * 2, lane);
                        continue;
                    }
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint4 v[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 v0 = acc[h * 32 + c * 8 + 2 * i], v1 = acc[h * 32 + c * 8 + 2 * i + 1];
                            v[i] = make_uint4(__float_as_uint(v0.x), __float_as_uint(v0.y), __float_as_uint(v1.x),
                                              __float_as_uint(v1.y));
                        }
                        store_rows64<kSplit>(v, stage,
                                     static_cast<unsigned char *>(p.out) + (warp_row * p.N + n + c * 16) * 4,
                                     (size_t)p.N * 4, keep, (p.N - n) * 4 - c * 64, lane);
                    }
                }
            }
        }
        if (kSplit && blockIdx.x / parts >= total) {   // no tile: the exchange is the cluster's all the same
            cluster_barrier();
            cluster_barrier();
        }
    }
    if (!go && issue) atomicOr(&g_product_error, MOE_DEVERR_COPY_TIMEOUT);
    __syncwarp();
    tcgen05_fence_before();
    if (kCtas == 2) cluster_barrier();   // nothing of the other block's reaches this one any more
    else __syncthreads();
    tcgen05_fence_after();
    if (warp == 9) tmem_free<kCtas, kTmemColumns>(tmem);
}

// ------------------------------------------------------------------- host

template <int kCtas, int kBN, bool kTransposed, bool kGated, bool kSplit = false>
static cudaError_t launch_tiles(const void *a, const void *w, ProductArgs p, cudaStream_t stream) {
    CUtensorMap map_a, map_few, map_w;
    if (!encode_bytes(&map_a, a, p.C, p.rows, 0, kRowTile) || !encode_bytes(&map_few, a, p.C, p.rows, 0, kFewRows) ||
        !encode_bytes(&map_w, w, kTransposed ? p.N : p.C, kTransposed ? p.C : p.N, p.E,
                      kTransposed ? kBlockK : weight_box<kCtas, kBN, kTransposed, kGated>()))
        return cudaErrorInvalidValue;
    auto kernel = expert_product_kernel<kCtas, kBN, kTransposed, kGated, kSplit>;
    constexpr int smem = ProductLayout<kCtas, kBN>::kBytes;
    static std::atomic<uint64_t> ready{0};
    const cudaError_t e = raise_shared_limit(reinterpret_cast<const void *>(kernel), smem, ready);
    if (e != cudaSuccess) return e;
    const int cols = kGated ? kBN / 2 : kBN;
    p.ntiles = ((kGated ? p.N / 2 : p.N) + cols - 1) / cols;
    // no more tiles than this exist; the blocks walk them
    const long long most = ((p.tails ? 0 : (long long)p.rows / (kCtas * kRowTile)) + (p.rows < p.E ? p.rows : p.E)) *
                           p.ntiles;
    const int groups = device_sm_count() / kCtas;
    cudaLaunchConfig_t cfg = {};
    const int parts = kSplit ? p.split : 1;
    cfg.gridDim = dim3((unsigned)(kSplit ? most * parts : kCtas * (most < groups ? (most > 0 ? most : 1) : groups)));
    cfg.blockDim = dim3(kProductThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kSplit ? parts : kCtas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, map_a, map_few, map_w, p);
}

// Into how many parts a tile's channels are split so that few tiles use the
// card: at least four stages each, and no more clusters than fit at once (of 152
// SMs, 15 clusters of eight, 36 of four, 76 of two).  Gated, 8 rows an expert, in
// one, two, four and eight parts: 2 experts x 2048 columns, 32 tiles, 22.6, 16.1,
// 13.2 and 32.8 us (four are taken); one expert, 16 tiles, 22.5, 15.6, 12.2 and 21.9
// (four: the 16 clusters of eight do not fit); one expert x 1024 columns, 8 tiles,
// two, four, eight: 15.5, 11.7, 11.2 (eight).  All over 7168 channels.
static int split_parts(long long tiles, int C) {
    const int stages = (C + kBlockK - 1) / kBlockK;
    for (int parts = 8; parts > 1; parts /= 2)
        if (tiles * parts <= device_sm_count() * (parts == 8 ? 0.79 : parts == 4 ? 0.95 : 1.0) && stages >= 4 * parts)
            return parts;
    return 1;
}

template <bool kTransposed, bool kGated>
static cudaError_t launch_product(const void *a, const void *w, ProductArgs p, cudaStream_t stream) {
    // Pairs where an expert has more than a single block's rows on average.  64 experts, 7168 x
    // 2048, rows each: 128: 188 us in pairs, 158 in single blocks; 160: 198 and 207; 256: 207 and
    // 230; 320: pairs and tails 360, pairs alone 380, single blocks 300.  256 experts of random
    // counts, in short runs: 262144 rows, pairs and tails 3.30 ms, pairs alone 3.28 to 3.33, single
    // blocks 3.39 to 3.41; 65536 rows, transposed, 4096 to 7168: 1.95, 2.16 to 2.19 and 1.89 to
    // 1.95 ms.  The tails start beside the pairs' end and wait for it: their reads may not come
    // before (see the kernel's wait).
    if (p.rows > (long long)p.E * kRowTile) {
        const cudaError_t e = launch_tiles<2, 256, kTransposed, kGated>(a, w, p, stream);
        if (e != cudaSuccess) return e;
        p.tails = true;
        return launch_tiles<1, 256, kTransposed, kGated>(a, w, p, stream);
    }
    const long long row_tiles = (long long)p.rows / kRowTile + (p.rows < p.E ? p.rows : p.E);   // at most
    constexpr int kNarrow = kGated ? 256 : 128;
    p.split = split_parts(row_tiles * ((p.N + kNarrow - 1) / kNarrow), p.C);
    if (p.split > 1) return launch_tiles<1, kNarrow, kTransposed, kGated, true>(a, w, p, stream);
    if constexpr (!kGated) {
        // tiles of 256 columns read A half as often (64 experts x 8 rows, 4096 to 7168 transposed:
        // 270 us, with 128 columns 285); where they are few, 128 columns spread over more SMs
        if (row_tiles * ((p.N + 255) / 256) < 4 * device_sm_count())
            return launch_tiles<1, 128, kTransposed, kGated>(a, w, p, stream);
    }
    return launch_tiles<1, 256, kTransposed, kGated>(a, w, p, stream);
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

cudaError_t product_error_word(int32_t **word) {
    static std::atomic<int32_t *> known[64];   // by device: the look-up takes a microsecond
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && (*word = known[dev].load(std::memory_order_acquire)) != nullptr) return cudaSuccess;
    e = cudaGetSymbolAddress(reinterpret_cast<void **>(word), g_product_error);
    if (e == cudaSuccess && dev < 64) known[dev].store(*word, std::memory_order_release);
    return e;
}

// Read and cleared in one step: a product on another stream whose wait runs out
// meanwhile is either in this read or in the next.
__global__ void take_product_error_kernel() { g_product_error_taken = atomicExch(&g_product_error, 0); }

cudaError_t read_product_error(int32_t *host_code, cudaStream_t stream) {
    *host_code = 0;
    cudaError_t e = cudaStreamSynchronize(stream);
    if (e != cudaSuccess) return e;
    // one reader at a time between the exchange and the copy of what it took
    static pthread_mutex_t reading = PTHREAD_MUTEX_INITIALIZER;
    pthread_mutex_lock(&reading);
    take_product_error_kernel<<<1, 1, 0, stream>>>();
    e = cudaGetLastError();
    int32_t v = 0;
    if (e == cudaSuccess)
        e = cudaMemcpyFromSymbolAsync(&v, g_product_error_taken, sizeof(v), 0, cudaMemcpyDeviceToHost, stream);
    const cudaError_t done = cudaStreamSynchronize(stream);   // v is written before this returns, whatever e is
    pthread_mutex_unlock(&reading);
    if (e == cudaSuccess) e = done;
    if (e == cudaSuccess) *host_code = v;
    return e;
}

}  // namespace moe
