// fused_adamw.hip — the reduce and the AdamW step of one bucket in a single pass, with 32-bit or
// 8-bit states: the fused path of fused.hip (same rows, same order of sums, same overflow verdict
// from the inputs) with the steps of adamw.hip and adamw8.hip.  The reduced gradient never goes
// to memory, so an element moves 2 Nd bytes of rows and 26 bytes of states and parameters (14 with
// 8-bit states), and the results are bit-identical to zero_reduce_shard and the step of its own.
#include "zs_adamw.h"

namespace zs {

// Row forms (zs_common.h) and blocks per CU go by the number of rows, with a border for each width
// of the states.  Measured on MI355X, a step's launches on the GPT-2 list, the form for few rows
// against the one for many:
//   32 bits: 1.36 ms against 1.76 at Nd = 8, 1.00 against 1.12 at 16, 0.817 against 0.826 at 32, 0.723
//     against 0.711 at 64;
//   8 bits: 1.03 against 1.24 at 8, 0.83 against 0.88 at 16, 0.75 against 0.72 at 32, 0.69 against 0.66
//     at 64.
// Few rows, 32 bits: fewest registers on whole tiles, one group of rows in flight on the others, at
//   four blocks per CU (1.40 ms at five at Nd = 8).
// Many rows, 32 bits: two groups on the others (180 registers, two wavefronts per SIMD): 0.82 ms
//   against 0.85 with one group on the ragged list at Nd = 1024.
// Few rows, 8 bits: a group at once on whole tiles too, five blocks (1.07 ms with fewest registers,
//   1.23 at three blocks).
// Many rows, 8 bits: fewest registers, one group on the others, at three blocks (7.5B list, Nd = 64: 3.05
//   ms; 3.15 at five, 3.17 with two groups).
constexpr int64_t kManyRows = 48, kManyRows8 = 24;
// Reserved where fewer blocks are faster: with the kernels' own 16 and 24 KB, four and three blocks
// fit a CU's 160 KB.
constexpr unsigned kFewBlocksLds = 16 * 1024;
constexpr int64_t kBlockLds = kTileCols * 4 + sizeof(TileMap) + kFewBlocksLds;
constexpr int64_t kBlockLds8 = kBlockLds + kBlock / 64 * sizeof(RunMax);
static_assert(4 * kBlockLds <= kLdsPerCu && 5 * kBlockLds > kLdsPerCu, "four blocks per CU");
static_assert(3 * kBlockLds8 <= kLdsPerCu && 4 * kBlockLds8 > kLdsPerCu, "three blocks per CU");

// A tile inside one live parameter: every thread sums 8 columns in a row (16-byte loads of every
// rank's row), the sums go through LDS, and the step takes the tile lane-strided.  The tile's
// reduced gradient as the thread's two quads:
template <int DT, int FORM>
__device__ __forceinline__ void tile_sums(float4* g_lds, const uint16_t* rows_u, int64_t nd, int64_t row_stride) {
    float acc[8];
    reduce_rows8<DT, FORM, true>(rows_u, threadIdx.x * kChunk, nd, row_stride, acc);
    g_lds[2 * threadIdx.x] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    g_lds[2 * threadIdx.x + 1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
}

struct BucketRows {
    int64_t base, row, stride, tile0, n_tile;
    const uint16_t* rows;
    int64_t row_stride;
};

// The other tiles: the sums of the 8-column groups that hold a live column of the bucket.  The rest
// of the LDS is left as it was: those sums belong to nobody.
template <int DT, int FORM>
__device__ __forceinline__ void mixed_sums(float4* g_lds, const DevPlan& P, const BucketRows& B,
                                           const uint8_t* __restrict__ live, int64_t x0) {
    const int64_t x = x0 + int64_t(threadIdx.x) * kChunk;
    const int64_t c = x - B.base;
    if (c < 0 || c >= B.row || live_mask8(P, live, x, param_of_column(P, x)) == 0) return;
    float acc[8];
    reduce_rows8<DT, FORM, true>(B.rows + (x0 - B.base), threadIdx.x * kChunk, P.nd, B.row_stride, acc);
    g_lds[2 * threadIdx.x] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    g_lds[2 * threadIdx.x + 1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
}

template <int DT, int WHOLE, int MIXED>
__global__ __launch_bounds__(kBlock) void reduce_adamw_kernel(DevPlan P, BucketRows B, const uint8_t* __restrict__ live,
                                                              float* __restrict__ p32, float* __restrict__ m,
                                                              float* __restrict__ v, const float4* __restrict__ scal,
                                                              const float* __restrict__ consts,
                                                              const int32_t* __restrict__ flag,
                                                              uint16_t* __restrict__ arena) {
    if (flag && *flag) return;
    __shared__ float4 g_lds[kTileCols / 4];
    __shared__ TileMap map;
    const AdamK K = load_adam_consts(consts);
    uint16_t* const lp_row = arena + P.nd * B.base + P.rank * B.stride;  // row r of the bucket's block
    for (int64_t w = blockIdx.x; w < B.n_tile; w += gridDim.x) {
        const int64_t j = B.tile0 + w;
        const Tile T(P, scal, j);
        if (T.whole) {
            if (!T.s.live()) continue;
            tile_sums<DT, WHOLE>(g_lds, B.rows + (T.x0 - B.base), P.nd, B.row_stride);
            float4 p4[2], m4[2], v4[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int64_t x = T.x0 + quad_col(q);
                p4[q] = load4f_nt(p32 + x);
                m4[q] = load4f_nt(m + x);
                v4[q] = load4f_nt(v + x);
            }
            __syncthreads();
            float4 g4[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) g4[q] = g_lds[quad_col(q) / 4];
            __syncthreads();  // the LDS is free for the block's next tile
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int64_t x = T.x0 + quad_col(q);
                adamw_quad<DT>(K, T.s, g4[q], p4[q], m4[q], v4[q], p32 + x, m + x, v + x, lp_row + (x - B.base));
            }
            continue;
        }
        mixed_sums<DT, MIXED>(g_lds, P, B, live, T.x0);
        mixed_tile(map, P, scal, T, j, [&](int64_t) {
#pragma unroll 1
            for (int q = 0; q < 2; ++q) {
                const int64_t x = T.x0 + quad_col(q);
                if (x >= B.base && x < B.base + B.row)
                    adamw_quad_mixed<DT>(map, K, int(quad_col(q)), g_lds[quad_col(q) / 4], load4f_nt(p32 + x),
                                         load4f_nt(m + x), load4f_nt(v + x), p32 + x, m + x, v + x, arena);
            }
        });
    }
}

template <int DT, int WHOLE, int MIXED>
__global__ __launch_bounds__(kBlock) void reduce_adamw8_kernel(DevPlan P, BucketRows B, const uint8_t* __restrict__ live,
                                                               AdamW8Args A) {
    if (A.flag && *A.flag) return;
    __shared__ float4 g_lds[kTileCols / 4];
    __shared__ TileMap map;
    __shared__ RunMax scratch[kBlock / 64];
    const AdamK K = load_adam_consts(A.consts);
    uint16_t* const lp_row = A.arena + P.nd * B.base + P.rank * B.stride;
    for (int64_t w = blockIdx.x; w < B.n_tile; w += gridDim.x) {
        const int64_t j = B.tile0 + w;
        const Tile T(P, A.scal, j);
        if (T.whole) {
            if (!T.s.live()) continue;
            tile_sums<DT, WHOLE>(g_lds, B.rows + (T.x0 - B.base), P.nd, B.row_stride);
            Run8 r[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int64_t x = T.x0 + quad_col(q);
                r[q] = run8_load(A, x);
                r[q].scale = gptr(A.scales)[(x >> kRunShift) + T.first];
            }
            __syncthreads();
            float4 g4[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) g4[q] = g_lds[quad_col(q) / 4];
            __syncthreads();
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int64_t x = T.x0 + quad_col(q);
                run8_step<DT>(K, T.s, A, x, (x >> kRunShift) + T.first, g4[q], r[q], lp_row + (x - B.base));
            }
            continue;
        }
        mixed_sums<DT, MIXED>(g_lds, P, B, live, T.x0);
        mixed_tile(map, P, A.scal, T, j, [&](int64_t first) {
#pragma unroll 1
            for (int q = 0; q < 2; ++q) {
                const int64_t x = T.x0 + quad_col(q);
                const int64_t run = x & ~(kRun - 1);
                if (run >= B.base + B.row || run + kRun <= B.base) continue;
                const bool in = x >= B.base && x < B.base + B.row;
                run8_mixed<DT>(map, K, A, &scratch[threadIdx.x >> 6], first, x, int(quad_col(q)), in,
                               g_lds[quad_col(q) / 4],
                               in ? run8_load(A, x) : Run8{make_float4(0.0f, 0.0f, 0.0f, 0.0f), 0, 0, 0});
            }
        });
    }
}

// Checks of a bucket's index and rows, as zero_reduce_adam_bucket.  rows->n_tile = 0: nothing to do.
static zero_status bucket_rows(const zero_plan* plan, int64_t b, const void* d_rows, int64_t row_stride,
                               const char* who, BucketRows* out) {
    *out = BucketRows{};
    if (b < 0 || b >= plan->n_buckets) return fail(ZERO_EINVAL, "%s: bucket %lld out of range", who, (long long)b);
    const int64_t* br = plan->h_bucket + b * kBucketFields;
    const int64_t base = br[BF_BASE], row = br[BF_ROW], stride = br[BF_STRIDE];
    if (row == 0) return ZERO_OK;
    if (!d_rows || !host_aligned16(d_rows)) return fail(ZERO_EINVAL, "%s: rows must be a 16-byte aligned pointer", who);
    if (row_stride < stride || row_stride % kChunk != 0)
        return fail(ZERO_EINVAL, "%s: row_stride %lld must be >= %lld and a multiple of 8", who, (long long)row_stride,
                    (long long)stride);
    const int64_t tile0 = base >> kTileShift;
    *out = BucketRows{base, row, stride, tile0, ((base + row + kTileCols - 1) >> kTileShift) - tile0,
                      static_cast<const uint16_t*>(d_rows), row_stride};
    return ZERO_OK;
}

}  // namespace zs

using namespace zs;

extern "C" zero_status zero_reduce_adamw_bucket(const zero_plan* plan, int64_t b, const void* d_rows, int64_t row_stride,
                                                const uint8_t* d_live, float* d_p32, float* d_m, float* d_v,
                                                const int32_t* d_flag, void* d_arena, void* d_work, void* stream) {
    const char* who = "zero_reduce_adamw_bucket";
    zero_status st = check_device(plan);
    BucketRows B;
    if (st != ZERO_OK || (st = bucket_rows(plan, b, d_rows, row_stride, who, &B)) != ZERO_OK || B.n_tile == 0) return st;
    if (!d_live || !d_p32 || !d_m || !d_v || !d_arena) return fail(ZERO_EINVAL, "%s: NULL pointer", who);
    if (!host_aligned16(d_p32) || !host_aligned16(d_m) || !host_aligned16(d_v) || !host_aligned16(d_arena))
        return fail(ZERO_EINVAL, "%s: shard arrays and arena must be 16-byte aligned", who);
    if ((st = check_work(d_work, who)) != ZERO_OK) return st;
    const int g = grid_for(B.n_tile);
    hipStream_t s = (hipStream_t)stream;
    const bool bf16 = plan->dtype == ZERO_BF16, many = plan->nd >= kManyRows;
    auto kern = many ? (bf16 ? reduce_adamw_kernel<ZERO_BF16, kRowsLow, kRowsPipe>
                             : reduce_adamw_kernel<ZERO_FP16, kRowsLow, kRowsPipe>)
                     : (bf16 ? reduce_adamw_kernel<ZERO_BF16, kRowsLow, kRowsGroup>
                             : reduce_adamw_kernel<ZERO_FP16, kRowsLow, kRowsGroup>);
    kern<<<g, kBlock, many ? 0u : kFewBlocksLds, s>>>(plan->dev, B, d_live, d_p32, d_m, d_v, work_scal(d_work),
                                                      work_consts(d_work), d_flag, static_cast<uint16_t*>(d_arena));
    return check_launch(who);
}

extern "C" zero_status zero_reduce_adamw8_bucket(const zero_plan* plan, int64_t b, const void* d_rows,
                                                 int64_t row_stride, const uint8_t* d_live, float* d_p32,
                                                 uint8_t* d_m8, uint8_t* d_r8, uint8_t* d_scales,
                                                 const int32_t* d_flag, void* d_arena, void* d_work, void* stream) {
    const char* who = "zero_reduce_adamw8_bucket";
    zero_status st = check_device(plan);
    BucketRows B;
    if (st != ZERO_OK || (st = bucket_rows(plan, b, d_rows, row_stride, who, &B)) != ZERO_OK || B.n_tile == 0) return st;
    if (!d_live || !d_p32 || !d_m8 || !d_r8 || !d_scales || !d_arena) return fail(ZERO_EINVAL, "%s: NULL pointer", who);
    if (!host_aligned16(d_p32) || !host_aligned16(d_m8) || !host_aligned16(d_r8) || !host_aligned16(d_scales) ||
        !host_aligned16(d_arena))
        return fail(ZERO_EINVAL, "%s: shard arrays, scales and arena must be 16-byte aligned", who);
    if ((st = check_work(d_work, who)) != ZERO_OK) return st;
    const AdamW8Args A{d_p32, d_m8, d_r8, reinterpret_cast<uint16_t*>(d_scales), work_scal(d_work),
                       work_consts(d_work), d_flag, static_cast<uint16_t*>(d_arena)};
    const int g = grid_for(B.n_tile);
    const bool bf16 = plan->dtype == ZERO_BF16, many = plan->nd >= kManyRows8;
    auto kern = many ? (bf16 ? reduce_adamw8_kernel<ZERO_BF16, kRowsLow, kRowsGroup>
                             : reduce_adamw8_kernel<ZERO_FP16, kRowsLow, kRowsGroup>)
                     : (bf16 ? reduce_adamw8_kernel<ZERO_BF16, kRowsGroup, kRowsGroup>
                             : reduce_adamw8_kernel<ZERO_FP16, kRowsGroup, kRowsGroup>);
    kern<<<g, kBlock, many ? kFewBlocksLds : 0u, (hipStream_t)stream>>>(plan->dev, B, d_live, A);
    return check_launch(who);
}
