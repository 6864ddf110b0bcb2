// norm.hip — the sum of squares of the reduced gradient over the live part of the shard, for
// clipping by the global norm (the ranks add their sums; the step forms the coefficient).
//
// One read of the shard (4 bytes per element), bound by memory: 120 us for the GPT-2 list's 194.7M
// elements at Nd = 8 on MI355X (6.5 TB/s), and 5 us for adding the parts.  Squares and sums are in double:
// the square of any fp32 value is exact there and cannot overflow, so the sum is finite exactly
// when every live value is, which makes the overflow verdict free.  The shard's tiles are dealt
// to at most kNormParts parts, each summed by one block in a fixed order, and the parts are
// added in a fixed order: the sum's bits do not depend on the grid or on timing.
#include "zs_adamw.h"

namespace zs {

constexpr int kFinishBlock = 1024;  // threads of the block that adds the parts
// Shards of at most this many tiles (of 2048 columns) are summed by one block in one launch.
// Measured on MI355X, a call among others, one launch against two: 6.1 us against 9.5 at 4 tiles,
// 6.6 against 9.5 at 15, 10.9 against 9.5 at 32 (4.9, 6.4 and 10.7 against 6.8 in a graph).
constexpr int64_t kOneBlockTiles = 16;

// Sum over the block's WAVES wavefronts, in thread 0: lanes by halving distance, then the
// wavefronts in order.
template <int WAVES>
__device__ __forceinline__ double block_sum(double v, double* lds) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_down(v, d);
    if (__lane_id() == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    double s = 0.0;
    if (threadIdx.x == 0)
        for (int w = 0; w < WAVES; ++w) s += lds[w];
    __syncthreads();
    return s;
}
__device__ __forceinline__ void write_sum(double s, double* sumsq, int32_t* flag) {
    *sumsq = s;
    if (flag && !(s < __builtin_inf())) atomicOr(flag, 1);
}

__device__ __forceinline__ void add_squares(double& acc, const float4& g) {
    acc = __builtin_fma(double(g.x), double(g.x), acc);
    acc = __builtin_fma(double(g.y), double(g.y), acc);
    acc = __builtin_fma(double(g.z), double(g.z), acc);
    acc = __builtin_fma(double(g.w), double(g.w), acc);
}

// The share of thread `tid` of kBlock of tile j (uniform across the wavefront): lane-strided where
// the tile lies inside one parameter, 8 columns in a row otherwise.
__device__ __forceinline__ void tile_squares(const DevPlan& P, const float* __restrict__ g32,
                                             const uint8_t* __restrict__ live, int64_t j, int tid, double& acc) {
    const int64_t x0 = j << kTileShift;
    const int64_t iu = ld_const(P.tile_first, j);
    const int64_t ic = iu < P.n ? iu : P.n - 1;
    if (iu < P.n && ld_const(P.off, ic) <= x0 && ld_const(P.end, ic) >= x0 + kTileCols) {
        if (!ld_const(live, ic)) return;
        const float4 a = load4f(g32 + x0 + 4 * tid);
        const float4 b = load4f(g32 + x0 + 4 * (kBlock + tid));
        add_squares(acc, a);
        add_squares(acc, b);
        return;
    }
    const int64_t x = x0 + int64_t(tid) * kChunk;
    if (x >= P.shard_numel) return;
    const unsigned mask = live_mask8(P, live, x, param_of_column(P, x));
    if (mask == 0) return;
    const float4 a = load4f(g32 + x);
    const float4 b = load4f(g32 + x + 4);
    const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int t = 0; t < 8; ++t) {
        const double d = (mask >> t) & 1u ? double(v[t]) : 0.0;
        acc = __builtin_fma(d, d, acc);
    }
}

__global__ __launch_bounds__(kBlock) void sumsq_parts_kernel(DevPlan P, const float* __restrict__ g32,
                                                             const uint8_t* __restrict__ live, int64_t n_parts,
                                                             double* __restrict__ parts) {
    __shared__ double lds[kBlock / 64];
    for (int64_t q = blockIdx.x; q < n_parts; q += gridDim.x) {
        double acc = 0.0;
        for (int64_t j = q; j < P.n_tiles; j += n_parts) tile_squares(P, g32, live, j, threadIdx.x, acc);
        const double s = block_sum<kBlock / 64>(acc, lds);
        if (threadIdx.x == 0) parts[q] = s;
    }
}

__global__ __launch_bounds__(kFinishBlock) void sumsq_finish_kernel(const double* __restrict__ parts, int64_t n_parts,
                                                                    double* __restrict__ sumsq,
                                                                    int32_t* __restrict__ flag) {
    __shared__ double lds[kFinishBlock / 64];
    double acc = 0.0;
    for (int64_t q = threadIdx.x; q < n_parts; q += kFinishBlock) acc += parts[q];
    const double s = block_sum<kFinishBlock / 64>(acc, lds);
    if (threadIdx.x == 0) write_sum(s, sumsq, flag);
}

// A small shard in one launch: the block's quarters take the tiles in turn.
__global__ __launch_bounds__(kFinishBlock) void sumsq_small_kernel(DevPlan P, const float* __restrict__ g32,
                                                                   const uint8_t* __restrict__ live,
                                                                   double* __restrict__ sumsq,
                                                                   int32_t* __restrict__ flag) {
    __shared__ double lds[kFinishBlock / 64];
    double acc = 0.0;
    const int quarter = __builtin_amdgcn_readfirstlane(int(threadIdx.x) / kBlock);
    for (int64_t j = quarter; j < P.n_tiles; j += kFinishBlock / kBlock)
        tile_squares(P, g32, live, j, threadIdx.x % kBlock, acc);
    const double s = block_sum<kFinishBlock / 64>(acc, lds);
    if (threadIdx.x == 0) write_sum(s, sumsq, flag);
}

}  // namespace zs

using namespace zs;

extern "C" zero_status zero_grad_sumsq(const zero_plan* plan, const float* d_g32, const uint8_t* d_live, double* d_sumsq,
                                       int32_t* d_flag, void* d_work, void* stream) {
    const char* who = "zero_grad_sumsq";
    zero_status st = check_device(plan);
    if (st != ZERO_OK) return st;
    if (!d_sumsq || reinterpret_cast<uintptr_t>(d_sumsq) % 8 != 0)
        return fail(ZERO_EINVAL, "%s: sumsq must be an 8-byte aligned pointer", who);
    if (plan->shard_numel != 0 && (!d_g32 || !d_live)) return fail(ZERO_EINVAL, "%s: NULL pointer", who);
    if (!host_aligned16(d_g32)) return fail(ZERO_EINVAL, "%s: g32 not 16-byte aligned", who);
    if (reinterpret_cast<uintptr_t>(d_flag) % 4 != 0) return fail(ZERO_EINVAL, "%s: flag not 4-byte aligned", who);
    if ((st = check_work(d_work, who)) != ZERO_OK) return st;
    hipStream_t s = (hipStream_t)stream;
    if (plan->dev.n_tiles <= kOneBlockTiles) {
        sumsq_small_kernel<<<1, kFinishBlock, 0, s>>>(plan->dev, d_g32, d_live, d_sumsq, d_flag);
        return check_launch(who);
    }
    double* parts = work_parts(d_work, plan->n);
    const int64_t n_parts = plan->dev.n_tiles < kNormParts ? plan->dev.n_tiles : kNormParts;
    sumsq_parts_kernel<<<grid_for(n_parts), kBlock, 0, s>>>(plan->dev, d_g32, d_live, n_parts, parts);
    if ((st = check_launch(who)) != ZERO_OK) return st;
    sumsq_finish_kernel<<<1, kFinishBlock, 0, s>>>(parts, n_parts, d_sumsq, d_flag);
    return check_launch(who);
}
