// adamw8.hip — the AdamW step over rank r's shard with its momentum and the root of its variance
// in 8 bits (the format is in zs_adamw.h), and the conversions from and to wider states.
//
// The step reads g32, p32 and two codes and writes p32, two codes and the 16-bit parameter: 10
// bytes in and 8 out per element (30 with 32-bit states), and the states take 2 bytes instead of 8.
// A wavefront takes a run of 256 columns, 4 a lane, so that a block's largest magnitude is one
// reduction inside the wavefront and every array is read and written in whole lines.
//
// Measured on MI355X: 569 us for the GPT-2 list's 194.7M elements at Nd = 8 (6.2 TB/s; counters: 1.97
// GB fetched and 1.57 written against 1.95 and 1.56 that the step needs), 360 us for the 7.5B list's
// 116.6M at Nd = 64 (5.8 TB/s).  The arithmetic is 74 vector instructions an element.  11 of them keep
// the smallest roots, the quotient's last bit and parameters that are -0 or infinite right; without
// those it took 547 and 351 us.  With the conversions, the root and the quotient written out it was 95
// instructions and 625 us.  More wavefronts than the 80 registers allow (forced to 64 registers) or
// fewer are slower, measured at 547 us: 611 at eight per SIMD, 556 at four, 594 at three.
#include <cmath>

#include "zs_adamw.h"

namespace zs {

// First column of column x's run.
__device__ __forceinline__ int64_t run_of(int64_t x) { return x & ~(kRun - 1); }

template <int DT>
__global__ __launch_bounds__(kBlock) void adamw8_kernel(DevPlan P, AdamW8Args A, const float* __restrict__ g32) {
    if (A.flag && *A.flag) return;
    __shared__ TileMap map;
    __shared__ RunMax scratch[kBlock / 64];
    const AdamK K = load_adam_consts(A.consts);
    for (int64_t j = blockIdx.x; j < P.n_tiles; j += gridDim.x) {
        const Tile T(P, A.scal, j);
        if (T.whole) {
            if (!T.s.live()) continue;
            uint16_t* lp = A.arena + T.row(P);
            // the second run's loads go out when the first is computed, before its stores: 4% faster
            // than both runs' loads at once
            const int64_t xa = T.x0 + quad_col(0), xb = T.x0 + quad_col(1);
            const int64_t block = (xa >> kRunShift) + T.first;
            const float4 ga = load4f_nt(g32 + xa);
            Run8 a = run8_load(A, xa);
            a.scale = gptr(A.scales)[block];
            const Out8 oa = run8_math(K, T.s, xa, ga, a);
            __builtin_amdgcn_sched_barrier(0);
            const float4 gb = load4f_nt(g32 + xb);
            Run8 b = run8_load(A, xb);
            b.scale = gptr(A.scales)[block + ((xb - xa) >> kRunShift)];
            __builtin_amdgcn_sched_barrier(0);
            run8_store<DT>(A, xa, block, a.p, oa, lp + quad_col(0));
            __builtin_amdgcn_sched_barrier(0);
            const Out8 ob = run8_math(K, T.s, xb, gb, b);
            run8_store<DT>(A, xb, block + ((xb - xa) >> kRunShift), b.p, ob, lp + quad_col(1));
            continue;
        }
        mixed_tile(map, P, A.scal, T, j, [&](int64_t first) {
#pragma unroll 1
            for (int q = 0; q < 2; ++q) {
                const int64_t x = T.x0 + quad_col(q);
                if (run_of(x) >= P.shard_numel) break;
                const bool in = x < P.shard_numel;
                const float4 none = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                run8_mixed<DT>(map, K, A, &scratch[threadIdx.x >> 6], first, x, int(quad_col(q)), in,
                               in ? load4f_nt(g32 + x) : none, in ? run8_load(A, x) : Run8{none, 0, 0, 0});
            }
        });
    }
}

// Codes to the nearest (ties to even) of 32-bit states, every parameter's, live or not.  A run at
// a time through the wavefront's scratch.
__global__ __launch_bounds__(kBlock) void adamw8_load_kernel(DevPlan P, const float* __restrict__ mm,
                                                             const float* __restrict__ vv, uint8_t* __restrict__ m8,
                                                             uint8_t* __restrict__ r8, uint16_t* __restrict__ scales) {
    __shared__ RunMax scratch[kBlock / 64];
    RunMax* S = &scratch[threadIdx.x >> 6];
    for (int64_t j = blockIdx.x; j < P.n_tiles; j += gridDim.x) {
#pragma unroll 1
        for (int q = 0; q < 2; ++q) {
            const int64_t x = (j << kTileShift) + quad_col(q);
            const int64_t run = run_of(x);
            if (run >= P.shard_numel) break;
            int64_t i = param_of_column(P, x);
            const uint32_t l4 = uint32_t(x - run);
            float m[4], r[4];
            int64_t own[4];
            uint32_t first[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                S->m[l4 + t] = 0;
                S->r[l4 + t] = 0;
            }
            wave_lds_fence();
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int64_t xt = x + t;
                own[t] = -1;
                while (i < P.n && P.end[i] <= xt) ++i;
                if (!(i < P.n && P.off[i] <= xt)) continue;
                own[t] = i;
                first[t] = uint32_t((P.off[i] > run ? P.off[i] : run) - run);
                m[t] = gptr(mm)[xt];
                r[t] = sqrtf(gptr(vv)[xt]);
                atomicMax(&S->m[first[t]], abs_bits(m[t]));
                atomicMax(&S->r[first[t]], abs_bits(r[t]));
            }
            wave_lds_fence();
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                if (own[t] < 0) continue;
                const int64_t xt = x + t;
                const uint32_t mb = moment_byte(S->m[first[t]]), rb = root_byte(S->r[first[t]]);
                gptr(m8)[xt] = mb == kScaleNan ? 0 : uint8_t(moment_near(m[t], mb));
                gptr(r8)[xt] = rb == kScaleNan ? 0 : uint8_t(root_near(r[t], rb));
                if (l4 + t == first[t]) gptr(scales)[(run >> kRunShift) + own[t]] = uint16_t(mb | (rb << 8));
            }
            wave_lds_fence();
        }
    }
}

// The states' values in bf16, which holds them exactly: 2 bytes in and 4 out per element.  8
// columns in a row per thread: 8-byte loads and 16-byte stores of whole lines (190 us for 194.7M
// elements on MI355X, 6.1 TB/s; 4-byte loads and 8-byte stores with a search per thread: 370).
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    return (__float_as_uint(a) >> 16) | (__float_as_uint(b) & 0xffff0000u);
}
__device__ __forceinline__ void unload8(const uint8_t* m8, const uint8_t* r8, uint32_t pair, uint16_t* m16,
                                        uint16_t* r16) {
    const float ms = pow2_of_byte(pair & 0xffu);
    const uint64_t mw = __builtin_nontemporal_load(gptr(reinterpret_cast<const uint64_t*>(m8)));
    const uint64_t rw = __builtin_nontemporal_load(gptr(reinterpret_cast<const uint64_t*>(r8)));
    float lo[4], hi[4];
    moment_values(uint32_t(mw), lo);
    moment_values(uint32_t(mw >> 32), hi);
    const uint32_t m[4] = {bf16_pair(lo[0] * ms, lo[1] * ms), bf16_pair(lo[2] * ms, lo[3] * ms),
                           bf16_pair(hi[0] * ms, hi[1] * ms), bf16_pair(hi[2] * ms, hi[3] * ms)};
    uint32_t r[4];
#pragma unroll
    for (int t = 0; t < 4; ++t)
        r[t] = bf16_pair(root_value(uint32_t(rw >> (16 * t)) & 0xffu, pair >> 8),
                         root_value(uint32_t(rw >> (16 * t + 8)) & 0xffu, pair >> 8));
    store16(m16, make_uint4(m[0], m[1], m[2], m[3]));
    store16(r16, make_uint4(r[0], r[1], r[2], r[3]));
}
__global__ __launch_bounds__(kBlock) void adamw8_unload_kernel(DevPlan P, const uint8_t* __restrict__ m8,
                                                               const uint8_t* __restrict__ r8,
                                                               const uint16_t* __restrict__ scales,
                                                               uint16_t* __restrict__ m16, uint16_t* __restrict__ r16) {
    __shared__ TilePlaces places;
    for (int64_t j = blockIdx.x; j < P.n_tiles; j += gridDim.x) {
        const int64_t x0 = j << kTileShift;
        const int64_t x = x0 + int64_t(threadIdx.x) * kChunk;
        const int64_t iu = ld_const(P.tile_first, j);
        const int64_t ic = iu < P.n ? iu : P.n - 1;
        if (iu < P.n && ld_const(P.off, ic) <= x0 && ld_const(P.end, ic) >= x0 + kTileCols) {
            unload8(m8 + x, r8 + x, gptr(scales)[(x >> kRunShift) + ic], m16 + x, r16 + x);
            continue;
        }
        for_places(
            places, P, j, iu, [](int, int64_t) {},
            [&](int64_t first) {
                if (x >= P.shard_numel) return;
                const int xr = int(x - x0);
                const int64_t block = (x >> kRunShift) + first;
                int k = places.find(xr);
                if (places.holds(k, xr) && places.end[k] >= xr + kChunk) {
                    unload8(m8 + x, r8 + x, gptr(scales)[block + k], m16 + x, r16 + x);
                    return;
                }
#pragma unroll
                for (int t = 0; t < kChunk; ++t) {
                    while (k < places.count && places.end[k] <= xr + t) ++k;
                    if (!places.holds(k, xr + t)) continue;
                    const uint32_t pair = gptr(scales)[block + k];
                    float m[4];
                    moment_values(gptr(m8)[x + t], m);
                    gptr(m16)[x + t] = uint16_t(bf16_pair(m[0] * pow2_of_byte(pair & 0xffu), 0.0f));
                    gptr(r16)[x + t] = uint16_t(bf16_pair(root_value(gptr(r8)[x + t], pair >> 8), 0.0f));
                }
            });
    }
}

}  // namespace zs

using namespace zs;

extern "C" zero_status zero_adamw8_step(const zero_plan* plan, const float* d_g32, float* d_p32, uint8_t* d_m8,
                                        uint8_t* d_r8, uint8_t* d_scales, const uint8_t* d_live, int32_t* d_steps,
                                        const zero_adamw_hparams* hp, int32_t* d_flag, void* d_arena,
                                        void* d_work, void* stream) {
    const char* who = "zero_adamw8_step";
    zero_status st = check_device(plan);
    if (st != ZERO_OK) return st;
    if (plan->shard_numel != 0 && (!d_g32 || !d_p32 || !d_m8 || !d_r8 || !d_scales || !d_arena))
        return fail(ZERO_EINVAL, "%s: NULL pointer", who);
    if (!host_aligned16(d_g32) || !host_aligned16(d_p32) || !host_aligned16(d_m8) || !host_aligned16(d_r8) ||
        !host_aligned16(d_scales) || !host_aligned16(d_arena))
        return fail(ZERO_EINVAL, "%s: shard arrays, scales and arena must be 16-byte aligned", who);
    hipStream_t s = (hipStream_t)stream;
    if ((st = launch_adamw_prepare(plan, d_live, d_steps, hp, d_flag, d_work, s, who)) != ZERO_OK) return st;
    if (plan->shard_numel == 0) return ZERO_OK;
    const AdamW8Args A{d_p32, d_m8, d_r8, reinterpret_cast<uint16_t*>(d_scales), work_scal(d_work),
                       work_consts(d_work), d_flag, static_cast<uint16_t*>(d_arena)};
    const int g = grid_for(plan->dev.n_tiles);
    if (plan->dtype == ZERO_BF16) adamw8_kernel<ZERO_BF16><<<g, kBlock, 0, s>>>(plan->dev, A, d_g32);
    else adamw8_kernel<ZERO_FP16><<<g, kBlock, 0, s>>>(plan->dev, A, d_g32);
    return check_launch(who);
}

extern "C" zero_status zero_adamw8_load(const zero_plan* plan, const float* d_m, const float* d_v, uint8_t* d_m8,
                                        uint8_t* d_r8, uint8_t* d_scales, void* stream) {
    const char* who = "zero_adamw8_load";
    const zero_status st = check_device(plan);
    if (st != ZERO_OK) return st;
    if (plan->shard_numel == 0) return ZERO_OK;
    if (!d_m || !d_v || !d_m8 || !d_r8 || !d_scales) return fail(ZERO_EINVAL, "%s: NULL pointer", who);
    if (!host_aligned16(d_m) || !host_aligned16(d_v) || !host_aligned16(d_m8) || !host_aligned16(d_r8) ||
        !host_aligned16(d_scales))
        return fail(ZERO_EINVAL, "%s: state arrays and scales must be 16-byte aligned", who);
    adamw8_load_kernel<<<grid_for(plan->dev.n_tiles), kBlock, 0, (hipStream_t)stream>>>(
        plan->dev, d_m, d_v, d_m8, d_r8, reinterpret_cast<uint16_t*>(d_scales));
    return check_launch(who);
}

extern "C" zero_status zero_adamw8_unload(const zero_plan* plan, const uint8_t* d_m8, const uint8_t* d_r8,
                                          const uint8_t* d_scales, void* d_m16, void* d_r16, void* stream) {
    const char* who = "zero_adamw8_unload";
    const zero_status st = check_device(plan);
    if (st != ZERO_OK) return st;
    if (plan->shard_numel == 0) return ZERO_OK;
    if (!d_m8 || !d_r8 || !d_scales || !d_m16 || !d_r16) return fail(ZERO_EINVAL, "%s: NULL pointer", who);
    if (!host_aligned16(d_m8) || !host_aligned16(d_r8) || !host_aligned16(d_scales) || !host_aligned16(d_m16) ||
        !host_aligned16(d_r16))
        return fail(ZERO_EINVAL, "%s: state arrays and scales must be 16-byte aligned", who);
    adamw8_unload_kernel<<<grid_for(plan->dev.n_tiles), kBlock, 0, (hipStream_t)stream>>>(
        plan->dev, d_m8, d_r8, reinterpret_cast<const uint16_t*>(d_scales), static_cast<uint16_t*>(d_m16),
        static_cast<uint16_t*>(d_r16));
    return check_launch(who);
}
