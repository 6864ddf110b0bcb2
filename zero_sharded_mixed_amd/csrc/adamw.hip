// adamw.hip — the AdamW step over rank r's shard with its states in 32 bits, with the 16-bit
// write of the updated parameters into row r of every bucket's all-gather block, and the prepare
// launch that the 32-bit, the 8-bit and the fused steps share.
//
// Two launches, as for zero_adam_step.  adamw_prepare_kernel (one thread per parameter) reads the
// overflow flag (and sets it where the sum of squares of all ranks is not finite), advances the live parameters' step counts and forms every scalar of the step in
// double: the clip coefficient from the sum of squares, the gradient multiplier, the rate from
// the schedule's factor, and per parameter the step size, the bias correction and the decay.
// adamw_kernel then streams the shard: 16 bytes in and 14 out per element, bound by memory (6.2 TB/s on
// the GPT-2 list at Nd = 8, 948 us; 6.0 TB/s on the 7.5B list at Nd = 64, 580 us, on MI355X; counters:
// 5.86 GB moved of 5.84 needed).
#include <cmath>

#include "zs_adamw.h"

namespace zs {

struct AdamWHost {  // the hyperparameters by value, and the rounding noise's key without the step count
    double lr, beta1, beta2, eps, weight_decay, grad_scale, max_norm;
    const zero_loss_scaler* scaler;
    const double* sumsq;
    const float* lr_factor;
    const float* decay;
    float* norm_out;
    uint32_t key;
};

__global__ void adamw_prepare_kernel(DevPlan P, const uint8_t* __restrict__ live, int32_t* __restrict__ steps,
                                     int32_t* flag, AdamWHost H, float4* __restrict__ scal,
                                     float* __restrict__ consts) {
    const int64_t gid = blockIdx.x * int64_t(blockDim.x) + threadIdx.x;
    if (flag) {
        // The sum over the ranks is not finite on every rank as soon as one rank's gradient is not, while
        // only that rank's flag is set: all of them skip the step, and their flags say so to what
        // follows (the step's other launches, the loss scale).
        const bool lost = H.sumsq && !(fabs(*H.sumsq) < __builtin_inf());
        if (lost && gid == 0) atomicOr(flag, 1);
        if (lost || *flag) return;
    }
    if (gid == 0) {
        double mult = H.scaler ? H.grad_scale / double(H.scaler->scale) : H.grad_scale;
        if (H.sumsq) {
            // a sum that is not finite gives a multiplier that is not: without a flag that skips
            // the step, the parameters show it
            const double norm = sqrt(*H.sumsq) * fabs(mult);
            double coef = H.max_norm > 0.0 ? H.max_norm / (norm + 1e-6) : 1.0;
            coef = coef > 1.0 ? 1.0 : coef;
            if (!(norm < __builtin_inf())) coef = __builtin_nan("");
            if (H.norm_out) {
                H.norm_out[0] = float(norm);
                H.norm_out[1] = float(coef);
            }
            mult = mult * coef;
        }
        consts[AC_BETA1] = float(H.beta1);
        consts[AC_BETA2] = float(H.beta2);
        consts[AC_C1] = float(1.0 - H.beta1);
        consts[AC_C2] = float(1.0 - H.beta2);
        consts[AC_EPS] = float(H.eps);
        consts[AC_GSCALE] = float(mult);
    }
    const double lr = H.lr_factor ? H.lr * double(*H.lr_factor) : H.lr;
    for (int64_t i = gid; i < P.n; i += int64_t(gridDim.x) * blockDim.x) {
        if (!live[i]) {
            scal[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            continue;
        }
        const int32_t t = steps[i] + 1;
        steps[i] = t;
        const double bc1 = 1.0 - pow(H.beta1, double(t));
        const double bc2 = 1.0 - pow(H.beta2, double(t));
        const double shrink = lr * H.weight_decay * (H.decay ? double(H.decay[i]) : 1.0);
        scal[i] = make_float4(float(lr / bc1), float(1.0 / sqrt(bc2)), float(shrink),
                              __uint_as_float(mix32(uint32_t(t) ^ H.key)));
    }
}

struct AdamWArgs {
    const float* g32;
    float* p32;
    float* m;
    float* v;
    const float4* scal;
    const float* consts;
    const int32_t* flag;
    uint16_t* arena;
};

// From this many tiles on, the kernel reserves LDS for two blocks per CU (two_blocks_lds).  Measured
// on MI355X, calls among others, reserved against not: 22.9 us against 18.4 on the ragged list's 1270 tiles,
// 46 both at 4.0K tiles of the GPT-2 list, 81 against 80 at 7.9K, 159 against 165 at 15.8K, 312
// against 320 at 31.7K, 919 against 925 at 95K.
constexpr int64_t kManyTiles = 12 * 1024;
constexpr unsigned kManyTilesLds = two_blocks_lds(sizeof(TileMap));  // beside the kernel's own map
static_assert(kManyTilesLds + sizeof(TileMap) <= kBlockLdsMax, "within the LDS limit of a block");

// One block per tile of 2048 columns, lane-strided, every load and store in whole lines and
// nontemporal.  In a tile inside one parameter the scalars are uniform, and the two quads of a
// thread go one behind the other (the second's loads are issued when the first is computed,
// before its stores): with all eight loads at once the same kernel ran 4% slower on the GPT-2
// list and 2% slower on the 7.5B one.  The other tiles look their columns' owners up in LDS
// (zs_adamw.h): 16 us on the ragged list against 38 with the plan's tables in global memory.
template <int DT>
__global__ __launch_bounds__(kBlock) void adamw_kernel(DevPlan P, AdamWArgs A) {
    if (A.flag && *A.flag) return;
    __shared__ TileMap map;
    const AdamK K = load_adam_consts(A.consts);
    for (int64_t j = blockIdx.x; j < P.n_tiles; j += gridDim.x) {
        const Tile T(P, A.scal, j);
        if (T.whole) {
            if (!T.s.live()) continue;
            uint16_t* lp = A.arena + T.row(P);
            float4 g[2], p[2], m[2], v[2];
            const auto load = [&](int q) {
                const int64_t x = T.x0 + quad_col(q);
                g[q] = load4f_nt(A.g32 + x);
                p[q] = load4f_nt(A.p32 + x);
                m[q] = load4f_nt(A.m + x);
                v[q] = load4f_nt(A.v + x);
                __builtin_amdgcn_sched_barrier(0);
            };
            const auto compute = [&](int q) {
                adamw_elem(K, T.s, g[q].x, p[q].x, m[q].x, v[q].x);
                adamw_elem(K, T.s, g[q].y, p[q].y, m[q].y, v[q].y);
                adamw_elem(K, T.s, g[q].z, p[q].z, m[q].z, v[q].z);
                adamw_elem(K, T.s, g[q].w, p[q].w, m[q].w, v[q].w);
                __builtin_amdgcn_sched_barrier(0);
            };
            const auto store = [&](int q) {
                const int64_t x = T.x0 + quad_col(q);
                store4f(A.p32 + x, p[q]);
                store4f(A.m + x, m[q]);
                store4f(A.v + x, v[q]);
                store8(lp + quad_col(q), pack4<DT>(p[q]));
            };
            load(0);
            compute(0);
            load(1);
            store(0);
            compute(1);
            store(1);
            continue;
        }
        mixed_tile(map, P, A.scal, T, j, [&](int64_t) {
#pragma unroll 1
            for (int q = 0; q < 2; ++q) {
                const int64_t x = T.x0 + quad_col(q);
                if (x < P.shard_numel)
                    adamw_quad_mixed<DT>(map, K, int(quad_col(q)), load4f_nt(A.g32 + x), load4f_nt(A.p32 + x),
                                         load4f_nt(A.m + x), load4f_nt(A.v + x), A.p32 + x, A.m + x, A.v + x, A.arena);
            }
        });
    }
}

zero_status check_work(const void* work, const char* who) {
    if (!work || !host_aligned16(work)) return fail(ZERO_EINVAL, "%s: work must be a 16-byte aligned pointer", who);
    return ZERO_OK;
}

zero_status launch_adamw_prepare(const zero_plan* plan, const uint8_t* d_live, int32_t* d_steps,
                                 const zero_adamw_hparams* hp, int32_t* d_flag, void* work, hipStream_t s,
                                 const char* who) {
    if (!d_live || !d_steps || !hp) return fail(ZERO_EINVAL, "%s: NULL pointer", who);
    const zero_status st = check_work(work, who);
    if (st != ZERO_OK) return st;
    if (reinterpret_cast<uintptr_t>(d_flag) % 4 != 0) return fail(ZERO_EINVAL, "%s: flag not 4-byte aligned", who);
    const auto at_least_0 = [](double x) { return std::isfinite(x) && x >= 0.0; };
    if (!at_least_0(hp->lr) || !(hp->beta1 >= 0.0) || !(hp->beta1 < 1.0) || !(hp->beta2 >= 0.0) || !(hp->beta2 < 1.0) ||
        !at_least_0(hp->weight_decay) || !std::isfinite(hp->grad_scale) || !at_least_0(hp->max_norm))
        return fail(ZERO_EINVAL, "%s: hyperparameters out of range", who);
    // eps keeps the padding's update, 0 / (0 + eps), a number, and its reciprocal finite
    if (!std::isfinite(float(hp->eps)) || !(float(hp->eps) >= 0x1p-126f))
        return fail(ZERO_EINVAL, "%s: eps must be a normal number of fp32, above zero", who);
    if (!hp->grad_sumsq && (hp->max_norm > 0.0 || hp->norm_out))
        return fail(ZERO_EINVAL, "%s: max_norm and norm_out need grad_sumsq", who);
    if (reinterpret_cast<uintptr_t>(hp->grad_sumsq) % 8 != 0 ||
        (reinterpret_cast<uintptr_t>(hp->loss_scaler) | reinterpret_cast<uintptr_t>(hp->lr_factor) |
         reinterpret_cast<uintptr_t>(hp->decay) | reinterpret_cast<uintptr_t>(hp->norm_out)) % 4 != 0)
        return fail(ZERO_EINVAL, "%s: misaligned hyperparameter pointer", who);
    uint32_t key = mix32(uint32_t(plan->rank) ^ kRoot3);
    key = mix32(key ^ uint32_t(hp->seed));
    key = mix32(key ^ uint32_t(hp->seed >> 32));
    const AdamWHost H{hp->lr, hp->beta1, hp->beta2, hp->eps, hp->weight_decay, hp->grad_scale, hp->max_norm,
                      hp->loss_scaler, hp->grad_sumsq, hp->lr_factor, hp->decay, hp->norm_out, key};
    adamw_prepare_kernel<<<grid_for((plan->n + 255) / 256, 1024), 256, 0, s>>>(
        plan->dev, d_live, d_steps, d_flag, H, work_scal(work), work_consts(work));
    return check_launch(who);
}

}  // namespace zs

using namespace zs;

extern "C" zero_status zero_adamw_get_sizes(const zero_plan* plan, zero_adamw_sizes* out) {
    if (!plan || !out) return fail(ZERO_EINVAL, "zero_adamw_get_sizes: NULL argument");
    out->work_bytes = work_bytes(plan->n);
    out->n_scales = ((plan->shard_numel + kRun - 1) >> kRunShift) + plan->n;
    return ZERO_OK;
}

extern "C" zero_status zero_adamw_prepare(const zero_plan* plan, const uint8_t* d_live, int32_t* d_steps,
                                          const zero_adamw_hparams* hp, int32_t* d_flag, void* d_work,
                                          void* stream) {
    const zero_status st = check_device(plan);
    if (st != ZERO_OK) return st;
    return launch_adamw_prepare(plan, d_live, d_steps, hp, d_flag, d_work, (hipStream_t)stream, "zero_adamw_prepare");
}

extern "C" zero_status zero_adamw_step(const zero_plan* plan, const float* d_g32, float* d_p32, float* d_m, float* d_v,
                                       const uint8_t* d_live, int32_t* d_steps, const zero_adamw_hparams* hp,
                                       int32_t* d_flag, void* d_arena, void* d_work, void* stream) {
    const char* who = "zero_adamw_step";
    zero_status st = check_device(plan);
    if (st != ZERO_OK) return st;
    // an empty shard still advances the step counts of live parameters; its arrays may be NULL
    if (plan->shard_numel != 0 && (!d_g32 || !d_p32 || !d_m || !d_v || !d_arena))
        return fail(ZERO_EINVAL, "%s: NULL pointer", who);
    if (!host_aligned16(d_g32) || !host_aligned16(d_p32) || !host_aligned16(d_m) || !host_aligned16(d_v) ||
        !host_aligned16(d_arena))
        return fail(ZERO_EINVAL, "%s: shard arrays and arena must be 16-byte aligned", who);
    hipStream_t s = (hipStream_t)stream;
    if ((st = launch_adamw_prepare(plan, d_live, d_steps, hp, d_flag, d_work, s, who)) != ZERO_OK) return st;
    if (plan->shard_numel == 0) return ZERO_OK;
    const AdamWArgs A{d_g32, d_p32, d_m, d_v, work_scal(d_work), work_consts(d_work), d_flag,
                      static_cast<uint16_t*>(d_arena)};
    const int g = grid_for(plan->dev.n_tiles);
    const unsigned lds = plan->dev.n_tiles >= kManyTiles ? kManyTilesLds : 0u;
    if (plan->dtype == ZERO_BF16) adamw_kernel<ZERO_BF16><<<g, kBlock, lds, s>>>(plan->dev, A);
    else adamw_kernel<ZERO_FP16><<<g, kBlock, lds, s>>>(plan->dev, A);
    return check_launch(who);
}
