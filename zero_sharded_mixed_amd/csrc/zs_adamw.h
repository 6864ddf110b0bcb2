// zs_adamw.h — the AdamW arithmetic and the 8-bit state format, shared by the steps of their own
// (adamw.hip, adamw8.hip) and the steps taken straight from the ranks' rows (fused_adamw.hip).
//
// AdamW [Loshchilov and Hutter, "Decoupled Weight Decay Regularization"], with s the gradient
// multiplier (grad_scale, over the loss scale, times the clip coefficient), lr the step's rate and
// d the parameter's decay multiplier:
//   g = s * g32,  m = beta1 m + (1 - beta1) g,  v = beta2 v + (1 - beta2) g^2,
//   p -= lr * weight_decay * d * p,
//   p -= (lr / (1 - beta1^t)) * m / (sqrt(v) / sqrt(1 - beta2^t) + eps).
#pragma once

#include <cmath>

#include "zs_adam.h"

namespace zs {

// ------------------------------------------------------------------- the caller's workspace --
// [fp32 hyperparameters][float4 per parameter][double per partial sum of squares], each part
// starting on a 256-byte boundary.  Every value a step reads is written earlier in that step, so
// steps on different streams need different workspaces and nothing has to be cleared.
constexpr int64_t kNormParts = 2048;  // partial sums of squares (norm.hip)
constexpr int64_t kWorkConstBytes = 256;
inline int64_t work_scal_bytes(int64_t n) { return (16 * n + 255) / 256 * 256; }
inline int64_t work_bytes(int64_t n) { return kWorkConstBytes + work_scal_bytes(n) + 8 * kNormParts; }
inline float* work_consts(void* w) { return static_cast<float*>(w); }
inline float4* work_scal(void* w) { return reinterpret_cast<float4*>(static_cast<char*>(w) + kWorkConstBytes); }
inline double* work_parts(void* w, int64_t n) {
    return reinterpret_cast<double*>(static_cast<char*>(w) + kWorkConstBytes + work_scal_bytes(n));
}

// One parameter's scalars of a step, formed in double and rounded to fp32 once: step size
// lr / (1 - beta1^t), 1 / sqrt(1 - beta2^t), lr * weight_decay * d, and the 32-bit key of the
// 8-bit states' rounding noise.
struct AdamWScal {
    float step, inv_sqrt_bc2, shrink;
    uint32_t key;
};
__device__ __forceinline__ AdamWScal scal_of(const float4& f) {
    return AdamWScal{f.x, f.y, f.z, __float_as_uint(f.w)};
}
// at a block-uniform index (scalar loads)
__device__ __forceinline__ AdamWScal ld_const_scal(const float4* p, int64_t i) {
    const float* f = reinterpret_cast<const float*>(p + i);
    return AdamWScal{ld_const(f, 0), ld_const(f, 1), ld_const(f, 2), __float_as_uint(ld_const(f, 3))};
}

// ------------------------------------------------------------------------- 32-bit states --
// One element in fp32 with every rounding spelled out.  Without decay (shrink = 0) the bits are
// those of adam_elem: fma(-0, p, p) is p.
__device__ __forceinline__ void adamw_elem(const AdamK& K, const AdamWScal& s, float g32, float& p, float& m, float& v) {
    p = __builtin_fmaf(-s.shrink, p, p);
    adam_elem(K, g32, p, m, v, s.step, s.inv_sqrt_bc2);
}

template <int DT>
__device__ __forceinline__ uint64_t pack4(const float4& p) {
    return uint64_t(uint32_t(from_f32<DT>(p.x)) | (uint32_t(from_f32<DT>(p.y)) << 16)) |
           uint64_t(uint32_t(from_f32<DT>(p.z)) | (uint32_t(from_f32<DT>(p.w)) << 16)) << 32;
}
__device__ __forceinline__ void store8(uint16_t* to, uint64_t v) {
    __builtin_nontemporal_store(v, gptr(reinterpret_cast<uint64_t*>(to)));
}

// The update of 4 consecutive columns of one parameter: stores p, m, v at p32, m, v and the four
// new 16-bit parameters at lp.
template <int DT>
__device__ __forceinline__ void adamw_quad(const AdamK& K, const AdamWScal& s, const float4& g, float4 p, float4 m,
                                           float4 v, float* p32, float* mm, float* vv, uint16_t* lp) {
    adamw_elem(K, s, g.x, p.x, m.x, v.x);
    adamw_elem(K, s, g.y, p.y, m.y, v.y);
    adamw_elem(K, s, g.z, p.z, m.z, v.z);
    adamw_elem(K, s, g.w, p.w, m.w, v.w);
    store4f(p32, p);
    store4f(mm, m);
    store4f(vv, v);
    store8(lp, pack4<DT>(p));
}

// -------------------------------------------------------------------------- 8-bit states --
// The momentum m and the root r of the variance (v = r^2; the root halves the range that has to
// be covered, and it is what the update divides by) are held in 8 bits times a power of two per
// block.  A block is the part of one parameter inside one aligned run of 256 shard columns: the
// blocks of a parameter without a gradient stay as they are whatever its neighbours do, and no
// parameter's scale depends on another's.  Block (run c, parameter i) has its scales at index
// c + i: walking the shard, either c or i grows from one block to the next, so no two blocks
// share an index and no table is needed.
//   m: sign, 4 exponent and 3 fraction bits, bias 7 (the OCP e4m3 code; its NaN is not used),
//      largest value 448; scale byte b stands for 2^(b - 127);
//   r: 4 exponent and 4 fraction bits without a sign, bias 15: 2^-18 .. 1.9375.
// A scale is the power of two that puts the block's largest value into the top binade (the next
// one where it lies above the top code).  Relative precision then does not depend on the scale,
// scaling is exact, and a code times its scale is exact in bf16 (the smallest scales are bounded
// so that it never leaves bf16's normal range).  A block with a value that is not finite gets
// scale 255 and codes 0, and reads as NaN: (+inf) * 0.
//
// Rounding is up or down with the probability that keeps the mean.  To the nearest, a moving
// average with beta2 = 0.999 would not move: a step changes r by a few hundredths of a percent, and
// half a code is 1.6 to 3.1%.  The noise is 16 bits for m and 16 for r of a hash of (seed, rank,
// step count, column), so a step's result is a function of its inputs.  A root that is not zero
// is never rounded to zero: the update divides by it.
constexpr int kRunShift = 8;
constexpr int64_t kRun = int64_t(1) << kRunShift;  // columns of a run: one wavefront, 4 columns a lane
constexpr uint32_t kScaleNan = 255;

// Bijective 32-bit mixing: multiplications by odd constants (fraction bits of the golden ratio and
// of sqrt 2) with the high bits folded down after each.
constexpr uint32_t kGold = 0x9E3779B9u, kRoot2 = 0xB504F333u, kRoot3 = 0xBB67AE85u;
__host__ __device__ __forceinline__ uint32_t mix32(uint32_t h) {
    h *= kGold;
    h ^= h >> 15;
    h *= kRoot2;
    return h ^ (h >> 16);
}

__device__ __forceinline__ uint32_t abs_bits(float f) { return __float_as_uint(f) & 0x7fffffffu; }
__device__ __forceinline__ float pow2_of_byte(uint32_t b) { return __uint_as_float(b << 23); }  // 255 -> +inf
// 2^(127 - b); 0 for the not-finite block (its codes become 0)
__device__ __forceinline__ float inverse_of_byte(uint32_t b) { return __uint_as_float((b == kScaleNan ? 0u : 254u - b) << 23); }

// Scale bytes from the bits of a block's largest magnitude (any NaN or infinity compares above
// every finite value).  Adding the carry moves a value above the top code (1.75 or 1.9375 times
// its power of two) into the next exponent.
__device__ __forceinline__ uint32_t moment_byte(uint32_t big) {
    const uint32_t e = (big + 0x1fffffu) >> 23;
    return big >= 0x7f800000u ? kScaleNan : (e < 24u ? 24u : e) - 8u;
}
__device__ __forceinline__ uint32_t root_byte(uint32_t big) {
    const uint32_t e = (big + 0x07ffffu) >> 23;
    return big >= 0x7f800000u ? kScaleNan : (e < 32u ? 32u : e);
}

// Codes.  Multiplying by the inverse scale is exact; the second factor moves the code's exponent
// range onto fp32's smallest exponents, so that the code is the number's leading bits, its own
// subnormals falling on fp32's.  `noise` is added below the code's last bit.
__device__ __forceinline__ uint32_t moment_code(float m, float inverse, uint32_t noise) {
    const uint32_t t = __float_as_uint((__uint_as_float(abs_bits(m)) * inverse) * 0x1p-120f);
    return ((t + noise) >> 20) | ((__float_as_uint(m) >> 24) & 0x80u);
}
__device__ __forceinline__ uint32_t root_code(float r, float inverse, uint32_t noise) {
    const uint32_t t = __float_as_uint((r * inverse) * 0x1p-112f);
    const uint32_t c = (t + noise) >> 19;
    return c == 0u && r > 0.0f ? 1u : c;
}
// To the nearest, ties to the even code.
__device__ __forceinline__ uint32_t moment_code_near(float m, float inverse) {
    const uint32_t t = __float_as_uint((__uint_as_float(abs_bits(m)) * inverse) * 0x1p-120f);
    return moment_code(m, inverse, 0x7ffffu + ((t >> 20) & 1u));
}
__device__ __forceinline__ uint32_t root_code_near(float r, float inverse) {
    const uint32_t t = __float_as_uint((r * inverse) * 0x1p-112f);
    return root_code(r, inverse, 0x3ffffu + ((t >> 19) & 1u));
}
__device__ __forceinline__ float moment_value(uint32_t code) {
    return __uint_as_float(((code & 0x7fu) << 20) | ((code & 0x80u) << 24)) * 0x1p120f;
}
__device__ __forceinline__ float root_value(uint32_t code) { return __uint_as_float(code << 19) * 0x1p112f; }

// The noise of column x for a parameter's key.
__device__ __forceinline__ uint32_t noise_of(uint32_t key, int64_t x) {
    return mix32(uint32_t(x) ^ key ^ (uint32_t(uint64_t(x) >> 32) * kRoot3));
}
__device__ __forceinline__ uint32_t moment_noise(uint32_t h) { return ((h & 0xffffu) << 4) + 8u; }
__device__ __forceinline__ uint32_t root_noise(uint32_t h) { return ((h >> 16) << 3) + 4u; }

// One element from the decoded states: new p, m and r, not yet rounded to 8 bits.  Products and
// sums are rounded one by one, no contraction: a value next to a code's border then falls on the
// side that the formula in fp32 gives.
__device__ __forceinline__ void adamw8_elem(const AdamK& K, const AdamWScal& s, float g32, float& p, float& m, float& r) {
#pragma clang fp contract(off)
    const float g = g32 * K.gs;
    m = K.b1 * m + K.c1 * g;
    r = sqrtf(K.b2 * (r * r) + K.c2 * (g * g));
    p = __builtin_fmaf(-s.shrink, p, p);
    p = __builtin_fmaf(-s.step, m / __builtin_fmaf(r, s.inv_sqrt_bc2, K.eps), p);
}

// Largest of a value over the 64 lanes (every lane active), in a scalar register: shifts within
// rows of 16 lanes, then the rows' last lanes broadcast, all in the vector ALU.
template <int CTRL>
__device__ __forceinline__ uint32_t max_dpp(uint32_t v) {
    const uint32_t o = uint32_t(__builtin_amdgcn_update_dpp(0, int(v), CTRL, 0xf, 0xf, false));
    return o > v ? o : v;
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = max_dpp<0x111>(v);  // row_shr:1
    v = max_dpp<0x112>(v);
    v = max_dpp<0x114>(v);
    v = max_dpp<0x118>(v);
    v = max_dpp<0x142>(v);  // row_bcast:15
    v = max_dpp<0x143>(v);  // row_bcast:31
    return uint32_t(__builtin_amdgcn_readlane(int(v), 63));
}
__device__ __forceinline__ uint32_t max4_bits(float a, float b, float c, float d) {
    const uint32_t x = abs_bits(a) > abs_bits(b) ? abs_bits(a) : abs_bits(b);
    const uint32_t y = abs_bits(c) > abs_bits(d) ? abs_bits(c) : abs_bits(d);
    return x > y ? x : y;
}

// What an 8-bit step works on.
struct AdamW8Args {
    float* p32;
    uint8_t* m8;
    uint8_t* r8;
    uint16_t* scales;  // [n_scales] low byte m's, high byte r's
    const uint8_t* live;
    const float4* scal;
    const float* consts;
    const int32_t* flag;
    uint16_t* arena;
};

// A run inside one live parameter: lane l has columns x .. x + 3, x = run start + 4 l.
struct Run8 {
    float4 p;
    uint32_t m8, r8, scale;
};
__device__ __forceinline__ Run8 run8_load(const AdamW8Args& A, int64_t x, int64_t block) {
    Run8 q;
    q.p = load4f_nt(A.p32 + x);
    q.m8 = __builtin_nontemporal_load(gptr(reinterpret_cast<const uint32_t*>(A.m8 + x)));
    q.r8 = __builtin_nontemporal_load(gptr(reinterpret_cast<const uint32_t*>(A.r8 + x)));
    q.scale = gptr(A.scales)[block];
    return q;
}
template <int DT>
__device__ __forceinline__ void run8_step(const AdamK& K, const AdamWScal& s, const AdamW8Args& A, int64_t x,
                                          int64_t block, const float4& g, Run8 q, uint16_t* lp) {
    const uint32_t pair = uint32_t(__builtin_amdgcn_readfirstlane(int(q.scale)));
    const float ms = pow2_of_byte(pair & 0xffu), rs = pow2_of_byte(pair >> 8);
    float m[4], r[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        m[t] = moment_value((q.m8 >> (8 * t)) & 0xffu) * ms;
        r[t] = root_value((q.r8 >> (8 * t)) & 0xffu) * rs;
    }
    adamw8_elem(K, s, g.x, q.p.x, m[0], r[0]);
    adamw8_elem(K, s, g.y, q.p.y, m[1], r[1]);
    adamw8_elem(K, s, g.z, q.p.z, m[2], r[2]);
    adamw8_elem(K, s, g.w, q.p.w, m[3], r[3]);
    const uint32_t mb = moment_byte(wave_max(max4_bits(m[0], m[1], m[2], m[3])));
    const uint32_t rb = root_byte(wave_max(max4_bits(r[0], r[1], r[2], r[3])));
    const float mi = inverse_of_byte(mb), ri = inverse_of_byte(rb);
    uint32_t mw = 0, rw = 0;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const uint32_t h = noise_of(s.key, x + t);
        mw |= moment_code(m[t], mi, moment_noise(h)) << (8 * t);
        rw |= root_code(r[t], ri, root_noise(h)) << (8 * t);
    }
    if (mb == kScaleNan) mw = 0;
    if (rb == kScaleNan) rw = 0;
    store4f(A.p32 + x, q.p);
    __builtin_nontemporal_store(mw, gptr(reinterpret_cast<uint32_t*>(A.m8 + x)));
    __builtin_nontemporal_store(rw, gptr(reinterpret_cast<uint32_t*>(A.r8 + x)));
    store8(lp, pack4<DT>(q.p));
    if (__lane_id() == 0) gptr(A.scales)[block] = uint16_t(mb | (rb << 8));
}

// A wavefront's scratch for a run of several blocks: the largest magnitudes of m and r of every
// block, at the block's first column inside the run.
struct RunMax {
    uint32_t m[kRun], r[kRun];
};
// Orders a wavefront's own LDS accesses: its lanes run together and its LDS operations complete
// in order, so this only has to hold the compiler and wait for what is in flight.
__device__ __forceinline__ void wave_lds_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
    __builtin_amdgcn_wave_barrier();
}

// The blocks of a run that holds several parameters, dead slots or a row gap: the columns
// [lo, hi) of it that belong to live parameters, element by element.  x: the lane's first column;
// i: the first parameter whose range ends after x; g_of(x): the reduced gradient of a column.
template <int DT, class G>
__device__ __forceinline__ void run8_mixed(const DevPlan& P, const AdamK& K, const AdamW8Args& A, RunMax* S, int64_t x,
                                           int64_t i, int64_t lo, int64_t hi, G g_of) {
    const int64_t run = x & ~(kRun - 1);
    const uint32_t l4 = uint32_t(x - run);
    float m[4] = {0, 0, 0, 0}, r[4] = {0, 0, 0, 0};
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
        first[t] = 0;
        if (xt < lo || xt >= hi) continue;
        while (i < P.n && P.end[i] <= xt) ++i;
        if (!(i < P.n && P.off[i] <= xt) || !A.live[i]) continue;
        own[t] = i;
        first[t] = uint32_t((P.off[i] > run ? P.off[i] : run) - run);
        const uint32_t pair = gptr(A.scales)[(run >> kRunShift) + i];
        const AdamWScal s = scal_of(A.scal[i]);
        float p = gptr(A.p32)[xt];
        m[t] = moment_value(gptr(A.m8)[xt]) * pow2_of_byte(pair & 0xffu);
        r[t] = root_value(gptr(A.r8)[xt]) * pow2_of_byte(pair >> 8);
        adamw8_elem(K, s, g_of(xt), p, m[t], r[t]);
        gptr(A.p32)[xt] = p;
        const int32_t b = P.bucket[i];
        const int64_t O = P.b_base[b];
        gptr(A.arena)[P.nd * O + P.rank * P.b_stride[b] + (xt - O)] = from_f32<DT>(p);
        atomicMax(&S->m[first[t]], abs_bits(m[t]));
        atomicMax(&S->r[first[t]], abs_bits(r[t]));
    }
    wave_lds_fence();  // also: every lane has read its old scales before one is written
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        if (own[t] < 0) continue;
        const int64_t xt = x + t;
        const uint32_t mb = moment_byte(S->m[first[t]]), rb = root_byte(S->r[first[t]]);
        const uint32_t h = noise_of(scal_of(A.scal[own[t]]).key, xt);
        gptr(A.m8)[xt] = mb == kScaleNan ? 0 : uint8_t(moment_code(m[t], inverse_of_byte(mb), moment_noise(h)));
        gptr(A.r8)[xt] = rb == kScaleNan ? 0 : uint8_t(root_code(r[t], inverse_of_byte(rb), root_noise(h)));
        if (l4 + t == first[t]) gptr(A.scales)[(run >> kRunShift) + own[t]] = uint16_t(mb | (rb << 8));
    }
    wave_lds_fence();  // the scratch is free for the wavefront's next run
}

// Checks of a step's hyperparameters, and the prepare launch into `work` (adamw.hip).
zero_status launch_adamw_prepare(const zero_plan* plan, const uint8_t* d_live, int32_t* d_steps,
                                 const zero_adamw_hparams* hp, const int32_t* d_flag, void* work, hipStream_t s,
                                 const char* who);
zero_status check_work(const void* work, const char* who);

}  // namespace zs
