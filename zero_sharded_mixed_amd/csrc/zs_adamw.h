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
// [fp32 hyperparameters][4 words per parameter][double per partial sum of squares], each part
// starting on a 256-byte boundary.  Every value a step reads is written earlier in that step, so
// steps on different streams need different workspaces and nothing has to be cleared.
// Partial sums of squares (norm.hip): eight blocks of 256 threads a CU.  Measured on MI355X, the GPT-2
// list at Nd = 8 and at 192: 122 and 12.6 us with 2048 parts, 180 and 14.4 with 1024, 128 and 13.1 with
// 4096.
constexpr int64_t kNormParts = 2048;
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
// 8-bit states' rounding noise.  The second is at least 1, and 0 for a parameter without a
// gradient: one load tells a step's kernels both.
struct AdamWScal {
    float step, inv_sqrt_bc2, shrink;
    uint32_t key;
    __device__ __forceinline__ bool live() const { return inv_sqrt_bc2 != 0.0f; }
};
__device__ __forceinline__ AdamWScal scal_of(const float4& f) {
    return AdamWScal{f.x, f.y, f.z, __float_as_uint(f.w)};
}
// at a block-uniform index (scalar loads)
__device__ __forceinline__ AdamWScal ld_const_scal(const float4* p, int64_t i) {
    const float* f = reinterpret_cast<const float*>(p + i);
    return AdamWScal{ld_const(f, 0), ld_const(f, 1), ld_const(f, 2), __float_as_uint(ld_const(f, 3))};
}

// A tile, block-uniform: its first column, the first parameter whose range ends after it, whether
// that parameter covers the whole tile, its scalars, and the arena index of the tile's first column
// in its row.  All loaded at once, so that they cost two memory round trips, not one each.
struct Tile {
    int64_t x0, first;
    bool whole;
    AdamWScal s;
    int32_t bucket;
    __device__ __forceinline__ Tile(const DevPlan& P, const float4* scal, int64_t j) {
        x0 = j << kTileShift;
        first = ld_const(P.tile_first, j);
        const int64_t ic = first < P.n ? first : P.n - 1;
        const int64_t off = ld_const(P.off, ic), end = ld_const(P.end, ic);
        s = ld_const_scal(scal, ic);
        bucket = ld_const(P.bucket, ic);
        whole = (first < P.n) & (off <= x0) & (end >= x0 + kTileCols);
    }
    __device__ __forceinline__ int64_t row(const DevPlan& P) const {
        const int64_t O = ld_const(P.b_base, bucket);
        return P.nd * O + P.rank * ld_const(P.b_stride, bucket) + (x0 - O);
    }
};

// ------------------------------------------------------- the parameters of a mixed tile --
// A tile that several parameters, dead slots or a row gap share.  The block copies the places,
// scalars and rows of its parameters into LDS in one round of loads, kTileParams of them at a
// time, so that a column's owner costs no chain of global loads.  A tile of more parameters is
// gone through once per kTileParams: a column is taken when its owner is there.
constexpr int kTileParams = 256;
struct TilePlaces {
    int32_t begin[kTileParams], end[kTileParams];  // columns relative to the tile, cut to it
    int count;

    __device__ __forceinline__ int find(int xr) const {  // first k whose range ends after xr
        int lo = 0, hi = count;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (end[mid] > xr) hi = mid; else lo = mid + 1;
        }
        return lo;
    }
    __device__ __forceinline__ bool holds(int k, int xr) const { return k < count && begin[k] <= xr; }
};
struct TileMap : TilePlaces {
    float4 scal[kTileParams];
    int64_t row[kTileParams];  // arena index of the tile's first column in the parameter's own row
    __device__ __forceinline__ AdamWScal scalars(int k) const { return scal_of(scal[k]); }
};
__device__ __forceinline__ int32_t cut_to_tile(int64_t x) { return int32_t(x < 0 ? 0 : x > kTileCols ? kTileCols : x); }

// For every kTileParams parameters [first, ..) of mixed tile j, `from` the first of them all: M filled
// (and more(k, i) for entry k, parameter i), then f(first), all threads of the block in it, and a
// barrier: what f reads of LDS may be written again.
template <class M, class More, class F>
__device__ __forceinline__ void for_places(M& map, const DevPlan& P, int64_t j, int64_t from, More more, F f) {
    const int64_t x0 = j << kTileShift;
    const int64_t last = ld_const(P.tile_first, j + 1);  // reaches past the tile, or does not exist
    const int64_t end = last < P.n ? last + 1 : P.n;
#pragma unroll 1
    for (int64_t first = from; first < end; first += kTileParams) {
        const int k = threadIdx.x;
        const int64_t i = first + k;
        if (i < end) {
            map.begin[k] = cut_to_tile(P.off[i] - x0);
            map.end[k] = cut_to_tile(P.end[i] - x0);
            more(k, i);
        }
        if (k == 0) map.count = int(end - first < kTileParams ? end - first : kTileParams);
        __syncthreads();
        f(first);
        __syncthreads();
    }
}
static_assert(kTileParams == kBlock, "a thread per parameter of the map");
template <class F>
__device__ __forceinline__ void mixed_tile(TileMap& M, const DevPlan& P, const float4* scal, const Tile& T, int64_t j,
                                           F f) {
    for_places(
        M, P, j, T.first,
        [&](int k, int64_t i) {
            M.scal[k] = scal[i];
            const int32_t b = P.bucket[i];
            const int64_t O = P.b_base[b];
            M.row[k] = P.nd * O + P.rank * P.b_stride[b] + (T.x0 - O);
        },
        f);
}

// ------------------------------------------------------------------------- 32-bit states --
// p less its decay.  Without decay (shrink = 0) every p keeps its bits: fma(-0, p, p) would turn -0 into
// 0 and an infinity into NaN.
__device__ __forceinline__ float decayed(const AdamWScal& s, float p) {
    const float q = __builtin_fmaf(-s.shrink, p, p);
    return s.shrink == 0.0f ? p : q;
}

// One element in fp32 with every rounding spelled out.  Without decay the bits are those of adam_elem.
__device__ __forceinline__ void adamw_elem(const AdamK& K, const AdamWScal& s, float g32, float& p, float& m, float& v) {
    p = decayed(s, p);
    adam_elem(K, g32, p, m, v, s.step, s.inv_sqrt_bc2);
}

template <int DT>
__device__ __forceinline__ uint64_t pack4(const float4& p) {
    return uint64_t(uint32_t(from_f32<DT>(p.x)) | (uint32_t(from_f32<DT>(p.y)) << 16)) |
           uint64_t(uint32_t(from_f32<DT>(p.z)) | (uint32_t(from_f32<DT>(p.w)) << 16)) << 32;
}
// Four fp32 values rounded to 16 bits, to the nearest even.  bf16 has a conversion instruction for
// pairs, which agrees with from_f32 on every value but the payload of a NaN.
typedef float zs_pair_f32 __attribute__((ext_vector_type(2)));
typedef __bf16 zs_pair_bf16 __attribute__((ext_vector_type(2)));
template <int DT>
__device__ __forceinline__ uint64_t pack4_fast(const float4& p) {
    if constexpr (DT == ZERO_BF16) {
        const zs_pair_f32 a = {p.x, p.y}, b = {p.z, p.w};
        return uint64_t(__builtin_bit_cast(uint32_t, __builtin_convertvector(a, zs_pair_bf16))) |
               uint64_t(__builtin_bit_cast(uint32_t, __builtin_convertvector(b, zs_pair_bf16))) << 32;
    } else {
        return pack4<DT>(p);
    }
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

// The same for 4 columns of a mixed tile, xr the first's place in it; columns of dead parameters or of
// nobody are loaded and not written.  Where every lane's columns lie inside one parameter each, as
// above; else each column is computed with its owner's scalars in all lanes alike (one lane's
// boundary would otherwise cost the wavefront both ways).
template <int DT>
__device__ __forceinline__ void adamw_quad_mixed(const TileMap& M, const AdamK& K, int xr, const float4& g, float4 p,
                                                 float4 m, float4 v, float* p32, float* mm, float* vv, uint16_t* arena) {
    const float* gq = &g.x;
    float *pq = &p.x, *mq = &m.x, *vq = &v.x;
    int k = M.find(xr);
    const bool one = M.holds(k, xr) && M.end[k] >= xr + 4;
    if (__all(one)) {
        const AdamWScal s = M.scalars(k);
        if (s.live()) adamw_quad<DT>(K, s, g, p, m, v, p32, mm, vv, arena + M.row[k] + xr);
        return;
    }
    int64_t row[4];  // -1: not written
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        while (k < M.count && M.end[k] <= xr + t) ++k;
        row[t] = -1;
        if (!M.holds(k, xr + t)) continue;
        const AdamWScal s = M.scalars(k);
        if (!s.live()) continue;
        row[t] = M.row[k];
        adamw_elem(K, s, gq[t], pq[t], mq[t], vq[t]);
    }
    // rows of one bucket are one
    if (row[0] >= 0 && row[0] == row[1] && row[0] == row[2] && row[0] == row[3]) {
        store4f(p32, p);
        store4f(mm, m);
        store4f(vv, v);
        store8(arena + row[0] + xr, pack4<DT>(p));
        return;
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        if (row[t] < 0) continue;
        gptr(p32)[t] = pq[t];
        gptr(mm)[t] = mq[t];
        gptr(vv)[t] = vq[t];
        gptr(arena)[row[t] + xr + t] = from_f32<DT>(pq[t]);
    }
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
// 2^(127 - b); 0 for the block that is not finite (its codes become 0)
__device__ __forceinline__ float inverse_of_byte(uint32_t b) {
    return __uint_as_float((b == kScaleNan ? 0u : 254u - b) << 23);
}

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

// Decoding.  The momentum's code has a conversion instruction.  The root's becomes the leading bits
// of an fp32 number with the smallest exponents (its subnormals fall on fp32's), moved in place by
// ldexp: code << 19 stands for its value times 2^-112.
typedef float zs_f32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ void moment_values(uint32_t word, float (&m)[4]) {
    const zs_f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(int(word), false);
    const zs_f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8(int(word), true);
    m[0] = a.x;
    m[1] = a.y;
    m[2] = b.x;
    m[3] = b.y;
}
__device__ __forceinline__ float root_value(uint32_t code, uint32_t byte) {
    const float r = __builtin_amdgcn_ldexpf(__uint_as_float(code << 19), int(byte) - 15);
    return byte == kScaleNan ? __builtin_nanf("") : r;
}

// Rounding codes of scaled values.  The momentum's instruction adds the noise's 20 high bits below
// the code's last bit; for the root they are added by hand.
template <int SEL>
__device__ __forceinline__ uint32_t moment_round(float scaled, uint32_t noise, uint32_t word) {
    return uint32_t(__builtin_amdgcn_cvt_sr_fp8_f32(scaled, noise, int(word), SEL));
}
__device__ __forceinline__ uint32_t root_bits(float r, uint32_t byte) {
    return __float_as_uint(__builtin_amdgcn_ldexpf(r, 15 - int(byte)));
}
__device__ __forceinline__ uint32_t root_round(float r, uint32_t byte, uint32_t noise) {
    const uint32_t c = (root_bits(r, byte) + noise) >> 19;
    return c == 0u && r > 0.0f ? 1u : c;
}
// To the nearest, ties to the even code.
__device__ __forceinline__ uint32_t moment_near(float m, uint32_t byte) {
    const uint32_t t = __float_as_uint((__uint_as_float(abs_bits(m)) * inverse_of_byte(byte)) * 0x1p-120f);
    return ((t + 0x7ffffu + ((t >> 20) & 1u)) >> 20) | ((__float_as_uint(m) >> 24) & 0x80u);
}
__device__ __forceinline__ uint32_t root_near(float r, uint32_t byte) {
    return root_round(r, byte, 0x3ffffu + ((root_bits(r, byte) >> 19) & 1u));
}

// The noise of column x for a parameter's key.
__device__ __forceinline__ uint32_t noise_of(uint32_t key, int64_t x) {
    return mix32(uint32_t(x) ^ key ^ (uint32_t(uint64_t(x) >> 32) * kRoot3));
}
// 16 bits each and half of what is below them: for m at the top of 20 of 32 bits, for r as 19 bits
__device__ __forceinline__ uint32_t moment_noise(uint32_t h) { return (h << 16) | 0x8000u; }
__device__ __forceinline__ uint32_t root_noise(uint32_t h) { return ((h >> 13) & ~7u) | 4u; }

// Square root to within a unit in the last place: the reciprocal root's estimate and one Newton
// step with the exact residual, half the instructions of the correctly rounded sequence, from which
// it differs once in 10^4 values.  0 gives 0; below 2^-126 it falls short (see moved_root).
__device__ __forceinline__ float root_of(float v) {
    const float y = __builtin_amdgcn_rsqf(fmaxf(v, 0x1p-126f));
    const float q = v * y;
    return __builtin_fmaf(__builtin_fmaf(-q, q, v), 0.5f * y, q);
}

// sqrt(b2 r^2 + c2 g^2).  The states reach down to 2^-113 and gradients to 2^-149, whose squares leave
// fp32's range, so where the larger of the two lies below 1/2 both are brought to it by a power of two,
// which is exact: the variance is then at least min(b2, c2) / 4, every rounding is the formula's own
// without its range, and a root above zero stays above zero.  With beta2 = 0 the old root is dropped
// first (a NaN stays): beside a gradient far below it, it would not fit.
__device__ __forceinline__ float moved_root(const AdamK& K, float r, float g) {
#pragma clang fp contract(off)
    r *= K.b2 > 0.0f ? 1.0f : 0.0f;
    const int e = min(__builtin_amdgcn_frexp_expf(fmaxf(r, fabsf(g))), 0);
    r = __builtin_amdgcn_ldexpf(r, -e);
    g = __builtin_amdgcn_ldexpf(g, -e);
    return __builtin_amdgcn_ldexpf(root_of(K.b2 * (r * r) + K.c2 * (g * g)), e);
}

// m / den: the product with the reciprocal's estimate (off by a unit or two) and one correction by the
// exact residual, which leaves the nearest value, but for one in 2^20 that lies next to the middle.
// Where |m| < 2^-102 the residual loses bits below fp32's range, and the product's unit stays.  den is
// finite and at least 2^-126, as eps is.
__device__ __forceinline__ float quotient_of(float m, float den) {
    const float y = __builtin_amdgcn_rcpf(den);
    const float q = m * y;
    return __builtin_fmaf(__builtin_fmaf(-q, den, m), y, q);
}

// One element from the decoded states: new p, m and r, not yet rounded to 8 bits.  Products and
// sums of m and v are rounded one by one, no contraction: a value next to a code's border then
// falls on the side that the formula in fp32 gives.  The root and the quotient are an estimate and
// one correction each: with the compiler's correctly rounded sequences the step's arithmetic takes as
// long as its memory traffic.
__device__ __forceinline__ void adamw8_elem(const AdamK& K, const AdamWScal& s, float g32, float& p, float& m, float& r) {
#pragma clang fp contract(off)
    const float g = g32 * K.gs;
    m = K.b1 * m + K.c1 * g;
    r = moved_root(K, r, g);
    p = decayed(s, p);
    p = __builtin_fmaf(-s.step, quotient_of(m, __builtin_fmaf(r, s.inv_sqrt_bc2, K.eps)), p);
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
    return max(max(max(abs_bits(a), abs_bits(b)), abs_bits(c)), abs_bits(d));
}

// What an 8-bit step works on.
struct AdamW8Args {
    float* p32;
    uint8_t* m8;
    uint8_t* r8;
    uint16_t* scales;  // [n_scales] low byte m's, high byte r's
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
__device__ __forceinline__ Run8 run8_load(const AdamW8Args& A, int64_t x) {
    Run8 q;
    q.p = load4f_nt(A.p32 + x);
    q.m8 = __builtin_nontemporal_load(gptr(reinterpret_cast<const uint32_t*>(A.m8 + x)));
    q.r8 = __builtin_nontemporal_load(gptr(reinterpret_cast<const uint32_t*>(A.r8 + x)));
    q.scale = 0;
    return q;
}
struct Out8 {
    uint32_t m8, r8, scale;
};
// New states of the run, q.p updated in place.
__device__ __forceinline__ Out8 run8_math(const AdamK& K, const AdamWScal& s, int64_t x, const float4& g, Run8& q) {
    const uint32_t pair = uint32_t(__builtin_amdgcn_readfirstlane(int(q.scale)));
    const float ms = pow2_of_byte(pair & 0xffu);
    float m[4], r[4];
    moment_values(q.m8, m);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        m[t] *= ms;
        r[t] = root_value((q.r8 >> (8 * t)) & 0xffu, pair >> 8);
    }
    adamw8_elem(K, s, g.x, q.p.x, m[0], r[0]);
    adamw8_elem(K, s, g.y, q.p.y, m[1], r[1]);
    adamw8_elem(K, s, g.z, q.p.z, m[2], r[2]);
    adamw8_elem(K, s, g.w, q.p.w, m[3], r[3]);
    const uint32_t mb = moment_byte(wave_max(max4_bits(m[0], m[1], m[2], m[3])));
    const uint32_t rb = root_byte(wave_max(max4_bits(r[0], r[1], r[2], r[3])));
    const float mi = inverse_of_byte(mb);
    uint32_t h[4];
    Out8 o{0, 0, mb | (rb << 8)};
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        h[t] = noise_of(s.key, x + t);
        o.r8 |= root_round(r[t], rb, root_noise(h[t])) << (8 * t);
    }
    o.m8 = moment_round<0>(m[0] * mi, moment_noise(h[0]), o.m8);
    o.m8 = moment_round<1>(m[1] * mi, moment_noise(h[1]), o.m8);
    o.m8 = moment_round<2>(m[2] * mi, moment_noise(h[2]), o.m8);
    o.m8 = moment_round<3>(m[3] * mi, moment_noise(h[3]), o.m8);
    if (mb == kScaleNan) o.m8 = 0;
    if (rb == kScaleNan) o.r8 = 0;
    return o;
}
template <int DT>
__device__ __forceinline__ void run8_store(const AdamW8Args& A, int64_t x, int64_t block, const float4& p, const Out8& o,
                                           uint16_t* lp) {
    store4f(A.p32 + x, p);
    __builtin_nontemporal_store(o.m8, gptr(reinterpret_cast<uint32_t*>(A.m8 + x)));
    __builtin_nontemporal_store(o.r8, gptr(reinterpret_cast<uint32_t*>(A.r8 + x)));
    store8(lp, pack4_fast<DT>(p));
    if (__lane_id() == 0) gptr(A.scales)[block] = uint16_t(o.scale);
}
template <int DT>
__device__ __forceinline__ void run8_step(const AdamK& K, const AdamWScal& s, const AdamW8Args& A, int64_t x,
                                          int64_t block, const float4& g, Run8 q, uint16_t* lp) {
    const Out8 o = run8_math(K, s, x, g, q);
    run8_store<DT>(A, x, block, q.p, o, lp);
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

// The lane's 4 columns of a run of a mixed tile, xr the first's place in it, x in the shard; every
// lane of the wavefront calls it (`in`: whether its columns exist; q.scale is not used).  A run
// that one parameter covers is the step above.  Else the blocks' largest magnitudes go through
// the wavefront's scratch, and only live columns are written.
template <int DT>
__device__ __forceinline__ void run8_mixed(const TileMap& M, const AdamK& K, const AdamW8Args& A, RunMax* S,
                                           int64_t first, int64_t x, int xr, bool in, const float4& g, Run8 q) {
    const int run = xr & ~int(kRun - 1), l4 = xr - run;
    const int64_t block = (x >> kRunShift) + first;
    int k = M.find(xr);
    if (M.holds(k, run) && M.end[k] >= run + kRun) {  // the same k in every lane
        const AdamWScal s = M.scalars(k);
        if (!s.live()) return;
        q.scale = gptr(A.scales)[block + k];
        run8_step<DT>(K, s, A, x, block + k, g, q, A.arena + M.row[k] + xr);
        return;
    }
    const float* gq = &g.x;
    float* pq = &q.p.x;
    int own[4], at[4];
    uint32_t pair[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        S->m[l4 + t] = 0;
        S->r[l4 + t] = 0;
        while (k < M.count && M.end[k] <= xr + t) ++k;
        const bool on = in && M.holds(k, xr + t) && M.scalars(k).live();
        own[t] = on ? k : -1;
        at[t] = on && M.begin[k] > run ? M.begin[k] - run : 0;
        pair[t] = on ? gptr(A.scales)[block + k] : 0;
    }
    wave_lds_fence();
    float m[4], r[4];
    moment_values(q.m8, m);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        if (own[t] < 0) continue;
        m[t] *= pow2_of_byte(pair[t] & 0xffu);
        r[t] = root_value((q.r8 >> (8 * t)) & 0xffu, pair[t] >> 8);
        adamw8_elem(K, M.scalars(own[t]), gq[t], pq[t], m[t], r[t]);
        atomicMax(&S->m[at[t]], abs_bits(m[t]));
        atomicMax(&S->r[at[t]], abs_bits(r[t]));
    }
    wave_lds_fence();  // also: every lane has its old scales before one is written
    uint32_t mw = 0, rw = 0;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        if (own[t] < 0) continue;
        const uint32_t mb = moment_byte(S->m[at[t]]), rb = root_byte(S->r[at[t]]);
        const uint32_t h = noise_of(M.scalars(own[t]).key, x + t);
        if (mb != kScaleNan)
            mw |= (moment_round<0>(m[t] * inverse_of_byte(mb), moment_noise(h), 0) & 0xffu) << (8 * t);
        if (rb != kScaleNan) rw |= root_round(r[t], rb, root_noise(h)) << (8 * t);
        if (l4 + t == at[t]) gptr(A.scales)[block + own[t]] = uint16_t(mb | (rb << 8));
    }
    const bool all = own[0] >= 0 && own[1] >= 0 && own[2] >= 0 && own[3] >= 0;
    if (all && M.row[own[0]] == M.row[own[3]]) {  // rows of one bucket are one
        store4f(A.p32 + x, q.p);
        *gptr(reinterpret_cast<uint32_t*>(A.m8 + x)) = mw;
        *gptr(reinterpret_cast<uint32_t*>(A.r8 + x)) = rw;
        store8(A.arena + M.row[own[0]] + xr, pack4<DT>(q.p));
    } else {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            if (own[t] < 0) continue;
            gptr(A.p32)[x + t] = pq[t];
            gptr(A.m8)[x + t] = uint8_t(mw >> (8 * t));
            gptr(A.r8)[x + t] = uint8_t(rw >> (8 * t));
            gptr(A.arena)[M.row[own[t]] + xr + t] = from_f32<DT>(pq[t]);
        }
    }
    wave_lds_fence();  // the scratch is free for the wavefront's next run
}

// Checks of a step's hyperparameters, and the prepare launch into `work` (adamw.hip).
zero_status launch_adamw_prepare(const zero_plan* plan, const uint8_t* d_live, int32_t* d_steps,
                                 const zero_adamw_hparams* hp, int32_t* d_flag, void* work, hipStream_t s,
                                 const char* who);
zero_status check_work(const void* work, const char* who);

}  // namespace zs
