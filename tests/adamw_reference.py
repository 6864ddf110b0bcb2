"""The AdamW operators in numpy, from their definition: 64 bits throughout, and for the 8-bit codes,
which a value next to a border decides, also the formula's own fp32 roundings one by one.  Works on
the oracle's plan (its parameters' places in the shard)."""
from __future__ import annotations

import numpy as np

import oracle

U = 2.0 ** -24  # half a unit in the last place of fp32, relative
RUN = 256


def owners(pl) -> np.ndarray:
    """Parameter of every shard column, -1 in the row gaps."""
    own = np.full(pl.shard_len, -1, np.int64)
    for i in range(pl.n):
        o, s = int(pl.params[i, oracle.P_OFFSET]), int(pl.params[i, oracle.P_SHARD])
        own[o:o + s] = i
    return own


def block_index(own: np.ndarray, first: int = 0) -> np.ndarray:
    return ((np.arange(own.size) + first) >> 8) + np.maximum(own, 0)


# ---------------------------------------------------------------------- 8-bit formats ----

M_VALUES = np.array([(f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)) for e in range(16)
                     for f in range(8)])
M_VALUES = np.concatenate([M_VALUES, -M_VALUES])
R_VALUES = np.array([(f / 16 * 2.0 ** -14 if e == 0 else (1 + f / 16) * 2.0 ** (e - 15)) for e in range(16)
                     for f in range(16)])


def scale_of(byte: np.ndarray) -> np.ndarray:
    b = byte.astype(np.int64)
    return np.where(b == 255, np.nan, np.ldexp(1.0, b - 127))


def decode(m8, r8, scales, idx):
    """(m, r) in 64 bits."""
    s = scales.reshape(-1, 2)
    return M_VALUES[m8] * scale_of(s[idx, 0]), R_VALUES[r8] * scale_of(s[idx, 1])


def block_bytes(x: np.ndarray, idx: np.ndarray, on: np.ndarray, n_scales: int, top: float, emax: int, least: int):
    """Scale byte of every block (-1: a block without a column that is on): the least power of two
    under which the largest |x| is at most `top`, but at least 2^least; 255 if a value is not finite."""
    big = np.full(n_scales, -1.0)
    with np.errstate(invalid="ignore"):
        np.maximum.at(big, idx[on], np.where(np.isfinite(x[on]), np.abs(x[on]), np.inf))
    mant, e = np.frexp(np.where(np.isfinite(big) & (big > 0), big, 1.0))  # big = 2 mant * 2^(e - 1)
    e = np.where(2 * mant > top / 2.0 ** emax, e, e - 1) - emax
    byte = np.where(big > 0, np.maximum(e, least), least) + 127
    byte = np.where(np.isinf(big), 255, byte)
    return np.where(big < 0, -1, byte)


def split(x: np.ndarray, scale: np.ndarray, values: np.ndarray):
    """For |x| / scale: the code below (or at) it, and the share of the way to the next code."""
    t = np.abs(x.astype(np.float64)) / scale
    k = np.searchsorted(values, t, side="right") - 1
    hi = np.minimum(k + 1, values.size - 1)
    gap = values[hi] - values[k]
    return k, np.where(gap > 0, (t - values[k]) / np.where(gap > 0, gap, 1), 0.0)


def mix32(h: np.ndarray) -> np.ndarray:
    h = (np.asarray(h, np.uint64) * np.uint64(0x9E3779B9)) & np.uint64(0xFFFFFFFF)
    h ^= h >> np.uint64(15)
    h = (h * np.uint64(0xB504F333)) & np.uint64(0xFFFFFFFF)
    return h ^ (h >> np.uint64(16))


def noise(seed: int, rank: int, t: np.ndarray, x: np.ndarray) -> np.ndarray:
    k = mix32(rank ^ 0xBB67AE85)
    k = mix32(k ^ np.uint64(seed & 0xFFFFFFFF))
    k = mix32(k ^ np.uint64(seed >> 32))
    key = mix32(np.asarray(t, np.uint64) ^ k)
    x = np.asarray(x, np.uint64)
    high = ((x >> np.uint64(32)) * np.uint64(0xBB67AE85)) & np.uint64(0xFFFFFFFF)
    return mix32((x & np.uint64(0xFFFFFFFF)) ^ key ^ high)


def encode(x, idx, on, n_scales, kind, h=None):
    """(codes, scale bytes) of fp32 values; h None: to the nearest, ties to the even code."""
    top, emax, least, values, bits = (448.0, 8, -111, M_VALUES[:127], 20) if kind == "m" else \
        (1.9375, 0, -95, R_VALUES, 19)
    byte = block_bytes(x, idx, on, n_scales, top, emax, least)
    b = np.where(byte < 0, 127, byte)[idx]
    bad = b == 255
    k, share = split(np.where(bad | ~np.isfinite(x), 0, x), np.ldexp(1.0, np.where(bad, 0, b - 127)), values)
    if h is None:
        up = (share > 0.5) | ((share == 0.5) & (k % 2 == 1))
    else:
        # a share has `bits` bits below the code, more only among the code's subnormals, where r's is
        # rounded to that many first
        part = share * 2.0 ** bits if kind == "m" else np.rint(share * 2.0 ** bits)
        r = (((h & np.uint64(0xFFFF)).astype(np.int64) << 4) + 8) if kind == "m" else \
            (((h >> np.uint64(16)).astype(np.int64) << 3) + 4)
        up = part + r >= 1 << bits
    c = k + up
    if kind == "m":
        c = c | np.where(np.signbit(x), 128, 0)
    else:
        c = np.where((c == 0) & (x > 0), 1, c)
    return np.where(bad, 0, c).astype(np.uint8), byte


# --------------------------------------------------------------------------- the step ----

class Step:
    """One step's scalars, per parameter, in 64 bits.  t: step counts after the increment."""

    def __init__(self, hp: dict, t: np.ndarray, n: int):
        g = lambda k, d=None: hp.get(k, d)  # noqa: E731
        self.b1, self.b2, self.eps = g("beta1", 0.9), g("beta2", 0.999), g("eps", 1e-8)
        mult = g("grad_scale", 1.0) / g("scale", 1.0)
        self.norm, self.coef = None, 1.0
        if g("sumsq") is not None:
            self.norm = np.sqrt(hp["sumsq"]) * abs(mult)
            self.coef = min(1.0, hp["max_norm"] / (self.norm + 1e-6)) if g("max_norm", 0.0) > 0 else 1.0
        self.mult = mult * self.coef
        lr = hp["lr"] * float(np.float32(g("lr_factor", 1.0)))
        t = np.maximum(t, 1).astype(np.float64)
        self.step = lr / (1 - self.b1 ** t)
        self.rbc2 = 1 / np.sqrt(1 - self.b2 ** t)
        d = np.ones(n) if g("decay") is None else np.asarray(g("decay"), np.float64)
        self.shrink = lr * g("weight_decay", 0.0) * d


def adamw64(st: Step, i, g32, p, m, v, estimates=False):
    """New (p, m, v) of columns whose parameters are i, in 64 bits, and how far fp32 may be off each:
    every operation rounds by at most U relative, and a scalar rounded once carries U.  estimates (the
    8-bit step): the root and the reciprocal may be off by a unit in the last place, 2 U, and the
    quotient is a product besides."""
    unit = 2 if estimates else 1
    with np.errstate(all="ignore"):
        g = g32.astype(np.float64) * st.mult                      # the scalar, the product: 2 U
        bm, cg = st.b1 * m, (1 - st.b1) * g
        m1 = bm + cg
        em = U * (2 * abs(bm) + 4 * abs(cg) + abs(m1))            # beta U + product U; g 2 U, 1-beta U, product U; sum U
        bv, cg2 = st.b2 * v, (1 - st.b2) * g * g
        v1 = bv + cg2
        ev = U * (2 * bv + 7 * cg2 + v1)                          # g^2: 2 * 2 U + U; 1-beta U, product U; sum U
        root = np.sqrt(v1)
        er = ev / (2 * np.where(root > 0, root, 1)) + unit * U * root
        den = root * st.rbc2[i] + st.eps
        ed = er * st.rbc2[i] + U * (2 * root * st.rbc2[i] + st.eps + den)
        up = st.step[i] * m1 / den
        quotient = 3 if estimates else 1                          # reciprocal 2 U and product U, or U
        eu = st.step[i] * em / den + abs(up) * (ed / den + (quotient + 2) * U)  # and step U, product U
        sh = st.shrink[i] * p
        p1 = p - sh - up
        ep = 2 * U * abs(sh) + eu + U * (abs(p - sh) + abs(p1))
    tiny = 2.0 ** -140  # a few units of fp32's subnormals, where relative bounds end
    k = 1.0 + 2.0 ** -12  # products of several roundings
    return (p1, m1, v1), (k * ep + tiny, k * em + tiny, k * ev + tiny)


def adamw8_f32(st: Step, i, g32, m, r):
    """New (m, r) of an 8-bit step with the formula's roundings to fp32, one by one."""
    f = np.float32
    with np.errstate(all="ignore"):
        g = g32.astype(f) * f(st.mult)
        m1 = f(st.b1) * m.astype(f) + f(1 - st.b1) * g
        r = r.astype(f)
        r1 = np.sqrt(f(st.b2) * (r * r) + f(1 - st.b2) * (g * g))
    return m1, r1
