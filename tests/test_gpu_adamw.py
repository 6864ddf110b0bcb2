"""The AdamW operators (sum of squares, step with 32-bit and 8-bit states, reduce + step) on the
device, against the numpy reference in 64 bits: layouts with empty and one-element parameters,
row gaps, several buckets, dead parameters, each type, sizes from one column to past 2^32 of them;
what must stay as it was; non-finite values; captured graphs; two steps at once."""
import math

import numpy as np
import pytest
import torch

import adamw_reference as R
import oracle
import zero_sharded_mixed_amd as Z
from gpu_harness import DEV, ragged_numels, say
from zero_sharded_mixed_amd import _binding as B

pytestmark = pytest.mark.gpu

TORCH16 = {Z.ZERO_BF16: torch.bfloat16, Z.ZERO_FP16: torch.float16}
MLP = [256 * 128, 256, 256 * 256, 256, 512 * 256, 512]


def lists():
    rng = np.random.default_rng(11)
    return {
        "one": ([1], 1, 0, 0), "one-of-8": ([1], 8, 7, 0), "three": ([3, 0, 5], 2, 1, 0),
        "mlp": (MLP, 8, 3, 0), "runs": ([256, 256 * 3, 255, 257, 2048, 2049, 4096, 1, 6000], 1, 0, 0),
        "runs-2": ([2 * 2048 * 3, 2 * 513, 2 * 300, 2 * 2047, 2 * 2048], 2, 1, 6000),
        "ragged-1": (ragged_numels(rng, 300, 1, 9000), 1, 0, 30000),
        "ragged-7": (ragged_numels(rng, 400, 7, 60000), 7, 5, 50000),
        "ragged-64": (ragged_numels(rng, 500, 64, 300000), 64, 63, 0),
        "ragged-32": (ragged_numels(rng, 300, 32, 200000), 32, 9, 200000),
        "tiny": ([1] * 700 + [0] * 300 + [2] * 300 + [5000], 1, 0, 1000),
    }


LISTS = lists()
NAMES = list(LISTS)


class Case:
    """A plan, the oracle's plan of the same list, and this rank's buffers with random contents
    (the gaps too: what a call must leave alone is compared bit by bit)."""

    def __init__(self, name, dtype=Z.ZERO_BF16, seed=0, dead=0.25):
        self.numels, self.nd, self.rank, self.bucket = LISTS[name]
        self.dtype, self.name = dtype, name
        self.st = Z.ShardStep(self.numels, self.nd, self.rank, self.bucket, dtype)
        self.pl = oracle.plan(self.numels, self.nd, self.rank, self.bucket)
        self.own = R.owners(self.pl)
        self.idx = R.block_index(self.own)
        self.n, self.S = len(self.numels), self.pl.shard_len
        rng = self.rng = np.random.default_rng(seed)
        self.live = (rng.random(self.n) >= dead).astype(np.uint8)
        self.live[0] = 1
        self.on = (self.own >= 0) & (self.live[self.own] != 0)
        size = np.exp(rng.normal(size=self.n + 1) * 2)[self.own] * 1e-3
        f = np.float32
        self.g = (rng.normal(size=self.S) * size).astype(f)
        self.p = (rng.normal(size=self.S) * 0.02).astype(f)
        self.m = (rng.normal(size=self.S) * size * 0.3).astype(f)
        self.v = (size * np.exp(rng.normal(size=self.S) * 0.5)).astype(f) ** 2
        self.t = rng.integers(0, 2000, self.n).astype(np.int32)
        self.t[rng.random(self.n) < 0.3] = 0
        self.arena = rng.integers(0, 1 << 16, self.nd * self.S, dtype=np.uint16)
        self.decay = (rng.random(self.n) < 0.7).astype(f) * f(1.5)
        self.reset()

    def reset(self, bits=32):
        st = self.st
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
        st.p32, st.g32, st.steps, st.live = dev(self.p), dev(self.g), dev(self.t), dev(self.live)
        st.m, st.v = dev(self.m), dev(self.v)
        st.arena = dev(self.arena.view(np.int16))
        st.flag = torch.zeros(1, dtype=torch.int32, device=DEV)
        st.adamw_bits = 0
        st.enable_adamw(bits)
        return st

    def hp(self, **kw):
        d = dict(lr=2e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1, grad_scale=1.0 / self.nd,
                 decay=torch.from_numpy(self.decay).to(DEV))
        d.update(kw)
        return Z.AdamWParams(**d)

    def ref(self, hp, **kw):
        d = dict(lr=hp.lr, beta1=hp.beta1, beta2=hp.beta2, eps=hp.eps, weight_decay=hp.weight_decay,
                 grad_scale=hp.grad_scale, max_norm=hp.max_norm,
                 decay=None if hp.decay is None else hp.decay.cpu().numpy())
        d.update(kw)
        return R.Step(d, self.t + self.live, self.n)

    def row_of(self, arena):
        """Own rows of every bucket, as shard columns, and the rest of the arena."""
        out = np.zeros(self.S, np.uint16)
        rest = arena.copy()
        for b in range(self.pl.n_buckets):
            O, L = int(self.pl.buckets[b, oracle.B_BASE]), int(self.pl.buckets[b, oracle.B_STRIDE])
            at = self.nd * O + self.rank * L
            out[O:O + L] = arena[at:at + L]
            rest[at:at + L] = 0
        return out, rest


def host(t):
    return t.detach().cpu().numpy()


def close(got, want, far, on, what):
    err = np.abs(got.astype(np.float64) - want)
    bad = on & ~(err <= far)
    assert not bad.any(), f"{what}: {bad.sum()} off; first at {np.flatnonzero(bad)[0]}: " \
        f"{got[bad][0]!r} for {want[bad][0]!r} +- {far[bad][0]!r}"


def check_parameters(c, st, want, far, what):
    """p32 within its tolerance, the 16-bit rows the nearest to the kernel's own p32, and every
    other bit of both as before."""
    p = host(st.p32)
    close(p, want, far, c.on, what + " p32")
    assert np.array_equal(p[~c.on].view(np.uint32), c.p[~c.on].view(np.uint32)), what
    row, rest = c.row_of(host(st.arena).view(np.uint16))
    old, old_rest = c.row_of(c.arena)
    assert np.array_equal(rest, old_rest) and np.array_equal(row[~c.on], old[~c.on]), what
    assert np.array_equal(row[c.on], oracle.from_f32(p[c.on], c.dtype)), what
    assert np.array_equal(host(st.steps), c.t + c.live), what


# ------------------------------------------------------------------------- sum of squares ----

@pytest.mark.parametrize("name", NAMES)
def test_sumsq_is_the_sum_over_live_columns(name):
    """Exact squares added in double: within the count times 2^-53 of the exact sum, and the same
    bits again and with few blocks.  Dead parameters and gaps hold inf and NaN."""
    c = Case(name)
    say(f"[sumsq] {name}")
    c.g[~c.on] = np.tile(np.array([np.inf, np.nan], np.float32), c.S)[:(~c.on).sum()]
    st = c.reset()
    got = float(st.grad_sumsq())
    want = math.fsum(float(x) ** 2 for x in c.g[c.on])
    assert abs(got - want) <= want * 2.0 ** -53 * (c.on.sum() + 2)
    assert int(st.flag) == 0
    assert float(st.grad_sumsq()) == got
    with B.library(B.SMALL_GRID_LIB_PATH):
        small = Case(name)
        small.g[:] = c.g
        assert float(small.reset().grad_sumsq()) == got


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("check", [True, False])
def test_sumsq_of_a_value_that_is_not_finite_sets_the_flag(bad, check):
    c = Case("ragged-7")
    c.g[np.flatnonzero(c.on)[-1]] = bad
    st = c.reset()
    assert not math.isfinite(float(st.grad_sumsq(check=check)))
    assert int(st.flag) == int(check)


def test_sumsq_does_not_overflow_where_fp32_squares_would():
    c = Case("mlp")
    c.g[:] = 3e38
    got = float(c.reset().grad_sumsq())
    assert abs(got / (float(np.float32(3e38)) ** 2 * c.on.sum()) - 1) < 1e-11


def test_sumsq_of_nothing_is_zero():
    c = Case("mlp")
    c.live[:] = 0
    assert float(c.reset().grad_sumsq()) == 0.0
    st = Z.ShardStep([0, 0], 4, 1, 0, Z.ZERO_BF16)
    st.enable_adamw()
    st.sumsq.fill_(5)
    assert float(st.grad_sumsq()) == 0.0


# ------------------------------------------------------------------------- 32-bit states ----

@pytest.mark.parametrize("dtype", [Z.ZERO_BF16, Z.ZERO_FP16])
@pytest.mark.parametrize("name", NAMES)
def test_adamw_step(name, dtype):
    c = Case(name, dtype, seed=1)
    say(f"[adamw] {name} {dtype}")
    st, hp = c.reset(), c.hp()
    st.adamw(hp)
    (p, m, v), (ep, em, ev) = R.adamw64(c.ref(hp), np.maximum(c.own, 0), c.g, c.p.astype(np.float64),
                                        c.m.astype(np.float64), c.v.astype(np.float64))
    check_parameters(c, st, p, ep, name)
    for got, want, far, old in ((st.m, m, em, c.m), (st.v, v, ev, c.v)):
        close(host(got), want, far, c.on, name + " state")
        assert np.array_equal(host(got)[~c.on], old[~c.on])


@pytest.mark.parametrize("name", ["mlp", "ragged-7", "tiny"])
def test_without_decay_adamw_has_adam_s_bits(name):
    c = Case(name, seed=2)
    a = c.reset()
    a.adamw(c.hp(weight_decay=0.0))
    got = [a.p32, a.m, a.v, a.steps, a.arena]
    b = c.reset()
    b.adam(2e-3, 0.9, 0.99, 1e-8, 1.0 / c.nd)
    for x, y in zip(got, [b.p32, b.m, b.v, b.steps, b.arena]):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("max_norm", [0.0, 1e-4, 1e9])
def test_clip_scale_and_schedule(bits, max_norm):
    """The multiplier is grad_scale / loss scale times min(1, max_norm / (norm + 1e-6)); the rate
    takes the factor on the device; the norm and the coefficient come out in fp32 (half a unit)."""
    c = Case("ragged-7", Z.ZERO_FP16, seed=3)
    st = c.reset(bits)
    st.enable_loss_scaler(2.0 ** 10)
    factor = torch.full((1,), 0.3, device=DEV)
    st.grad_sumsq()
    sumsq = float(st.sumsq)
    hp = c.hp(max_norm=max_norm, lr_factor=factor, grad_sumsq=st.sumsq, norm_out=st.norm_out)
    st.adamw(hp)
    ref = c.ref(hp, sumsq=sumsq, scale=2.0 ** 10, lr_factor=0.3)
    norm, coef = (float(x) for x in st.norm_out)
    assert abs(norm - ref.norm) <= R.U * ref.norm * 1.001 and abs(coef - ref.coef) <= R.U * ref.coef * 1.001
    assert coef < 1.0 if max_norm == 1e-4 else coef == 1.0  # clipped, or not
    if bits == 32:
        (p, m, v), (ep, em, ev) = R.adamw64(ref, np.maximum(c.own, 0), c.g, c.p.astype(np.float64),
                                            c.m.astype(np.float64), c.v.astype(np.float64))
        check_parameters(c, st, p, ep, "clipped")
        close(host(st.m), m, em, c.on, "clipped m")
        close(host(st.v), v, ev, c.on, "clipped v")


@pytest.mark.parametrize("bits", [32, 8])
def test_a_set_flag_skips_the_step_and_a_norm_that_is_not_finite_shows_without_one(bits):
    c = Case("ragged-7", seed=4)
    c.g[np.flatnonzero(c.on)[7]] = np.inf
    st = c.reset(bits)
    names = ["p32", "steps", "arena"] + (["m8", "r8", "scales"] if bits == 8 else ["m", "v"])
    before = [getattr(st, k).clone() for k in names]
    st.norm_out.fill_(-1)
    st.grad_sumsq()
    st.adamw(c.hp(max_norm=1.0))
    assert all(torch.equal(getattr(st, k), b) for k, b in zip(names, before))
    assert st.norm_out.tolist() == [-1, -1]
    st.adamw(c.hp(max_norm=1.0), use_flag=False)
    p = host(st.p32)
    assert np.isnan(p[c.on]).all() and not np.isnan(p[~c.on]).any()


@pytest.mark.parametrize("bits", [32, 8])
def test_empty_and_all_dead_shards(bits):
    st = Z.ShardStep([0, 0], 4, 1, 0, Z.ZERO_BF16)
    st.enable_adamw(bits)
    st.adamw(Z.AdamWParams(lr=1e-3))
    assert st.steps.tolist() == [1, 1]
    c = Case("mlp")
    c.live[:] = 0
    st = c.reset(bits)
    st.adamw(c.hp())
    assert np.array_equal(host(st.p32), c.p) and np.array_equal(host(st.steps), c.t)


def test_zero_gradients_from_zero_states_leave_only_the_decay():
    """0 / (0 + eps) is zero: p shrinks by lr * weight_decay * d and nothing becomes NaN."""
    c = Case("ragged-7")
    c.g[:], c.m[:], c.v[:] = 0, 0, 0
    for bits in (32, 8):
        st, hp = c.reset(bits), c.hp()
        st.adamw(hp)
        want = c.p * (1.0 - 2e-3 * 0.1 * c.decay[np.maximum(c.own, 0)].astype(np.float64))
        close(host(st.p32), want, 2 * R.U * np.abs(c.p).astype(np.float64), c.on, "decay")


# -------------------------------------------------------------------------- 8-bit states ----

def codes(st):
    return host(st.m8), host(st.r8), host(st.scales)


@pytest.mark.parametrize("name", NAMES)
def test_load_and_unload(name):
    """Codes to the nearest with the least scales, of live and dead parameters; what they stand for
    comes back exactly; gaps stay as they were."""
    c = Case(name, seed=5)
    say(f"[load] {name}")
    c.m[c.rng.random(c.S) < 0.1] = 0
    c.m[c.rng.random(c.S) < 0.1] *= np.float32(1e-6)
    c.v[c.rng.random(c.S) < 0.1] = 0
    c.v[c.rng.random(c.S) < 0.1] *= np.float32(1e-14)
    st = c.reset()
    n_scales = st.plan.adamw_n_scales
    m8, r8, sc = (torch.full((k,), 77, dtype=torch.uint8, device=DEV) for k in (c.S, c.S, 2 * n_scales))
    Z.zero_adamw8_load(st.plan, st.m, st.v, m8, r8, sc)
    inside = c.own >= 0
    wm, bm = R.encode(c.m, c.idx, inside, n_scales, "m")
    wr, br = R.encode(np.sqrt(c.v), c.idx, inside, n_scales, "r")
    want = np.stack([np.where(bm < 0, 77, bm), np.where(br < 0, 77, br)], 1).reshape(-1)
    assert np.array_equal(host(sc), want.astype(np.uint8))
    assert np.array_equal(host(m8), np.where(inside, wm, 77))
    assert np.array_equal(host(r8), np.where(inside, wr, 77))
    assert np.all(host(r8)[inside & (c.v > 0)] > 0)
    m16, r16 = (torch.full((c.S,), 3.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    Z.zero_adamw8_unload(st.plan, m8, r8, sc, m16, r16)
    m, r = R.decode(host(m8), host(r8), host(sc), c.idx)
    assert np.array_equal(host(m16.double()), np.where(inside, m, 3.0))
    assert np.array_equal(host(r16.double()), np.where(inside, r, 3.0))


@pytest.mark.parametrize("dtype", [Z.ZERO_BF16, Z.ZERO_FP16])
@pytest.mark.parametrize("name", NAMES)
def test_adamw8_step(name, dtype):
    """From decoded states: p32 as the 64-bit step; new codes at most one code from the 64-bit value
    and bit for bit those of the formula in fp32 with the documented noise; dead parameters' codes
    and scales, gaps and unused scales as before."""
    c = Case(name, dtype, seed=6)
    say(f"[adamw8] {name} {dtype}")
    st = c.reset(8)
    n_scales = st.plan.adamw_n_scales
    gap = c.own < 0
    for t in (st.m8, st.r8):
        t[torch.from_numpy(gap).to(DEV)] = 77
    seed = 0x0123456789ABCDEF
    hp = c.hp(seed=seed)
    m8, r8, sc = codes(st)
    m0, r0 = R.decode(m8, r8, sc, c.idx)
    st.adamw(hp)
    own = np.maximum(c.own, 0)
    ref = c.ref(hp)
    (p, m, v), (ep, em, ev) = R.adamw64(ref, own, c.g, c.p.astype(np.float64), m0, r0 * r0, True)
    check_parameters(c, st, p, ep, name)
    gm, gr, gs = codes(st)
    # bit for bit
    m1, r1 = R.adamw8_f32(ref, own, c.g, m0, r0)
    h = R.noise(seed, c.rank, (c.t + c.live)[own], np.arange(c.S))
    wm, bm = R.encode(m1, c.idx, c.on, n_scales, "m", h)
    wr, br = R.encode(r1, c.idx, c.on, n_scales, "r", h)
    old = sc.reshape(-1, 2)
    want = np.stack([np.where(bm < 0, old[:, 0], bm), np.where(br < 0, old[:, 1], br)], 1).reshape(-1)
    assert np.array_equal(gs, want.astype(np.uint8))
    assert np.array_equal(gm, np.where(c.on, wm, m8))
    assert np.array_equal(gr, np.where(c.on, wr, r8))
    # and near the value in 64 bits: a code's neighbours lie within 1/8 (1/16) of it, or the smallest code
    mv, rv = R.decode(gm, gr, gs, c.idx)
    s = gs.reshape(-1, 2)[c.idx]
    close(mv, m, np.abs(m) / 8 + 2.0 ** -9 * R.scale_of(s[:, 0]) + em, c.on, "m codes")
    root = np.sqrt(v)
    close(rv, root, root / 16 + 2.0 ** -18 * R.scale_of(s[:, 1]) + ev / np.maximum(root, 1e-30), c.on, "r codes")


@pytest.mark.parametrize("name", ["mlp", "ragged-7", "ragged-64", "tiny"])
@pytest.mark.parametrize("bits", [32, 8])
def test_few_blocks_give_the_same_bits(name, bits):
    """Every block takes many tiles in turn: the loops over tiles, and a wavefront's scratch used
    run after run."""
    got = []
    for path in (B.LIB_PATH, B.SMALL_GRID_LIB_PATH):
        with B.library(path):
            c = Case(name, seed=7)
            st = c.reset(bits)
            for _ in range(2):
                st.adamw(c.hp(seed=9))
            got.append([st.p32, st.arena, st.steps] + ([st.m8, st.r8, st.scales] if bits == 8 else [st.m, st.v]))
            torch.cuda.synchronize()
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_rounding_keeps_the_mean():
    """One value of m and r in every column of a 2^20-column parameter, 1 - beta small: the mean of
    the codes' values lies within 5 standard errors of the unrounded value, and a second step count,
    rank or seed rounds differently."""
    n = 1 << 20
    st = Z.ShardStep([n], 1, 0, 0, Z.ZERO_BF16)
    st.enable_adamw(8)
    out = []
    for seed, t0 in ((1, 0), (1, 1), (2, 0)):
        st.m8.fill_(0)
        st.r8.fill_(0)
        st.scales.fill_(0)
        st.steps.fill_(t0)
        g = 0.01137
        st.g32.fill_(g)
        st.g32[::256] = 0.1  # every block's largest, so that the others lie between codes
        st.adamw(Z.AdamWParams(lr=0.0, beta1=0.9, beta2=0.999, seed=seed))
        m, r = (t.double().view(-1, 256)[:, 1:].reshape(-1) for t in st.adamw_states())
        out.append((m, r))
        for x, want in ((m, (1 - 0.9) * g), (r, math.sqrt(1 - 0.999) * g)):
            assert x.unique().numel() == 2
            lo, hi = x.min().item(), x.max().item()
            assert lo <= want <= hi
            share = (want - lo) / (hi - lo)
            se = (hi - lo) * math.sqrt(share * (1 - share) / x.numel()) + (hi - lo) * 2.0 ** -16 + want * 4 * R.U
            assert abs(x.mean().item() - want) < 5 * se
    assert not torch.equal(out[0][0], out[1][0]) and not torch.equal(out[0][0], out[2][0])


def test_a_moving_average_of_codes_follows_its_input():
    """beta2 = 0.999 moves r by a few hundredths of a percent a step, far below half a code: rounded
    to the nearest it would stay.  From a root 8 times too large, 3000 steps of a constant gradient
    bring v to g^2 (1 + 63 * 0.999^3000) = 4.13 g^2.  Rounding keeps r's mean and so adds r's variance
    to v's: a step moves r by at most 5e-4 of it, up with chance p = 5e-4 / d by a code of relative
    size d <= 1/16, which adds at most p d^2 = 3.2e-5 of v a step, 10% of it in 3000 steps; the mean
    over 65536 columns is held to a quarter."""
    n = 1 << 16
    st = Z.ShardStep([n], 1, 0, 0, Z.ZERO_BF16)
    st.m.fill_(0)
    g = 0.01
    st.v.fill_((8 * g) ** 2)
    st.enable_adamw(8)
    st.g32.fill_(g)
    hp = Z.AdamWParams(lr=0.0, beta1=0.9, beta2=0.999, seed=3)
    for _ in range(3000):
        st.adamw(hp)
    m, r = st.adamw_states()
    v = r.double().square().mean().item() / g ** 2
    assert abs(v / (1 + 63 * 0.999 ** 3000) - 1) < 0.25, v
    assert abs(m.double().mean().item() / g - 1) < 0.01


def test_a_root_above_zero_never_becomes_zero():
    c = Case("ragged-7", seed=8)
    c.v[:] = np.where(c.rng.random(c.S) < 0.5, 1e-30, 1.0)
    c.g[:] = 0
    st = c.reset(8)
    for _ in range(3):
        st.adamw(c.hp())
    assert np.all(host(st.r8)[c.on] > 0)


@pytest.mark.parametrize("name", ["mlp", "runs", "tiny"])
def test_a_block_that_is_not_finite_reads_as_nan_and_no_other_does(name):
    c = Case(name, seed=9)
    at = np.flatnonzero(c.on)[c.on.sum() // 2]
    c.g[at] = np.inf
    st = c.reset(8)
    st.adamw(c.hp(), use_flag=False)
    m, r = (host(t.double()) for t in st.adamw_states())
    hit = (c.idx == c.idx[at]) & (c.own >= 0)
    assert np.isnan(m[hit]).all() and np.isnan(r[hit]).all()
    rest = (c.own >= 0) & ~hit
    assert np.isfinite(m[rest]).all() and np.isfinite(r[rest]).all()


# ----------------------------------------------------------------------------- fused path ----

@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype", [Z.ZERO_BF16, Z.ZERO_FP16])
@pytest.mark.parametrize("name", NAMES)
def test_reduce_and_step_in_one_pass_has_the_same_bits(name, dtype, bits):
    """zero_reduce_shard, then the step, against the fused launches on the same rows, over two
    steps; rows of a stride of their own."""
    c = Case(name, dtype, seed=10)
    say(f"[fused] {name} {dtype} {bits}")
    rows = []
    for b in c.st.buckets:
        stride = int(b.row_stride) + 24
        x = torch.randn(c.nd, stride, device=DEV) * 1e-2
        rows.append((x.to(TORCH16[dtype]), stride))
    got = []
    for fused in (False, True):
        st = c.reset(bits)
        for k in range(2):
            if fused:
                st.g32.fill_(float("nan"))
                st.reduce_adamw(lambda b: rows[b], c.hp(seed=5))
            else:
                st.reduce(lambda b: rows[b])
                st.adamw(c.hp(seed=5))
        got.append([st.p32, st.arena, st.steps] + ([st.m8, st.r8, st.scales] if bits == 8 else [st.m, st.v]))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    # few blocks, and a set flag
    with B.library(B.SMALL_GRID_LIB_PATH):
        c2 = Case(name, dtype, seed=10)
        st = c2.reset(bits)
        for k in range(2):
            st.reduce_adamw(lambda b: rows[b], c2.hp(seed=5))
        again = [st.p32, st.arena, st.steps] + ([st.m8, st.r8, st.scales] if bits == 8 else [st.m, st.v])
        for a, b in zip(got[0], again):
            assert torch.equal(a, b)
        before = [t.clone() for t in again]
        st.flag.fill_(1)
        st.reduce_adamw(lambda b: rows[b], c2.hp(seed=5))
        assert all(torch.equal(a, b) for a, b in zip(before, again))


# -------------------------------------------------------------------- together, as used ----

@pytest.mark.parametrize("bits", [32, 8])
def test_a_run_of_steps_as_a_program_takes_them(bits):
    """pack -> reduce -> sum of squares -> clipped step -> loss scale -> unpack, 4 steps (one of
    them with an overflow, skipped), each against the reference from the state before it."""
    c = Case("ragged-7", Z.ZERO_FP16, seed=12, dead=0.2)
    st = c.reset(bits)
    st.enable_loss_scaler(2.0 ** 8, growth_interval=2)
    params = [torch.zeros(n, dtype=torch.float16, device=DEV) for n in c.numels]
    own = np.maximum(c.own, 0)
    for k in range(4):
        scale = float(Z.read_loss_scaler(st.scaler).scale)
        grads = [torch.randn(n, device=DEV).mul_(1e-2 * scale).half() for n in c.numels]
        if k == 2:
            i = int(np.flatnonzero((c.live != 0) & (np.array(c.numels) > 7 * c.nd))[0])
            grads[i].fill_(float("inf"))
        st.flag.zero_()
        st.pack(Z.ptr_table([g if on else None for g, on in zip(grads, c.live)]))
        L = [int(b.row_stride) for b in st.buckets]
        st.reduce(lambda b: (st.own_row(st.packed, b).repeat(c.nd), L[b]))  # every rank sends the same row
        before = {a: host(getattr(st, a)).copy() for a in ("p32", "steps", "g32")}
        if bits == 8:
            m0, r0 = R.decode(*codes(st), c.idx)
            v0 = r0 * r0
        else:
            m0, v0 = host(st.m).astype(np.float64), host(st.v).astype(np.float64)
        st.grad_sumsq()
        hp = c.hp(max_norm=0.5, seed=21)
        st.adamw(hp)
        if k == 2:
            assert int(st.flag) == 1 and np.array_equal(host(st.p32), before["p32"])
            assert np.array_equal(host(st.steps), before["steps"])
        else:
            ref = R.Step(dict(lr=hp.lr, beta1=hp.beta1, beta2=hp.beta2, eps=hp.eps, weight_decay=hp.weight_decay,
                              grad_scale=hp.grad_scale, max_norm=hp.max_norm, decay=c.decay, scale=scale,
                              sumsq=math.fsum(float(x) ** 2 for x in before["g32"][c.on])),
                         before["steps"] + c.live, c.n)
            (p, _, _), (ep, _, _) = R.adamw64(ref, own, before["g32"], before["p32"].astype(np.float64), m0, v0,
                                           bits == 8)
            close(host(st.p32), p, ep, c.on, f"step {k}")
            assert abs(float(st.norm_out[1]) - ref.coef) <= 2 * R.U * ref.coef
        st.update_loss_scale()
        st.unpack(Z.ptr_table(params))
    assert int(Z.read_loss_scaler(st.scaler).overflows) == 1
    assert host(st.steps)[c.live != 0].tolist() == (c.t[c.live != 0] + 3).tolist()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("path", ["unfused", "fused"])
def test_a_captured_step_replays_like_eager_steps(bits, path):
    """The whole step in a graph, the rate's factor changed between replays, with eager work and
    synchronisation between them."""
    c = Case("ragged-7", seed=13)
    factor = torch.ones(1, device=DEV)
    rows = [(torch.randn(c.nd, int(b.row_stride), device=DEV).mul_(1e-2).bfloat16(), int(b.row_stride))
            for b in c.st.buckets]
    hp = c.hp(seed=4, lr_factor=factor, max_norm=0.0 if path == "fused" else 0.1)

    def step(st):
        st.flag.zero_()
        if path == "fused":
            st.reduce_adamw(lambda b: rows[b], hp)
        else:
            st.reduce(lambda b: rows[b])
            st.grad_sumsq()
            st.adamw(hp)

    def state(st):
        return [st.p32, st.steps, st.arena] + ([st.m8, st.r8, st.scales] if bits == 8 else [st.m, st.v])

    st = c.reset(bits)
    eager = []
    for k in range(4):
        factor.fill_(1.0 / (k + 1))
        step(st)
        eager.append([t.clone() for t in state(st)])
    st = c.reset(bits)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(st)
    for k in range(4):
        factor.fill_(1.0 / (k + 1))
        graph.replay()
        torch.cuda.synchronize()
        _ = (st.p32 * 2).sum().item()
        assert all(torch.equal(a, b) for a, b in zip(state(st), eager[k])), k


def test_two_steps_of_one_plan_at_once():
    """Two states with workspaces of their own on one plan, stepped on two streams without waiting
    for each other, give the bits that each gives alone."""
    c = Case("ragged-64", seed=14)
    st = c.reset(8)
    plan, hps = st.plan, [c.hp(seed=1, lr=1e-3), c.hp(seed=2, lr=5e-3, beta2=0.9)]

    def fresh():
        return dict(p32=st.p32.clone(), m8=st.m8.clone(), r8=st.r8.clone(), scales=st.scales.clone(),
                    steps=st.steps.clone(), arena=st.arena.clone(), work=torch.zeros_like(st.work),
                    sumsq=torch.zeros_like(st.sumsq))

    def go(s, hp, stream=None):
        for _ in range(5):
            Z.zero_grad_sumsq(plan, st.g32, st.live, s["sumsq"], s["work"], stream=stream)
            Z.zero_adamw8_step(plan, st.g32, s["p32"], s["m8"], s["r8"], s["scales"], st.live, s["steps"], hp, None,
                               s["arena"], s["work"], stream=stream)

    alone = []
    for hp in hps:
        s = fresh()
        go(s, hp)
        torch.cuda.synchronize()
        alone.append(s)
    both, streams = [fresh(), fresh()], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for s, hp, stream in zip(both, hps, streams):
        go(s, hp, stream)
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        for k in ("p32", "m8", "r8", "scales", "steps", "arena", "sumsq"):
            assert torch.equal(a[k], b[k]), k


def test_a_shard_of_many_tiles():
    """13,000 tiles: more than the sum has parts, and the size from which the 32-bit step limits its
    blocks per CU; checked at 200,000 columns and against the sum of the squares in double."""
    n0, n1 = 13000 * 2048 + 777, 5003
    plan = Z.zero_plan_create([n0, n1], 1, 0, 0, Z.ZERO_BF16)
    S = plan.shard_numel
    say(f"[many tiles] {S} columns")
    gen = torch.Generator(device=DEV)
    gen.manual_seed(19)
    rnd = lambda k: torch.randn(S, generator=gen, device=DEV) * k  # noqa: E731
    g, p, m, v = rnd(1e-2), rnd(2e-2), rnd(3e-3), rnd(1e-2).square()
    old = [x.clone() for x in (p, m, v)]
    live, steps = torch.ones(2, dtype=torch.uint8, device=DEV), torch.full((2,), 41, dtype=torch.int32, device=DEV)
    work = torch.zeros(plan.adamw_work_bytes, dtype=torch.uint8, device=DEV)
    arena, sumsq = torch.zeros(S, dtype=torch.bfloat16, device=DEV), torch.zeros(1, dtype=torch.float64, device=DEV)
    Z.zero_grad_sumsq(plan, g, live, sumsq, work)
    inside = (g[:n0 + n1].double() ** 2).sum().item()
    assert abs(float(sumsq) / inside - 1) <= 2.0 ** -53 * S
    hp = Z.AdamWParams(lr=1e-3, beta2=0.95, weight_decay=0.1, max_norm=0.5, grad_sumsq=sumsq)
    Z.zero_adamw_step(plan, g, p, m, v, live, steps, hp, None, arena, work)
    cols = np.unique(np.random.default_rng(20).integers(0, n0 + n1, 200000))
    at = torch.from_numpy(cols).to(DEV)
    pick = lambda t: host(t[at]).astype(np.float64)  # noqa: E731
    ref = R.Step(dict(lr=1e-3, beta2=0.95, weight_decay=0.1, max_norm=0.5, sumsq=float(sumsq)), np.array([42, 42]), 2)
    want, far = R.adamw64(ref, (cols >= n0).astype(np.int64), host(g[at]), *[pick(x) for x in old])
    for name, got, w, e in zip("pmv", (p, m, v), want, far):
        close(host(got[at]), w, e, np.ones(cols.size, bool), name)
    assert torch.equal(arena[:n0 + n1], p[:n0 + n1].bfloat16())


@pytest.mark.timeout(300)
def test_columns_past_two_to_the_32():
    """One parameter of 2^32 + 5003 elements and a short one behind it at nd = 1: the step and the
    sum over columns whose index needs more than 32 bits, checked at both ends."""
    n0, n1 = (1 << 32) + 5003, 700
    plan = Z.zero_plan_create([n0, n1], 1, 0, 0, Z.ZERO_BF16)
    S = plan.shard_numel
    dev = dict(device=DEV)
    u8 = dict(dtype=torch.uint8, device=DEV)
    sizes = Z.zero_adamw_get_sizes(plan)
    say(f"[past 2^32] {S} columns")
    g, p = torch.zeros(S, **dev), torch.zeros(S, **dev)
    m8, r8, sc = torch.zeros(S, **u8), torch.zeros(S, **u8), torch.zeros(2 * sizes.n_scales, **u8)
    arena, work = torch.zeros(S, dtype=torch.bfloat16, device=DEV), torch.zeros(sizes.work_bytes, **u8)
    live, steps = torch.ones(2, **u8), torch.zeros(2, dtype=torch.int32, device=DEV)
    sumsq = torch.zeros(1, dtype=torch.float64, device=DEV)
    k = 9000
    rng = np.random.default_rng(15)
    gh = [(rng.normal(size=k) * 1e-2).astype(np.float32) for _ in range(2)]
    lo = [0, n0 + n1 - k]
    for a, x in zip(lo, gh):
        g[a:a + k] = torch.from_numpy(x).to(DEV)
    hp = Z.AdamWParams(lr=1e-3, beta2=0.99, seed=77, weight_decay=0.1)
    Z.zero_grad_sumsq(plan, g, live, sumsq, work)
    want = sum(math.fsum(float(x) ** 2 for x in a) for a in gh)
    assert abs(float(sumsq) / want - 1) < 1e-12
    Z.zero_adamw8_step(plan, g, p, m8, r8, sc, live, steps, hp, None, arena, work)
    assert steps.tolist() == [1, 1]
    scales = sc.view(-1, 2)
    for a, x in zip(lo, gh):
        cols = np.arange(a, a + k)
        own = (cols >= n0).astype(np.int64)
        first = (a >> 8)
        idx = (cols >> 8) + own - first
        ref = R.Step(dict(lr=1e-3, beta2=0.99, weight_decay=0.1), np.array([1, 1]), 2)
        m1, r1 = R.adamw8_f32(ref, own, x, np.zeros(k), np.zeros(k))
        h = R.noise(77, 0, np.array([1, 1])[own], cols)
        # blocks that the sample cuts hold zeros besides
        wm, bm = R.encode(m1, idx, np.ones(k, bool), int(idx.max()) + 1, "m", h)
        wr, br = R.encode(r1, idx, np.ones(k, bool), int(idx.max()) + 1, "r", h)
        assert np.array_equal(host(m8[a:a + k]), wm) and np.array_equal(host(r8[a:a + k]), wr)
        got = host(scales[first:first + idx.max() + 1])
        used = np.unique(idx)
        assert np.array_equal(got[used], np.stack([bm, br], 1)[used])
        (pw, _, _), (ep, _, _) = R.adamw64(ref, own, x, np.zeros(k), np.zeros(k), np.zeros(k), True)
        close(host(p[a:a + k]), pw, ep, np.ones(k, bool), "p32")
    mid = slice(1 << 31, (1 << 31) + 100000)
    assert not p[mid].any() and not m8[mid].any()


# ------------------------------------------------------------------------------- refusals ----

def test_refused_calls_change_nothing():
    c = Case("mlp", seed=16)
    st = c.reset()
    before = [t.clone() for t in (st.p32, st.m, st.v, st.steps, st.arena)]
    for bad in (dict(lr=-1.0), dict(lr=float("nan")), dict(beta1=1.0), dict(beta2=-0.1), dict(eps=0.0),
                dict(eps=1e-60), dict(eps=1e-39), dict(eps=float("inf")), dict(weight_decay=-0.1), dict(weight_decay=float("inf")),
                dict(grad_scale=float("nan")), dict(max_norm=-1.0), dict(max_norm=float("nan"))):
        with pytest.raises(Z.ZeroError) as e:
            st.adamw(c.hp(**bad))
        assert e.value.status == Z.ZERO_EINVAL, bad
    with pytest.raises(Z.ZeroError, match="grad_sumsq"):
        Z.zero_adamw_step(st.plan, st.g32, st.p32, st.m, st.v, st.live, st.steps, c.hp(max_norm=1.0), None, st.arena,
                          st.work)
    with pytest.raises(Z.ZeroError, match="aligned"):
        Z.zero_adamw_step(st.plan, st.g32, st.p32, st.m, st.v, st.live, st.steps, c.hp(), None, st.arena,
                          torch.zeros(st.work.numel() + 8, dtype=torch.uint8, device=DEV)[8:])
    wide = torch.zeros(c.S + 4, device=DEV)
    with pytest.raises(Z.ZeroError, match="aligned"):
        Z.zero_grad_sumsq(st.plan, wide[1:c.S + 1], st.live, st.sumsq, st.work)
    with pytest.raises(Z.ZeroError, match="out of range"):
        Z.zero_reduce_adamw_bucket(st.plan, 1, st.packed, 8, st.live, st.p32, st.m, st.v, None, st.arena, st.work)
    with pytest.raises(Z.ZeroError, match="row_stride"):
        L = int(st.buckets[0].row_stride)
        Z.zero_reduce_adamw_bucket(st.plan, 0, st.packed, L - 8, st.live, st.p32, st.m, st.v, None, st.arena, st.work)
    with pytest.raises(ValueError, match="grad_sumsq"):
        st.reduce_adamw(lambda b: (st.packed, int(st.buckets[b].row_stride)), c.hp(max_norm=1.0))
    with pytest.raises(ValueError, match="8-bit"):
        st.adamw_states()
    with pytest.raises(ValueError):
        st.enable_adamw(16)
    fresh = Z.ShardStep(MLP, 8, 3, 0, Z.ZERO_BF16)
    for call in (fresh.grad_sumsq, lambda: fresh.adamw(c.hp())):
        with pytest.raises(ValueError, match="enable_adamw"):
            call()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(before, (st.p32, st.m, st.v, st.steps, st.arena)))
    st.enable_adamw(8)
    with pytest.raises(ValueError, match="not converted back"):
        st.enable_adamw(32)
    with pytest.raises(Z.ZeroError):
        st.adam(1e-3, 0.9, 0.999, 1e-8, 1.0)  # the 32-bit states are gone
