"""The AdamW operators at the borders of their ranges: the smallest states that 8 bits hold, a sum of
squares that another rank made infinite, parameters that are -0 or infinite, the quotient's rounding,
clipping with 8-bit states and in the fused path, many rows, states that are not numbers."""
import contextlib
import ctypes

import numpy as np
import pytest
import torch

import adamw_reference as R
import test_gpu_adamw as T
import zero_sharded_mixed_amd as Z
from gpu_harness import DEV, ragged_numels, say
from test_gpu_adamw import Case, check_parameters, close, codes, host
from zero_sharded_mixed_amd import _binding as B

pytestmark = pytest.mark.gpu


def states_of(st, bits):
    return [st.p32, st.arena, st.steps] + ([st.m8, st.r8, st.scales] if bits == 8 else [st.m, st.v])


# ----------------------------------------------------------- the smallest 8-bit states ----

def small_states(c, st, first, last):
    """Random codes (roots not zero) under root scales 2^first .. 2^last and momentum scales as far
    down; returns the decoded states."""
    n_scales = st.plan.adamw_n_scales
    rng = c.rng
    m8 = rng.integers(0, 256, c.S).astype(np.uint8)
    m8[(m8 & 127) == 127] = 5
    r8 = rng.integers(1, 256, c.S).astype(np.uint8)
    sc = np.stack([rng.integers(first + 119, last + 120, n_scales), rng.integers(first + 127, last + 128, n_scales)], 1)
    sc = sc.astype(np.uint8).reshape(-1)
    st.m8, st.r8, st.scales = (torch.from_numpy(a).to(DEV) for a in (m8, r8, sc))
    return R.decode(m8, r8, sc, c.idx), (m8, r8, sc)


def step8_small(ref, i, g32, m, r):
    """The 8-bit step's new states with fp32 roundings, on values first brought near 1 by a power of
    two each: what the formula gives where nothing leaves fp32's range."""
    f = np.float32
    g = g32.astype(f) * f(ref.mult)
    m1 = f(ref.b1) * m.astype(f) + f(1 - ref.b1) * g
    _, e = np.frexp(np.maximum(r, np.abs(g)))
    rs, gs = np.ldexp(r, -e).astype(f), np.ldexp(g.astype(np.float64), -e).astype(f)
    r1 = np.sqrt(f(ref.b2) * (rs * rs) + f(1 - ref.b2) * (gs * gs))
    return m1, np.ldexp(r1.astype(np.float64), e)


@pytest.mark.parametrize("gradient", [0.0, 1.0])
@pytest.mark.parametrize("name", ["mlp", "runs", "ragged-7", "tiny"])
def test_the_smallest_roots_are_kept(name, gradient):
    """Roots from 2^-113, the least code under the least scale, to 2^-55, whose squares leave fp32's
    range, with zero gradients and gradients of their size: codes and scales bit for bit those of the
    formula, p32 within the bounds of its roundings, with eps far below the roots."""
    c = Case(name, seed=31)
    say(f"[small roots] {name} {gradient}")
    st = c.reset(8)
    (m0, r0), (m8, r8, sc) = small_states(c, st, -95, -56)
    g = c.rng.normal(size=c.S) * r0 if gradient else np.zeros(c.S)
    st.g32 = torch.from_numpy(g.astype(np.float32)).to(DEV)
    g = host(st.g32)
    hp = c.hp(seed=5, eps=2.0 ** -126, beta2=0.999, grad_scale=1.0)
    st.adamw(hp)
    own, ref = np.maximum(c.own, 0), c.ref(hp)
    (p, _, _), (ep, _, _) = R.adamw64(ref, own, g, c.p.astype(np.float64), m0, r0 * r0, True)
    # em and ev of the bounds are relative, and m and the scaled squares stay in the normal range; eps is
    # the one addend that a root may pass by 2^70
    check_parameters(c, st, p, ep, name)
    m1, r1 = step8_small(ref, own, g, m0, r0)
    h = R.noise(5, c.rank, (c.t + c.live)[own], np.arange(c.S))
    n_scales = st.plan.adamw_n_scales
    wm, bm = R.encode(m1, c.idx, c.on, n_scales, "m", h)
    wr, br = R.encode(r1, c.idx, c.on, n_scales, "r", h)
    gm, gr, gs = codes(st)
    old = sc.reshape(-1, 2)
    assert np.array_equal(gs, np.stack([np.where(bm < 0, old[:, 0], bm), np.where(br < 0, old[:, 1], br)],
                                       1).reshape(-1).astype(np.uint8))
    assert np.array_equal(gr, np.where(c.on, wr, r8))
    assert np.array_equal(gm, np.where(c.on, wm, m8))


def test_the_smallest_roots_do_not_vanish_over_steps():
    """200 steps of zero gradients from roots of 2^-112 .. 2^-60: none becomes zero."""
    c = Case("runs", seed=32)
    st = c.reset(8)
    small_states(c, st, -95, -61)
    st.g32.fill_(0)
    for _ in range(200):
        st.adamw(c.hp(beta2=0.999))
    assert np.all(host(st.r8)[c.on] > 0)


@pytest.mark.parametrize("beta2", [0.999, 0.0])
@pytest.mark.parametrize("g", [2.0 ** -60, 2.0 ** -120, 2.0 ** -149 * 64])
def test_a_root_from_the_smallest_gradients_is_not_zero(beta2, g):
    """A first gradient whose square is zero in fp32, beside states that are zero and (with beta2 = 0)
    states that the step forgets: the root is sqrt(1 - beta2) |g| up to its rounding to a code."""
    n = 4096 + 300
    st = Z.ShardStep([n, 77], 1, 0, 0, Z.ZERO_BF16)
    if beta2 == 0.0:
        st.v.fill_(1.0)
    st.enable_adamw(8)
    st.g32.fill_(g)
    st.adamw(Z.AdamWParams(lr=0.0, beta2=beta2))
    r = st.adamw_states()[1][:n + 77].double().cpu().numpy()
    want = np.sqrt(1 - beta2) * g
    least = 2.0 ** -113
    assert np.all(r >= least) and np.all(np.abs(r - want) <= np.maximum(want / 16, least))


def test_a_nan_block_stays_nan_whatever_the_betas():
    c = Case("runs", seed=40)
    at = np.flatnonzero(c.on)[100]
    c.g[at] = np.nan
    st = c.reset(8)
    for g in (None, 0.0):
        if g is not None:
            st.g32.fill_(g)
        st.adamw(c.hp(beta1=0.0, beta2=0.0), use_flag=False)
    m, r = (host(t.float()) for t in st.adamw_states())
    hit = (c.idx == c.idx[at]) & c.on
    assert np.isnan(m[hit]).all() and np.isnan(r[hit]).all()
    assert not np.isnan(m[c.on & ~hit]).any() and not np.isnan(r[c.on & ~hit]).any()


# ---------------------------------------------- the verdict of a sum that other ranks made infinite ----

@pytest.mark.parametrize("total", [np.inf, np.nan])
@pytest.mark.parametrize("path", ["unfused", "fused"])
@pytest.mark.parametrize("bits", [32, 8])
def test_an_infinite_sum_of_all_ranks_skips_the_step_and_sets_the_flag(bits, path, total):
    """This rank's gradient is finite and its flag clear; the sum over the ranks is not.  Nothing
    changes, the flag says so (the loss scale then backs off on every rank), and the next step with a
    finite sum runs."""
    c = Case("ragged-7", seed=33)
    st = c.reset(bits)
    st.enable_loss_scaler(2.0 ** 8)
    rows = [(torch.randn(c.nd, int(b.row_stride), device=DEV).mul_(1e-2).bfloat16(), int(b.row_stride))
            for b in st.buckets]

    def step(extra):
        st.reduce(lambda b: rows[b])
        st.grad_sumsq()
        st.sumsq += extra  # the other ranks' sums
        hp = c.hp(max_norm=1.0, seed=3, grad_sumsq=st.sumsq, norm_out=st.norm_out)
        if path == "fused":
            st.reduce_adamw(lambda b: rows[b], hp)
        else:
            st.adamw(hp)

    before = [t.clone() for t in states_of(st, bits)]
    st.norm_out.fill_(-1)
    step(total)
    assert int(st.flag) == 1
    assert all(torch.equal(a, b) for a, b in zip(states_of(st, bits), before))
    assert st.norm_out.tolist() == [-1, -1]
    st.update_loss_scale()
    assert float(Z.read_loss_scaler(st.scaler).scale) == 2.0 ** 7
    st.flag.zero_()
    step(1.0)
    assert int(st.flag) == 0 and np.array_equal(host(st.steps), c.t + c.live)
    assert np.isfinite(host(st.p32)[c.on]).all()


def test_ranks_agree_on_a_skipped_step():
    """Two ranks, one with an infinite gradient in its shard: with the sums added both skip, both back
    their loss scales off, and both take the next step with the same norm."""
    n = [3000, 5001]
    ranks = [Z.ShardStep(n, 2, k, 0, Z.ZERO_FP16) for k in range(2)]
    for k, st in enumerate(ranks):
        st.enable_adamw(8 if k else 32)
        st.enable_loss_scaler(2.0 ** 10)
        st.p32.fill_(0.5)
    for turn, bad in enumerate((float("inf"), 1.0)):
        for k, st in enumerate(ranks):
            st.flag.zero_()
            st.g32.fill_(0.25 * 2.0 ** 10)
            st.g32[17] = bad if k == 0 else 1.0
            st.grad_sumsq()
        total = ranks[0].sumsq + ranks[1].sumsq
        for st in ranks:
            st.sumsq.copy_(total)
            st.adamw(Z.AdamWParams(lr=1e-3, max_norm=1.0))
        assert [int(st.flag) for st in ranks] == [1 - turn] * 2
        for st in ranks:
            st.update_loss_scale()
            assert float(Z.read_loss_scaler(st.scaler).scale) == 2.0 ** 9
            assert st.steps.tolist() == [turn, turn] and bool(torch.isfinite(st.p32).all())
            assert bool((st.p32 == 0.5).all()) == (turn == 0)
    assert torch.equal(ranks[0].norm_out, ranks[1].norm_out)


def test_a_misaligned_flag_is_refused():
    c = Case("mlp", seed=41)
    st = c.reset()
    hp = B._adamw_hp(st.plan, c.hp(), "hp")
    at = lambda t, k=0: ctypes.c_void_p(t.data_ptr() + k)  # noqa: E731
    args = [st.plan.handle, at(st.live), at(st.steps), ctypes.byref(hp)]
    assert Z.lib().zero_adamw_prepare(*args, at(st.flag, 2), at(st.work), None) == Z.ZERO_EINVAL
    assert "flag" in Z.zero_last_error()


# -------------------------------------------------------- parameters that are -0 or infinite ----

SPECIAL = np.array([-0.0, 0.0, np.inf, -np.inf, np.nan, 2.0 ** -149, -2.0 ** -149, 3e38], np.float32)


@pytest.mark.parametrize("how", ["weight_decay", "decay", "lr"])
@pytest.mark.parametrize("name", ["mlp", "ragged-7", "tiny"])
def test_without_decay_special_parameters_have_adam_s_bits(name, how):
    """-0, infinities and NaN among the parameters, half of the gradients and states zero: the bits of
    the Adam step, whether the decay is zero by the rate, the weight or the parameter's multiplier."""
    c = Case(name, seed=34)
    c.p[:] = c.rng.choice(SPECIAL, c.S)
    zero = c.rng.random(c.S) < 0.5
    c.g[zero], c.m[zero], c.v[zero] = 0, 0, 0
    lr = 0.0 if how == "lr" else 2e-3
    kw = dict(lr=lr, weight_decay=0.0 if how == "weight_decay" else 0.1)
    if how == "decay":
        kw["decay"] = torch.zeros(c.n, device=DEV)
    a = c.reset()
    a.adamw(c.hp(**kw))
    got = [a.p32, a.m, a.v, a.steps, a.arena]
    b = c.reset()
    b.adam(lr, 0.9, 0.99, 1e-8, 1.0 / c.nd)
    for x, y in zip(got, [b.p32, b.m, b.v, b.steps, b.arena]):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))


@pytest.mark.parametrize("name", ["mlp", "ragged-7", "tiny"])
def test_without_decay_special_parameters_stay_in_the_8_bit_step(name):
    """Zero gradients, zero states, no decay: p32 keeps its bits, also with decay for others."""
    c = Case(name, seed=35)
    c.p[:] = c.rng.choice(SPECIAL[[0, 1, 2, 3, 5, 6, 7]], c.S)
    c.g[:], c.m[:], c.v[:] = 0, 0, 0
    st = c.reset(8)
    st.adamw(c.hp(decay=torch.zeros(c.n, device=DEV)))
    assert np.array_equal(host(st.p32).view(np.uint32), c.p.view(np.uint32))


# ------------------------------------------------------------------ the quotient's rounding ----

def test_the_8_bit_step_s_quotient_is_the_nearest():
    """beta1 = beta2 = 0, lr = 1, p = 0: p becomes -g / (|g| + eps) with one rounding, every g = k / 4096
    (its square, its root and the sum with eps = 1/2 are exact).  The quotient k / (k + 2048) of a 12-bit
    by a 13-bit integer d stays at least 1 / (2 d) > 2^-14 of fp32's spacing away from the middle of
    two neighbours, and a residual's correction leaves an error of 2^-21 of it: the result is the
    nearest."""
    k = np.arange(1, 4096)
    g = (k / 4096).astype(np.float32)
    g[::2] *= -1
    st = Z.ShardStep([g.size], 1, 0, 0, Z.ZERO_BF16)
    st.enable_adamw(8)
    st.g32[:g.size] = torch.from_numpy(g).to(DEV)
    st.adamw(Z.AdamWParams(lr=1.0, beta1=0.0, beta2=0.0, eps=0.5))
    got = host(st.p32)[:g.size]
    want = (-g.astype(np.float64) / (np.abs(g.astype(np.float64)) + 0.5)).astype(np.float32)
    off = got.view(np.int32).astype(np.int64) - want.view(np.int32)
    assert not off.any(), f"{(off != 0).sum()} of {off.size} quotients, by up to {np.abs(off).max()} units"


def test_eps_outside_fp32_is_refused():
    st = Z.ShardStep([64], 1, 0, 0, Z.ZERO_BF16)
    st.enable_adamw()
    for eps in (1e39, 2.0 ** -127):
        with pytest.raises(Z.ZeroError, match="eps"):
            st.adamw(Z.AdamWParams(lr=1e-3, eps=eps))
    st.adamw(Z.AdamWParams(lr=1e-3, eps=3e38))
    assert not st.p32.any()


# -------------------------------------------------------- clipping, loss scale and schedule ----

@pytest.mark.parametrize("dtype", [Z.ZERO_BF16, Z.ZERO_FP16])
@pytest.mark.parametrize("max_norm", [0.0, 1e-4, 1e9])
@pytest.mark.parametrize("name", ["mlp", "ragged-7"])
def test_adamw8_under_clip_scale_and_schedule(name, max_norm, dtype):
    """The 8-bit step with a sum of squares, a loss scale and a rate factor: parameters, codes and
    scales, not the norm alone."""
    c = Case(name, dtype, seed=36)
    st = c.reset(8)
    st.enable_loss_scaler(2.0 ** 10)
    factor = torch.full((1,), 0.3, device=DEV)
    st.grad_sumsq()
    sumsq = float(st.sumsq)
    m8, r8, sc = codes(st)
    m0, r0 = R.decode(m8, r8, sc, c.idx)
    hp = c.hp(max_norm=max_norm, lr_factor=factor, grad_sumsq=st.sumsq, norm_out=st.norm_out, seed=17)
    st.adamw(hp)
    own, ref = np.maximum(c.own, 0), c.ref(hp, sumsq=sumsq, scale=2.0 ** 10, lr_factor=0.3)
    (p, _, _), (ep, _, _) = R.adamw64(ref, own, c.g, c.p.astype(np.float64), m0, r0 * r0, True)
    check_parameters(c, st, p, ep, name)
    m1, r1 = R.adamw8_f32(ref, own, c.g, m0, r0)
    h = R.noise(17, c.rank, (c.t + c.live)[own], np.arange(c.S))
    wm, bm = R.encode(m1, c.idx, c.on, st.plan.adamw_n_scales, "m", h)
    wr, br = R.encode(r1, c.idx, c.on, st.plan.adamw_n_scales, "r", h)
    old = sc.reshape(-1, 2)
    want = np.stack([np.where(bm < 0, old[:, 0], bm), np.where(br < 0, old[:, 1], br)], 1).reshape(-1)
    gm, gr, gs = codes(st)
    assert np.array_equal(gs, want.astype(np.uint8))
    assert np.array_equal(gm, np.where(c.on, wm, m8)) and np.array_equal(gr, np.where(c.on, wr, r8))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype", [Z.ZERO_BF16, Z.ZERO_FP16])
@pytest.mark.parametrize("name", ["mlp", "ragged-7", "ragged-64"])
def test_the_fused_step_takes_clip_scale_and_schedule(name, dtype, bits):
    """The unfused step forms the norm; the fused one is given the same sum: the same bits, with a
    coefficient below 1, a loss scale that changes between the steps and a rate factor."""
    c = Case(name, dtype, seed=37)
    rows = [((torch.randn(c.nd, int(b.row_stride), device=DEV) * 1e-2).to(T.TORCH16[dtype]), int(b.row_stride))
            for b in c.st.buckets]
    factor = torch.full((1,), 0.3, device=DEV)
    sums, got = [], []
    for fused in (False, True):
        st = c.reset(bits)
        st.enable_loss_scaler(2.0 ** 4, growth_interval=1)
        norms = []
        for k in range(2):
            if fused:
                hp = c.hp(seed=5, max_norm=1e-3, lr_factor=factor, grad_sumsq=sums[k], norm_out=st.norm_out)
                st.reduce_adamw(lambda b: rows[b], hp)
            else:
                st.reduce(lambda b: rows[b])
                sums.append(st.grad_sumsq().clone())
                st.adamw(c.hp(seed=5, max_norm=1e-3, lr_factor=factor))
            norms.append(st.norm_out.clone())
            st.update_loss_scale()
        assert 0 < float(norms[0][1]) < 1 and float(norms[1][0]) == float(norms[0][0]) / 2
        got.append(states_of(st, bits) + norms)
    for a, b in zip(*got):
        assert torch.equal(a, b)


# -------------------------------------------------------------------------- many rows, load ----

@contextlib.contextmanager
def layout(name, *what):
    T.LISTS[name] = what
    try:
        yield name
    finally:
        del T.LISTS[name]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype", [Z.ZERO_BF16, Z.ZERO_FP16])
@pytest.mark.parametrize("nd", [65, 100, 1024])
def test_the_fused_step_over_many_rows_has_the_same_bits(nd, dtype, bits):
    """Row counts above 64, whole tiles and tiles of several parameters, the last group of rows full
    and not."""
    rng = np.random.default_rng(nd)
    numels = [nd * 5000] + ragged_numels(rng, 60, nd, 40 * nd) + [nd * 2048 * 2]
    with layout("rows", numels, nd, nd - 1, 2 * 12000 * nd) as name:
        c = Case(name, dtype, seed=38)
    say(f"[rows] {nd} {dtype} {bits}: {c.S} columns, {len(c.st.buckets)} buckets")
    rows = []
    for b in c.st.buckets:
        stride = int(b.row_stride) + 8
        rows.append(((torch.randn(nd, stride, device=DEV) * 1e-2).to(T.TORCH16[dtype]), stride))
    got = []
    for fused in (False, True):
        st = c.reset(bits)
        if fused:
            st.reduce_adamw(lambda b: rows[b], c.hp(seed=5))
        else:
            st.reduce(lambda b: rows[b])
            st.adamw(c.hp(seed=5))
        got.append(states_of(st, bits))
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", ["mlp", "runs", "ragged-7", "tiny"])
def test_load_of_states_that_are_not_finite(name):
    """NaN and infinite states, variances below zero, -0 and fp32's subnormals: a block with a value
    that is not finite (the root of a variance below zero is NaN) has scale 255 and codes 0, the
    others the nearest codes."""
    c = Case(name, seed=39)
    hit = c.rng.random(c.S)
    for k, x in enumerate((np.nan, np.inf, -np.inf)):
        c.m[(hit > 0.002 * k) & (hit < 0.002 * k + 0.001)] = x
    for k, x in enumerate((np.nan, np.inf, -1.0, -2.0 ** -149)):
        c.v[(hit > 0.1 + 0.002 * k) & (hit < 0.101 + 0.002 * k)] = x
    for k, x in enumerate((0.0, -0.0, 2.0 ** -149, 2.0 ** -130)):
        c.v[(hit > 0.2 + 0.1 * k) & (hit < 0.25 + 0.1 * k)] = x
        c.m[(hit > 0.2 + 0.1 * k) & (hit < 0.25 + 0.1 * k)] = -x
    st = c.reset()
    n_scales = st.plan.adamw_n_scales
    m8, r8, sc = (torch.full((k,), 77, dtype=torch.uint8, device=DEV) for k in (c.S, c.S, 2 * n_scales))
    Z.zero_adamw8_load(st.plan, st.m, st.v, m8, r8, sc)
    inside = c.own >= 0
    with np.errstate(invalid="ignore"):
        root = np.sqrt(c.v)
    wm, bm = R.encode(c.m, c.idx, inside, n_scales, "m")
    wr, br = R.encode(root, c.idx, inside, n_scales, "r")
    assert (bm == 255).any() and (br == 255).any()
    want = np.stack([np.where(bm < 0, 77, bm), np.where(br < 0, 77, br)], 1).reshape(-1)
    assert np.array_equal(host(sc), want.astype(np.uint8))
    assert np.array_equal(host(m8), np.where(inside, wm, 77))
    assert np.array_equal(host(r8), np.where(inside, wr, 77))
    m16, r16 = (torch.zeros(c.S, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    Z.zero_adamw8_unload(st.plan, m8, r8, sc, m16, r16)
    bad_m, bad_r = (inside & (b[np.minimum(c.idx, n_scales - 1)] == 255) for b in (bm, br))
    assert np.array_equal(np.isnan(host(m16.float())), bad_m) and np.array_equal(np.isnan(host(r16.float())), bad_r)
