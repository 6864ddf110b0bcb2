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
