"""The AdamW reference against independent values: torch's e4m3 type and its AdamW in 64 bits."""
import numpy as np
import pytest
import torch

import adamw_reference as R


def test_moment_values_are_the_ocp_e4m3_codes():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).to(torch.float64).numpy()
    finite = ~np.isnan(want)
    assert finite.sum() == 254
    assert np.array_equal(R.M_VALUES[finite], want[finite])


def test_root_values_are_increasing_with_a_relative_step_of_a_sixteenth_at_most():
    assert np.all(np.diff(R.R_VALUES) > 0) and R.R_VALUES[0] == 0 and R.R_VALUES[255] == 1.9375
    assert R.R_VALUES[1] == 2.0 ** -18
    assert np.all(np.diff(R.R_VALUES)[16:] / R.R_VALUES[16:-1] <= 1 / 16)


def test_nearest_moment_codes_are_torch_s():
    rng = np.random.default_rng(1)
    x = (rng.standard_normal(4096) * np.exp(rng.uniform(-12, 6, 4096))).astype(np.float32)
    x[:256] = R.M_VALUES[np.r_[0:127, 128:255, 1, 2]][:256] * 2.0  # exact codes
    x[256:510] = (R.M_VALUES[np.r_[0:126, 128:256]][:254] + 0).astype(np.float32)
    x = np.clip(np.nan_to_num(x), -448, 448).astype(np.float32)
    x[0] = 448.0  # the block's scale is then 1
    idx = np.zeros(4096, np.int64)
    code, byte = R.encode(x, idx, np.ones(4096, bool), 1, "m")
    assert byte[0] == 127
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(code, want)


@pytest.mark.parametrize("big,top,emax,least,want", [
    (448.0, 448.0, 8, -111, 0), (448.0001, 448.0, 8, -111, 1), (449.0, 448.0, 8, -111, 1), (256.0, 448.0, 8, -111, 0),
    (255.9, 448.0, 8, -111, 0), (224.0, 448.0, 8, -111, -1), (1.9375, 1.9375, 0, -95, 0),
    (1.94, 1.9375, 0, -95, 1), (1e-38, 448.0, 8, -111, -111)])
def test_scales(big, top, emax, least, want):
    """The least power of two under which the largest value does not pass the top code."""
    byte = R.block_bytes(np.array([big, -big / 3]), np.zeros(2, int), np.ones(2, bool), 1, top, emax, least)
    assert byte[0] - 127 == want


def test_step_is_torch_s_adamw_in_64_bits():
    rng = np.random.default_rng(2)
    p0 = rng.standard_normal(300) * 0.02
    w = torch.nn.Parameter(torch.from_numpy(p0.copy()))
    opt = torch.optim.AdamW([w], lr=1e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
    p, m, v = p0, np.zeros(300), np.zeros(300)
    for t in range(1, 6):
        g = rng.standard_normal(300) * 1e-2
        w.grad = torch.from_numpy(g)
        opt.step()
        st = R.Step(dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1), np.array([t]), 1)
        (p, m, v), _ = R.adamw64(st, np.zeros(300, int), g, p, m, v)
        assert np.allclose(p, w.detach().numpy(), rtol=1e-12, atol=1e-15)


def test_noise_halves_are_even_and_independent():
    """Means of 2^20 draws of 16 bits lie within 5 standard errors, as do the products of the two
    halves and of neighbouring columns, for several keys."""
    n = 1 << 20
    for seed, rank, t in ((0, 0, 1), (1, 0, 1), (0, 1, 1), (0, 0, 2), ((1 << 63) + 5, 1023, 20000)):
        h = R.noise(seed, rank, np.full(1, t), np.arange(n))
        lo, hi = ((h & np.uint64(0xFFFF)) + 0.5) / 65536 - 0.5, ((h >> np.uint64(16)) + 0.5) / 65536 - 0.5
        se = 1 / np.sqrt(12 * n)
        assert abs(lo.mean()) < 5 * se and abs(hi.mean()) < 5 * se
        for a, b in ((lo, hi), (lo[1:], lo[:-1]), (hi[1:], hi[:-1]), (lo[256:], lo[:-256])):
            assert abs((a * b).mean()) < 5 / (12 * np.sqrt(n))
