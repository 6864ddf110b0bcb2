"""Argument checks of the AdamW entry points on the CPU: nothing here reaches a device."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from test_binding_checks import FakePlan, FakeTensor
from zero_sharded_mixed_amd import _binding as B

INC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")


class Plan(FakePlan):
    adamw_work_bytes, adamw_n_scales = 17000, 6
    handle = None


P, S = Plan(), FakePlan.shard_numel
F, I, U, D = torch.float32, torch.int32, torch.uint8, torch.float64


def good():
    t = FakeTensor
    return dict(g32=t(S, F), p32=t(S, F), m=t(S, F), v=t(S, F), m8=t(S, U), r8=t(S, U), scales=t(12, U), live=t(3, U),
                steps=t(3, I), flag=t(1, I), arena=t(8 * S), work=t(17000, U), sumsq=t(1, D), rows=t(8 * S),
                m16=t(S, torch.bfloat16), r16=t(S, torch.bfloat16))


CALLS = {
    "zero_grad_sumsq": lambda a, hp: B.zero_grad_sumsq(P, a["g32"], a["live"], a["sumsq"], a["work"], a["flag"], 0),
    "zero_adamw_prepare": lambda a, hp: B.zero_adamw_prepare(P, a["live"], a["steps"], hp, a["flag"], a["work"], 0),
    "zero_adamw_step": lambda a, hp: B.zero_adamw_step(P, a["g32"], a["p32"], a["m"], a["v"], a["live"], a["steps"],
                                                       hp, a["flag"], a["arena"], a["work"], 0),
    "zero_adamw8_step": lambda a, hp: B.zero_adamw8_step(P, a["g32"], a["p32"], a["m8"], a["r8"], a["scales"],
                                                         a["live"], a["steps"], hp, a["flag"], a["arena"], a["work"],
                                                         0),
    "zero_adamw8_load": lambda a, hp: B.zero_adamw8_load(P, a["m"], a["v"], a["m8"], a["r8"], a["scales"], 0),
    "zero_adamw8_unload": lambda a, hp: B.zero_adamw8_unload(P, a["m8"], a["r8"], a["scales"], a["m16"], a["r16"], 0),
    "zero_reduce_adamw_bucket": lambda a, hp: B.zero_reduce_adamw_bucket(
        P, 0, a["rows"], S, a["live"], a["p32"], a["m"], a["v"], a["flag"], a["arena"], a["work"], 0),
    "zero_reduce_adamw8_bucket": lambda a, hp: B.zero_reduce_adamw8_bucket(
        P, 0, a["rows"], S, a["live"], a["p32"], a["m8"], a["r8"], a["scales"], a["flag"], a["arena"], a["work"], 0),
}
USES = {
    "zero_grad_sumsq": "g32 live sumsq work flag", "zero_adamw_prepare": "live steps flag work",
    "zero_adamw_step": "g32 p32 m v live steps flag arena work",
    "zero_adamw8_step": "g32 p32 m8 r8 scales live steps flag arena work", "zero_adamw8_load": "m v m8 r8 scales",
    "zero_adamw8_unload": "m8 r8 scales m16 r16", "zero_reduce_adamw_bucket": "rows live p32 m v flag arena work",
    "zero_reduce_adamw8_bucket": "rows live p32 m8 r8 scales flag arena work",
}


@pytest.fixture
def called(monkeypatch):
    """The library's functions replaced by one that counts its calls and reports success."""
    count = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: count.append(name) or 0
    monkeypatch.setattr(B, "_lib", Lib())
    return count


@pytest.mark.parametrize("name", list(CALLS))
def test_good_arguments_reach_the_library_once(name, called):
    CALLS[name](good(), B.AdamWParams(lr=1e-3))
    assert called == [name]


@pytest.mark.parametrize("name,arg", [(n, a) for n, u in USES.items() for a in u.split()])
def test_every_buffer_is_checked_before_the_library_is_called(name, arg, called):
    ok = good()[arg]
    wrong_type = {F: torch.float16, I: torch.int64, U: torch.float32, D: torch.float32, torch.int16: torch.int32,
                  torch.bfloat16: torch.float16}[ok.dtype]
    for bad in (FakeTensor(ok.numel() - 1, ok.dtype), FakeTensor(ok.numel(), wrong_type),
                FakeTensor(ok.numel(), ok.dtype, device=None), FakeTensor(ok.numel(), ok.dtype, device=1),
                FakeTensor(ok.numel(), ok.dtype, contiguous=False)):
        with pytest.raises(ValueError, match=name):
            CALLS[name](dict(good(), **{arg: bad}), B.AdamWParams(lr=1e-3))
    assert called == []


@pytest.mark.parametrize("field,ok", [("grad_sumsq", FakeTensor(1, D)), ("lr_factor", FakeTensor(1, F)),
                                      ("decay", FakeTensor(3, F)), ("norm_out", FakeTensor(2, F)),
                                      ("loss_scaler", FakeTensor(8, I))])
def test_every_tensor_of_the_hyperparameters_is_checked(field, ok, called):
    for name in ("zero_adamw_prepare", "zero_adamw_step", "zero_adamw8_step"):
        CALLS[name](good(), B.AdamWParams(lr=1e-3, **{field: ok}))
        bad = [FakeTensor(ok.numel() - 1, ok.dtype), FakeTensor(ok.numel(), ok.dtype, device=1),
               FakeTensor(ok.numel(), ok.dtype, contiguous=False)]
        if field != "loss_scaler":
            bad.append(FakeTensor(ok.numel(), torch.float16))
        for b in bad:
            with pytest.raises(ValueError, match=name):
                CALLS[name](good(), B.AdamWParams(lr=1e-3, **{field: b}))
    assert len(called) == 3


@pytest.mark.parametrize("seed", [-1, 1 << 64])
def test_seed_range(seed, called):
    with pytest.raises(ValueError, match="seed"):
        CALLS["zero_adamw8_step"](good(), B.AdamWParams(lr=1e-3, seed=seed))
    assert called == []


def test_null_plans_are_refused():
    L = B._load(B.LIB_PATH)
    vp = ctypes.c_void_p
    hp = ctypes.byref(B.zero_adamw_hparams(1e-3, 0.9, 0.999, 1e-8))
    a = vp(16)
    out = B.zero_adamw_sizes()
    assert L.zero_adamw_get_sizes(None, ctypes.byref(out)) == B.ZERO_EINVAL
    assert L.zero_grad_sumsq(None, a, a, a, None, a, None) == B.ZERO_EINVAL
    assert L.zero_adamw_prepare(None, a, a, hp, None, a, None) == B.ZERO_EINVAL
    assert L.zero_adamw_step(None, a, a, a, a, a, a, hp, None, a, a, None) == B.ZERO_EINVAL
    assert L.zero_adamw8_step(None, a, a, a, a, a, a, a, hp, None, a, a, None) == B.ZERO_EINVAL
    assert L.zero_adamw8_load(None, a, a, a, a, a, None) == B.ZERO_EINVAL
    assert L.zero_adamw8_unload(None, a, a, a, a, a, None) == B.ZERO_EINVAL
    assert L.zero_reduce_adamw_bucket(None, 0, a, 8, a, a, a, a, None, a, a, None) == B.ZERO_EINVAL
    assert L.zero_reduce_adamw8_bucket(None, 0, a, 8, a, a, a, a, a, None, a, a, None) == B.ZERO_EINVAL


def test_struct_layouts_match_the_header(tmp_path):
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "zero_shard.h"', "int main(void) {"]
    structs = {"zero_adamw_hparams": B.zero_adamw_hparams, "zero_adamw_sizes": B.zero_adamw_sizes}
    for name, cls in structs.items():
        lines.append(f'printf("{name} %zu\\n", sizeof({name}));')
        lines += [f'printf("{name}.{f} %zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["return 0;", "}"]) + "\n")
    subprocess.run(["gcc", "-std=c11", "-I", INC, str(src), "-o", str(exe)], check=True)
    got = dict(x.split() for x in subprocess.run([str(exe)], capture_output=True, text=True,
                                                 check=True).stdout.splitlines())
    for name, cls in structs.items():
        assert int(got[name]) == ctypes.sizeof(cls)
        for f, _ in cls._fields_:
            assert int(got[f"{name}.{f}"]) == getattr(cls, f).offset, f


def test_noise_keys_differ_by_rank_seed_and_step():
    import adamw_reference as R
    x = np.arange(4096)
    base = R.noise(5, 1, np.array([3]), x)
    for other in ((6, 1, 3), (5 + (1 << 32), 1, 3), (5, 2, 3), (5, 1, 4)):
        assert (R.noise(other[0], other[1], np.array([other[2]]), x) == base).mean() < 0.01
