"""ShardStep's own sum of squares belongs to one gradient: a clipped step without grad_sumsq() since the
last reduce is refused.  On the CPU, with the entry points replaced by a record of their calls."""
import pytest
import torch

from zero_sharded_mixed_amd import AdamWParams, ShardStep, Zero3Schedule
from zero_sharded_mixed_amd import step as S


class Calls:
    """Stands for the binding: every entry point notes its name and its hyperparameters."""
    AdamWParams = AdamWParams

    def __init__(self):
        self.names, self.hp = [], None

    def __getattr__(self, name):
        def call(*a, **kw):
            self.names.append(name)
            self.hp = next((x for x in a if isinstance(x, AdamWParams)), self.hp)
        return call


class Plan:
    adamw_work_bytes, adamw_n_scales = 512, 4


class Summary:
    shard_numel = 64


class Bucket:
    block_offset, row_stride, first_param, n_params = 0, 64, 0, 1


@pytest.fixture(params=[32, 8])
def step(request, monkeypatch):
    calls = Calls()
    monkeypatch.setattr(S, "B", calls)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: None)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda self, stream: None)
    st = object.__new__(ShardStep)
    st.plan, st.summary, st.device, st.buckets, st.scaler, st.adamw_bits = Plan(), Summary(), "cpu", [Bucket()], None, 0
    st.nd, st.rank, st.n = 1, 0, 1
    st.packed = st.arena = torch.zeros(64, dtype=torch.int16)
    st.p32 = st.m = st.v = st.g32 = torch.zeros(64)
    st.live = st.steps = st.flag = None
    st.enable_adamw(request.param)
    st.calls = calls
    return st


CLIP, ROWS = AdamWParams(lr=1e-3, max_norm=1.0), lambda b: (None, 64)


def test_a_clipped_step_without_a_sum_is_refused(step):
    del step.calls.names[:]
    with pytest.raises(ValueError, match="grad_sumsq"):
        step.adamw(CLIP)
    assert step.calls.names == []
    assert torch.isnan(step.sumsq).all()  # a sum that nobody formed clips nothing in silence


def test_a_sum_lasts_until_the_next_reduce(step):
    step.reduce(ROWS)
    step.grad_sumsq()
    step.adamw(CLIP)
    assert step.calls.hp.grad_sumsq is step.sumsq and step.calls.hp.norm_out is step.norm_out
    step.adamw(CLIP)  # the same gradient once more
    step.reduce(ROWS)
    before = list(step.calls.names)
    with pytest.raises(ValueError, match="grad_sumsq"):
        step.adamw(CLIP)
    assert step.calls.names == before
    step.grad_sumsq()
    step.adamw(CLIP)


def test_a_layerwise_backward_ends_the_sum(step):
    step.grad_sumsq()
    z3 = object.__new__(Zero3Schedule)
    z3.st, z3.prefetch, z3.fused, z3.layers, z3.views, z3.order = step, False, False, [[0]], [[]], []
    z3.backward(lambda layer: None, ROWS)
    assert "zero_reduce_shard" in step.calls.names
    with pytest.raises(ValueError, match="grad_sumsq"):
        step.adamw(CLIP)


def test_steps_that_need_no_sum_of_their_own_run(step):
    step.reduce(ROWS)
    step.adamw(AdamWParams(lr=1e-3))
    assert step.calls.hp.grad_sumsq is None
    other = torch.ones(1, dtype=torch.float64)
    step.adamw(AdamWParams(lr=1e-3, max_norm=1.0, grad_sumsq=other))
    assert step.calls.hp.grad_sumsq is other
    step.reduce_adamw(ROWS, AdamWParams(lr=1e-3, max_norm=1.0, grad_sumsq=other))
    assert step.calls.hp.grad_sumsq is other
