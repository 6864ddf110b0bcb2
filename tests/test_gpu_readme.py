"""The README's Python example runs as it stands: one process in the place of eight ranks, every rank's
rows its own.  Four steps: Adam, fused Adam, AdamW with 8-bit states, fused AdamW."""
import os
import re

import pytest
import torch

import zero_sharded_mixed_amd as Z

pytestmark = pytest.mark.gpu
README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


@pytest.mark.skipif(not os.path.exists(README), reason="this copy of the repository has no README.md")
def test_the_example_runs_and_every_step_is_taken_once():
    code = re.search(r"## Use from Python\s+```python\n(.*?)```", open(README).read(), flags=re.S).group(1)
    numels, dev = [5000, 77, 4096 * 8], "cuda"
    fp32 = [torch.randn(n, device=dev) for n in numels]
    grads = [torch.randn(n, device=dev).mul_(1e-2).bfloat16() for n in numels]
    stride = Z.zero_plan_bucket_info(Z.zero_plan_create(numels, 8, 3, 10 ** 9, Z.ZERO_BF16), 0).row_stride
    rows = (torch.randn(8, stride, device=dev) * 1e-2).bfloat16()
    params16 = [torch.zeros(n, dtype=torch.bfloat16, device=dev) for n in numels]
    names = dict(numels=numels, r=3, fp32_params=fp32, grads=grads, recv_rows=[rows], row_stride=stride, loss_scale=1.0,
                 params16=params16, decay_of_each_parameter=torch.ones(3, device=dev),
                 schedule=torch.ones(1, device=dev))
    exec(code, names)
    st = names["st"]
    assert st.steps.tolist() == [4, 4, 4] and int(st.flag) == 0
    assert bool(torch.isfinite(st.p32).all()) and 0 < float(st.norm_out[1]) <= 1
    assert all(bool(p.isfinite().all()) for p in params16)
