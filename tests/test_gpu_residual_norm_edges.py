"""The residual norms where zeros, infinities and group borders meet, against 64-bit forms with derived bounds."""
import pytest
import torch

import test_gpu_residual_norm as base
from token_rows_ref import Batch

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


# few tokens leave groups of threads without any, others leave a group's last rounds without one
@pytest.mark.parametrize("kind,P,lens", [(1, 1, [1]), (1, 1, [65]), (3, 2, [3, 0, 130, 41, 7]), (3, 3, [701, 0, 13, 1, 266])])
@pytest.mark.parametrize("C,dtype", [(8, BF16), (64, BF16), (64, F32), (320, F32), (512, BF16), (640, BF16), (1132, F32)])
def test_without_an_eps(cpt, cuda_device, monkeypatch, kind, P, lens, C, dtype):
    """eps may be 0. No row here is zeros, so every result is finite, the sums over the tokens among them."""
    monkeypatch.setattr(base, "EPS", 0.0)
    b = Batch(cpt, kind, P, lens, 1)
    for gate in (0, 1, 2):
        for post, pre, p in ((True, True, 0.0), (True, True, 0.3), (True, False, 0.0), (False, True, 0.3)):
            c = base.Case(cpt, b, C, dtype, post=post, pre=pre, gate=gate, p=p, seed=gate)
            c.check_forward(*c.forward())
            t = c.backward()
            assert all(torch.isfinite(v).all() for v in t.values())
            c.check_backward(t)
