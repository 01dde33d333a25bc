"""Log-probabilities at the ends of the scale's range."""
import math

import pytest
import torch

from token_rows_ref import U, Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab", [40, 9000])
def test_the_largest_scale(cpt, cuda_device, dtype, vocab):
    """At a temperature of almost 0 the largest logits share the weight: log 2 each (off by 164 u and 2 u of itself, as in the
    forward call's derivation) and a gradient of half a target, 2^-1 of 2e38."""
    b = Batch(cpt, 0, 2, [16], 1)
    x = torch.zeros(b.lead + (vocab,), dtype=dtype, device="cuda")
    x[..., 1] = x[..., vocab - 1] = 2.0
    targets = torch.full((16,), 1, dtype=torch.int32, device="cuda")
    targets[3] = 0
    logp, stats = torch.full((16,), 7.0, device="cuda"), torch.full((16, 2), 7.0, device="cuda")
    d, dx = torch.ones(16, device="cuda"), torch.full_like(x, 7.0)
    for scale in (2.1e38, 3.4e38):
        for call in (lambda: cpt.cpt_token_logprob(b.plan, x, targets, logp, stats, scale=scale),
                     lambda: cpt.cpt_token_logprob_backward(b.plan, x, targets, stats, d, dx, scale=scale)):
            with pytest.raises(cpt.CptError) as e:
                call()
            assert e.value.status == cpt.CPT_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert (logp == 7.0).all() and (stats == 7.0).all() and (dx == 7.0).all()
    scale = 2e38
    cpt.cpt_token_logprob(b.plan, x, targets, logp, stats, scale=scale)
    cpt.cpt_token_logprob_backward(b.plan, x, targets, stats, d, dx, scale=scale)
    two = torch.arange(16, device="cuda") != 3
    off = (164 + 2) * U
    assert ((logp[two].double() + math.log(2)).abs() <= off).all() and logp[3] == -float("inf")
    rows = b.flat(dx)[b.real][torch.argsort(b.at)].double() / scale
    # half a step of bf16 or of binary32, and the weight's 300 u
    off = (2.0 ** -8 if dtype == torch.bfloat16 else U) + 300 * U
    assert ((rows[two, 1] - 0.5).abs() <= 0.5 * off).all() and ((rows[:, vocab - 1] + 0.5).abs() <= 0.5 * off).all()
    assert ((rows[3, 0] - 1.0).abs() <= off) and ((rows[3, 1] + 0.5).abs() <= 0.5 * off)
    rows[:, [0, 1, vocab - 1]] = 0
    assert (rows == 0).all()
