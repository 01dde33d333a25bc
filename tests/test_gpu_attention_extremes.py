"""The attention layer where scores, weights and references lie far apart,
against dense 64-bit forms (bounds as derived in attention_ref)."""
import math

import pytest
import torch

import attention_ref as ref
from test_gpu_attention import Batch

pytestmark = pytest.mark.gpu


# few query tiles (an item's key tiles are shared out between two pipelines and joined), or many
@pytest.mark.parametrize("heads", [(2, 1), (40, 20)])
@pytest.mark.parametrize("keys", [(200, 300), (100, 400), (300, 400), (300, 301), (130, 260)])
@pytest.mark.parametrize("score", [80.0, 87.0, 87.5, 88.0, 88.5, 91.0, 95.0])
def test_late_scores_in_two_tiles(cpt, cuda_device, score, keys, heads):
    """Two late keys score the same, 80 to 95 above all others, in one tile or in tiles that two
    pipelines take: both weigh as much, whatever reference each pipeline has. A score here is one product of two
    bf16 values, so it is exact; weights, lse and the gradients are checked within the usual bounds."""
    b = Batch(cpt, 0, 1, [512], *heads, 64, 512, 0, scale=1.0)
    b.q.zero_()
    b.q[..., 0] = 8.0
    b.k.zero_()
    for x in keys:
        b.k[x, :, 0] = score / 8   # a bf16 value
    b.v.div_(8)
    b.forward()
    b.check_forward()
    b.backward()
    b.check_backward()
    assert cpt.cpt_kernel_wait_timeouts() == 0


@pytest.mark.parametrize("heads", [(2, 1), (40, 20)])
@pytest.mark.parametrize("second", [-6.0, -2.0, -0.5])
@pytest.mark.parametrize("score", [86.0, 90.0, 94.0])
def test_late_scores_a_little_apart(cpt, cuda_device, score, second, heads):
    """As above with the later of the two a little lower, and a third a little lower still."""
    b = Batch(cpt, 0, 1, [512], *heads, 128, 512, 0, scale=1.0)
    b.q.zero_()
    b.q[..., 0] = 8.0
    b.k.zero_()
    for i, x in enumerate((200, 300, 420)):
        b.k[x, :, 0] = (score + i * second) / 8
    b.forward()
    b.check_forward()
    b.backward()
    b.check_backward()


# all scores in [0.5, 1) of 2 ** power: from a spacing of binary32 that is a few units (2 ** 26) to scores whose
# base-2 form is past the largest binary32 (2 ** 128)
@pytest.mark.parametrize("heads", [(2, 1), (80, 40)])
@pytest.mark.parametrize("sign", ["positive", "negative", "both"])
@pytest.mark.parametrize("power", [26, 30, 34, 40, 64, 100, 128])
def test_scores_of_any_size(cpt, cuda_device, power, sign, heads):
    """Finite scores of any size: the weights depend on their differences alone. Every score is one product of two
    bf16 values, exact in binary32, and the differences are whole steps of it. The weights expected are formed from the
    differences to the largest score: beside scores of 2 ** 64 the log-sum-exp of equal ones does not hold their
    number, not in 64 bits either."""
    b = Batch(cpt, 3, 1, [150, 260], *heads, 64, 200, 3, scale=1.0)
    g = torch.Generator(device="cuda").manual_seed(power)
    b.q.zero_()
    b.q[..., 0] = 2.0 ** (power // 2)
    b.k.zero_()
    # keys of 128 to 255 in 2 ** -8, and the largest of all (power 128: 0.996 * 2 ** 128, a binary32) among them
    step = torch.randint(128, 256, b.k.shape[:2], device="cuda", generator=g).float() / 256
    if sign == "negative":
        step = -step
    elif sign == "both":
        step *= torch.randint(0, 2, step.shape, device="cuda", generator=g) * 2 - 1
    b.k[..., 0] = step * 2.0 ** (power - power // 2)
    b.forward()
    assert b.out.bands_intact() and b.lse.bands_intact()
    kk, vv = (x.double().repeat_interleave(2, 1) for x in (b.k, b.v))
    scores = torch.einsum("ihd,jhd->hij", b.q.double(), kk).masked_fill(~b.see, -math.inf)
    p = torch.softmax(scores, -1).masked_fill(~b.see, 0.0)
    out, mag = (torch.einsum("hij,jhd->ihd", p, x) for x in (vv, vv.abs()))
    # the bound of attention64
    tol = (ref.U + 2 * ref.E32) * mag + ref.U * (1 + ref.U) * out.abs() + 1e-30
    real = ~b.pad
    assert ((b.out.t.double() - out).abs() <= tol)[real].all()
    lse = torch.logsumexp(scores, -1)
    assert ((b.lse.t.double() - lse).abs() <= ref.E32 + 2.0 ** -22 * lse.abs())[:, real].all()
    assert (b.out.t[b.pad] == 0).all() and (b.lse.t[:, b.pad] == -math.inf).all()
    assert cpt.cpt_kernel_wait_timeouts() == 0
