"""Dropout by token: every element against the generator's definition, in both row orders."""
import numpy as np
import pytest
import torch

from gpu_helpers import Guarded
from token_rows_ref import Batch, factor, gen, keep, kept

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
RNG = (0x123456789ABCDEF0, 7)


def _rng(seed=RNG[0], step=RNG[1]):
    return torch.tensor([seed, step], dtype=torch.int64, device="cuda")


@pytest.mark.parametrize("kind,P,lens", [
    (1, 1, [1]), (3, 1, [1]), (3, 8, [1, 0, 3]), (0, 2, [16, 24, 24]), (1, 4, [5, 90, 1, 0, 4]), (3, 3, [700, 13, 1, 266]),
    (0, 4, [8 * 300]), (3, 4, [4097]),
])
@pytest.mark.parametrize("C,dtype,p,order", [
    (8, BF16, 0.1, 1), (4, F32, 0.5, 1), (12, F32, 0.1, 0), (2568, BF16, 0.05, 0), (2568, BF16, 0.25, 1), (1132, F32, 0.9, 1),
])
def test_against_the_generator(cpt, cuda_device, kind, P, lens, C, dtype, p, order):
    b = Batch(cpt, kind, P, lens, order)
    x = b.randn(gen(1), C, dtype=dtype)
    out = Guarded(tuple(x.shape), dtype)
    cpt.cpt_dropout(b.plan, x, out.t, p, _rng(), 3, order=order)
    f = factor(*RNG, 3, b.at.cpu().numpy(), C, p)
    want = b.pick(x) * f
    got = b.pick(out.t)
    # one product of binary32 with a factor that is itself rounded, then the type's rounding
    tol = (2.0 ** -8 if dtype == BF16 else 0.0) + 3 * 2.0 ** -24
    assert ((got - want).abs() <= tol * want.abs()).all()
    assert torch.equal(got != 0, (f != 0) & (b.pick(x) != 0))
    assert b.padding_is_zero(out.t) and out.bands_intact()


def test_same_mask_in_every_order_and_layout(cpt, cuda_device):
    lens, C = [64, 16, 48], 40
    masks = []
    for kind in (0, 1, 3):
        for P in (1, 2, 4, 8):
            for order in (0, 1):
                b = Batch(cpt, kind, P, lens, order)
                x = torch.ones(b.lead + (C,), device="cuda")
                y = torch.empty_like(x)
                cpt.cpt_dropout(b.plan, x, y, 0.4, _rng(), 1, order=order)
                m = torch.zeros(b.T, C, device="cuda")
                m[b.at] = b.flat(y)[b.real]
                masks.append(m)
    assert all(torch.equal(masks[0], m) for m in masks[1:])
    assert torch.equal(masks[0].cpu() != 0, torch.from_numpy(keep(*RNG, 1, np.arange(128), C, 0.4)))


def test_step_site_seed_and_probabilities(cpt, cuda_device):
    b = Batch(cpt, 1, 1, [512], 1)
    x = torch.ones(b.lead + (64,), device="cuda")
    outs = []
    for rng, site in [(_rng(), 0), (_rng(), 1), (_rng(step=8), 0), (_rng(seed=RNG[0] + (1 << 32)), 0), (_rng(-1, -1), 2 ** 32 - 1)]:
        y = torch.empty_like(x)
        cpt.cpt_dropout(b.plan, x, y, 0.3, rng, site)
        # 32768 draws: five standard deviations of the share that is kept
        assert abs((y != 0).float().mean().item() - kept(0.3) / 65536) < 5 * (0.3 * 0.7 / 32768) ** 0.5
        outs.append(y)
    assert all(not torch.equal(outs[i], outs[j]) for i in range(5) for j in range(i))
    assert torch.equal(outs[4].reshape(512, 64).cpu() != 0, torch.from_numpy(keep(-1, -1, 2 ** 32 - 1, np.arange(512), 64, 0.3)))
    y = torch.empty_like(x)
    cpt.cpt_dropout(b.plan, x, y, 1.0, _rng())
    assert (y == 0).all()
    cpt.cpt_dropout(b.plan, x, y, 0.0)
    assert torch.equal(x, y)
    cpt.cpt_dropout(b.plan, x, y, 1e-9, _rng())     # nothing to drop at 16 bits
    assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_dropped_infinities_and_nan_are_zero(cpt, cuda_device, dtype):
    b = Batch(cpt, 3, 2, [9, 3], 1)
    x = torch.full(b.lead + (16,), float("nan"), dtype=dtype, device="cuda")
    x.view(b.R, 16)[:, ::2] = float("inf")
    y = torch.empty_like(x)
    cpt.cpt_dropout(b.plan, x, y, 0.5, _rng(), 9)
    m = torch.from_numpy(keep(*RNG, 9, b.at.cpu().numpy(), 16, 0.5)).cuda()
    got = b.pick(y)
    assert (got[~m] == 0).all() and not torch.isfinite(got[m]).any() and b.padding_is_zero(y)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_in_place(cpt, cuda_device, dtype):
    b = Batch(cpt, 3, 4, [1001, 77], 1)
    x = b.randn(gen(2), 136, dtype=dtype)
    y = torch.empty_like(x)
    cpt.cpt_dropout(b.plan, x, y, 0.2, _rng(), 5)
    cpt.cpt_dropout(b.plan, x, x, 0.2, _rng(), 5)
    assert torch.equal(x, y)


def test_its_gradient_is_the_same_call(cpt, cuda_device):
    """Linear in its input: <dropout(x), g> = <x, dropout(g)>, element by element."""
    b = Batch(cpt, 0, 2, [64], 1)
    x, g = b.randn(gen(3), 24), b.randn(gen(4), 24)
    y, d = torch.empty_like(x), torch.empty_like(x)
    cpt.cpt_dropout(b.plan, x, y, 0.35, _rng(), 2)
    cpt.cpt_dropout(b.plan, g, d, 0.35, _rng(), 2)
    one = torch.empty_like(x)
    cpt.cpt_dropout(b.plan, torch.ones_like(x), one, 0.35, _rng(), 2)
    assert torch.equal(y, x * one) and torch.equal(d, g * one)


def test_empty_batch(cpt, cuda_device):
    b = Batch(cpt, 3, 2, [0, 0], 1)
    x = torch.empty(2, 0, 8, device="cuda")
    cpt.cpt_dropout(b.plan, x, x, 0.1, _rng())
    torch.cuda.synchronize()
