"""The clipped policy loss against its 64-bit form, with derived bounds.

In u = 2^-24: exp is off by 4 u and the products after it by one each, so a token's term by 8 u; the sums are compensated
within a thread and go through at most 12 levels after it. A difference of logarithms is rounded once (u of
itself), which exp makes relative. exp(e) - e - 1 is off by 10 u of itself from its series and by 4 u of the
parts beyond it.
"""
import math

import pytest
import torch

from gpu_helpers import Guarded
from token_rows_ref import U, Batch, gen

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, cpt, b, ref=True, mask=True, weights=True, low=0.2, high=0.28, kl=0.04, spread=0.2, seed=0):
        g = gen(seed + b.T)
        r = lambda n, s=1.0: torch.randn(n, device="cuda", generator=g) * s  # noqa: E731
        self.cpt, self.b = cpt, b
        self.logp = -1.5 * r(b.T).abs()
        self.old = self.logp + r(b.T, spread)
        self.ref = self.logp + r(b.T, spread) if ref else None
        self.mask = torch.rand(b.T, device="cuda", generator=g) < 0.6 if mask else None
        self.adv = r(b.n)
        self.weights = torch.rand(b.n, device="cuda", generator=g) if weights else None
        self.low, self.high, self.kl = low, high, kl if ref else 0.0

    def run(self, **kw):
        terms, dlogp = Guarded((self.b.n, 4), torch.float32), Guarded((self.b.T,), torch.float32)
        terms.t.fill_(7.0)
        dlogp.t.fill_(7.0)
        self.cpt.cpt_policy_loss(self.b.plan, self.logp, self.old, self.adv, terms.t, dlogp.t,
                                 **{**dict(logp_ref=self.ref, mask=self.mask, weights=self.weights, clip_low=self.low,
                                           clip_high=self.high, kl_coef=self.kl), **kw})
        torch.cuda.synchronize()
        assert terms.bands_intact() and dlogp.bands_intact()
        return terms.t, dlogp.t

    def check(self, terms, dlogp):
        b, doc, n = self.b, self.b.doc, self.b.n
        on = torch.ones(b.T, dtype=torch.bool, device="cuda") if self.mask is None else self.mask != 0
        z = lambda v: torch.zeros(n, dtype=torch.float64, device="cuda").index_add_(0, doc, torch.where(on, v, 0.0))  # noqa: E731
        count = z(torch.ones(b.T, dtype=torch.float64, device="cuda"))
        share = 1.0 / count.clamp(min=1.0)
        A = self.adv.double()[doc]
        u = self.logp.double() - self.old.double()
        r = torch.exp(u)
        free, held_at = -A * r, -A * r.clamp(1.0 - self.low, 1.0 + self.high)
        held = held_at > free
        loss, g = torch.maximum(free, held_at), torch.where(held, 0.0, free)
        err = loss.abs() * (8 + u.abs()) * U
        gerr = g.abs() * (8 + u.abs()) * U
        kl = torch.zeros_like(loss)
        klerr = torch.zeros_like(loss)
        if self.ref is not None:
            e = self.ref.double() - self.logp.double()
            kl = torch.expm1(e) - e
            kl = torch.where(e.abs() < 1e-3, e * e * (0.5 + e / 6 + e * e / 24), kl)
            klerr = 10 * U * kl + torch.where(e.abs() < 0.49, 0.0, 4 * U * (torch.expm1(e).abs() + e.abs())) \
                + U * (e * torch.expm1(e)).abs()
            g = g - self.kl * torch.expm1(e)
            gerr = gerr + self.kl * (6 * U * torch.expm1(e).abs() + U * e.abs() * torch.exp(e))
        w = (torch.full((n,), 1.0 / n, dtype=torch.float64, device="cuda") if self.weights is None
             else self.weights.double()) * share
        assert torch.equal(terms[:, 3].double(), count)
        for col, value, off in ((0, loss + self.kl * kl, err + self.kl * klerr), (1, kl, klerr), (2, held.double(), 0.0 * kl)):
            want = z(value) * share
            tol = (z(off) + 16 * U * z(value.abs())) * share
            assert ((terms[:, col].double() - want).abs() <= tol).all(), col
        want = torch.where(on, g * w[doc], 0.0)
        tol = torch.where(on, (gerr + 6 * U * (g.abs() + (0 if self.ref is None else self.kl * torch.expm1(e).abs()))) * w[doc], 0.0)
        assert ((dlogp.double() - want).abs() <= tol).all()
        assert (dlogp[~on] == 0).all()


BATCHES = [(1, 1, [1]), (3, 8, [1, 0, 3]), (0, 2, [16, 24, 24]), (1, 4, [5, 90, 1, 0, 4]), (3, 3, [701, 0, 13, 1, 266]),
           (3, 2, [1] * 500), (1, 1, [100000]), (3, 4, [40000, 1, 0, 7, 3000, 511, 512, 513, 16385]), (1, 1, [8191, 8192, 8193])]


@pytest.mark.parametrize("kind,P,lens", BATCHES)
@pytest.mark.parametrize("ref,mask,weights", [(True, True, True), (False, True, False), (True, False, False), (False, False, True)])
def test_against_64_bits(cpt, cuda_device, kind, P, lens, ref, mask, weights):
    c = Case(cpt, Batch(cpt, kind, P, lens, 1), ref, mask, weights)
    c.check(*c.run())


@pytest.mark.parametrize("low,high", [(0.0, 0.0), (1.0, 0.0), (0.2, 1e30), (1.0, 1e30), (0.999, 3.0)])
def test_borders_of_the_clip(cpt, cuda_device, low, high):
    c = Case(cpt, Batch(cpt, 3, 2, [900, 77], 1), low=low, high=high, spread=0.8)
    c.check(*c.run())


def test_ratios_next_to_a_border(cpt, cuda_device):
    """Differences of logarithms within a few steps of a border: each falls on the side that it lies on."""
    b = Batch(cpt, 1, 1, [4096], 1)
    for A in (1.0, -1.0):
        c = Case(cpt, b, ref=False, mask=False)
        c.adv[:] = A
        border = math.log1p(c.high) if A > 0 else math.log1p(-c.low)
        for steps in (-2, -1, 0, 1, 2):
            c.logp = (c.old.double() + border).float()
            c.logp.view(torch.int32).add_(steps)
            c.check(*c.run())


def test_ratio_of_one_has_its_gradient(cpt, cuda_device):
    """On the sampling policy itself the ratio is 1 and the gradient -A w / N, clip or no clip."""
    b = Batch(cpt, 0, 2, [16, 24], 1)
    c = Case(cpt, b, ref=False, mask=False, low=0.0, high=0.0)
    c.old = c.logp.clone()
    terms, dlogp = c.run()
    want = (-c.adv * c.weights / torch.tensor([16.0, 24.0], device="cuda"))[b.doc]
    assert ((dlogp - want).abs() <= 4 * U * want.abs()).all()
    assert (terms[:, 2] == 0).all()


@pytest.mark.parametrize("size", [1e-6, 1e-4, 1e-2, 0.49, 0.51, 3.0, 40.0])
def test_kl_term_of_any_size(cpt, cuda_device, size):
    c = Case(cpt, Batch(cpt, 1, 1, [777], 1), mask=False, kl=1.0)
    g = gen(1)
    c.ref = c.logp + (torch.rand(777, device="cuda", generator=g) * 2 - 1) * size
    c.check(*c.run())


def test_masked_tokens_do_not_matter(cpt, cuda_device):
    b = Batch(cpt, 3, 2, [300, 0, 41], 1)
    c = Case(cpt, b)
    want = [t.clone() for t in c.run()]
    for t in (c.logp, c.old, c.ref):
        t[~c.mask] = float("nan")
    got = c.run()
    assert all(torch.equal(a, r) for a, r in zip(want, got))
    c.mask = c.mask.to(torch.uint8) * 255          # any value but 0 counts
    assert all(torch.equal(a, r) for a, r in zip(want, c.run()))
    c.mask = torch.zeros_like(c.mask)              # documents without a token
    terms, dlogp = c.run()
    assert (terms == 0).all() and (dlogp == 0).all()


def test_infinite_logarithms(cpt, cuda_device):
    b = Batch(cpt, 1, 1, [8], 1)
    c = Case(cpt, b, ref=False, mask=False, weights=False)
    c.adv[:] = 1.0
    c.logp[3] = float("-inf")      # a token that the policy no longer gives any weight: ratio 0
    terms, dlogp = c.run()
    assert torch.isfinite(terms).all() and torch.isfinite(dlogp).all() and dlogp[3] == 0
    c.old[5] = float("-inf")       # one that it had no weight in: held by the clip
    terms, dlogp = c.run()
    assert torch.isfinite(terms).all() and dlogp[5] == 0
    c.adv[:] = -1.0
    terms, dlogp = c.run()
    assert terms[0, 0] == float("inf")


def test_gradient_against_differences(cpt, cuda_device):
    """Step 2^-8 in every logarithm away from the borders: rounding of a loss of size 1, 2^-22 over 2^-7, and a third derivative
    of at most 4 times step^2 / 6."""
    b = Batch(cpt, 3, 2, [60, 31, 8], 1)
    c = Case(cpt, b, spread=0.1, low=0.5, high=0.9, kl=0.3)
    _, g = c.run()
    v = torch.randn(b.T, device="cuda", generator=gen(2)).clamp(-2, 2)
    keep, step, vals = c.logp.clone(), 2.0 ** -8, []
    for s in (1, -1):
        c.logp = keep + s * step * v
        vals.append((c.run()[0][:, 0].double() * c.weights.double()).sum().item())
    numeric, exact = (vals[0] - vals[1]) / (2 * step), (g.double() * v.double()).sum().item()
    total = (c.weights.double() * (1 + c.adv.double().abs())).sum().item()
    assert abs(numeric - exact) <= total * (2.0 ** -20 / step + 8 * 4 * step ** 2 / 6)


def test_the_same_bits_every_time(cpt, cuda_device):
    c = Case(cpt, Batch(cpt, 3, 4, [40000, 1, 0, 7, 3000], 1))
    first = c.run()
    for _ in range(3):
        assert all(torch.equal(a, r) for a, r in zip(first, c.run()))


def test_empty_batches(cpt, cuda_device):
    for lens in ([], [0, 0]):
        b = Batch(cpt, 3, 2, lens, 1)
        e = torch.empty(0, device="cuda")
        terms = torch.full((len(lens), 4), 7.0, device="cuda")
        cpt.cpt_policy_loss(b.plan, e, e, torch.zeros(len(lens), device="cuda"), terms, e)
        torch.cuda.synchronize()
        assert (terms == 0).all()
