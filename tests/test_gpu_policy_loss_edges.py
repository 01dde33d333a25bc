"""The clipped policy loss where a term is infinite, or beyond binary32, and what it is multiplied by is 0."""
import pytest
import torch

from test_gpu_policy_loss import Case
from token_rows_ref import Batch

pytestmark = pytest.mark.gpu

# documents of a warp, of a CTA, and of a cluster, with gradients in registers and without
LENS = [5, 90, 1, 0, 777, 4000, 9000, 17000]


@pytest.mark.parametrize("lens", [LENS[:5], LENS])
@pytest.mark.parametrize("side", ["logp", "ref"])
def test_infinite_kl(cpt, cuda_device, lens, side):
    """A token that the policy or the reference gives no weight at all (a logarithm of -inf): the KL term and the loss are
    infinite. The gradient 1 - exp(e) is -inf at e = inf and 1 at -inf."""
    b = Batch(cpt, 3, 2, lens, 1)
    c = Case(cpt, b, weights=False)
    first = torch.tensor([sum(lens[:d]) for d in range(b.n) if lens[d]], device="cuda")
    c.mask[first] = True
    _, want = [t.clone() for t in c.run()]
    (c.logp if side == "logp" else c.ref)[first] = float("-inf")
    terms, dlogp = c.run()
    some = torch.tensor(lens, device="cuda") > 0
    assert (terms[some, :2] == float("inf")).all() and (terms[~some] == 0).all()
    others = torch.ones(b.T, dtype=torch.bool, device="cuda")
    others[first] = False
    assert torch.equal(dlogp[others], want[others])
    if side == "logp":
        assert (dlogp[first] == float("-inf")).all()
    else:
        assert torch.isfinite(dlogp[first]).all()


@pytest.mark.parametrize("gap", [100.0, -1e30, float("inf"), float("nan")])
@pytest.mark.parametrize("lens", [LENS[:5], LENS])
def test_a_kl_that_is_only_reported(cpt, cuda_device, lens, gap):
    """With kl_coef 0 the loss and its gradient are those without a reference, however large the KL."""
    b = Batch(cpt, 3, 2, lens, 1)
    c = Case(cpt, b, kl=0.0)
    first = torch.tensor([sum(lens[:d]) for d in range(b.n) if lens[d]], device="cuda")
    c.mask[first] = True
    c.ref[first] = c.logp[first] + gap
    terms, dlogp = c.run()
    plain, want = c.run(logp_ref=None)
    assert torch.isfinite(want).all() and torch.equal(dlogp, want)
    assert torch.equal(terms[:, [0, 2, 3]], plain[:, [0, 2, 3]])
    some = torch.tensor(lens, device="cuda") > 0
    kl = terms[some, 1]
    if gap == -1e30:
        assert (kl > 1e25).all() and torch.isfinite(kl).all()     # exp(e) - e - 1 is -e
    else:
        assert torch.isnan(kl).all() if gap != gap else (kl == float("inf")).all()
    assert (terms[~some] == 0).all()


@pytest.mark.parametrize("gap", [100.0, 1e30, float("inf")])
@pytest.mark.parametrize("lens", [LENS[:5], LENS])
@pytest.mark.parametrize("ref", [False, True])
def test_no_advantage(cpt, cuda_device, lens, gap, ref):
    """An advantage of 0 leaves nothing of a ratio, however large."""
    b = Batch(cpt, 3, 2, lens, 1)
    c = Case(cpt, b, ref=ref, mask=False)
    c.adv[:] = 0.0
    c.logp = torch.where(torch.arange(b.T, device="cuda") % 3 == 0, -1.0, c.logp)
    c.ref = c.logp.clone() if ref else None        # no KL either
    c.old = torch.where(torch.arange(b.T, device="cuda") % 3 == 0, c.logp - gap, c.old)
    terms, dlogp = c.run()
    assert (terms[:, :3] == 0).all() and (dlogp == 0).all()
    assert torch.equal(terms[:, 3], torch.tensor(lens, device="cuda", dtype=torch.float32))


@pytest.mark.parametrize("lens", [LENS[:5], LENS])
def test_weights_of_nothing(cpt, cuda_device, lens):
    """A document without a token that counts may have any advantage and weight; one of weight 0 has no gradient, though its
    loss is infinite. Tokens that do not count have none, whatever their document's weight."""
    b = Batch(cpt, 3, 2, lens, 1)
    c = Case(cpt, b)
    doc = b.doc
    nothing, out = doc % 3 == 0, doc % 3 == 1
    c.mask &= ~nothing
    keep, (_, want) = c.weights.clone(), [t.clone() for t in c.run()]
    docs = torch.arange(b.n, device="cuda")
    for value in (float("nan"), float("inf")):
        c.adv[docs % 3 == 0] = value
        c.weights[docs % 3 == 0] = value
        terms, dlogp = c.run()
        assert (terms[docs % 3 == 0] == 0).all() and torch.equal(dlogp, want)
    c.weights = torch.where(docs % 3 == 1, 0.0, keep)
    c.adv[docs % 3 == 1] = -1.0
    first = torch.tensor([sum(lens[:d]) for d in range(b.n) if lens[d] and d % 3 == 1], device="cuda")
    c.mask[first] = True
    c.old[first] = c.logp[first] - 100.0
    terms, dlogp = c.run()
    assert (terms[doc[first], 0] == float("inf")).all()
    assert (dlogp[out] == 0).all() and torch.equal(dlogp[~out], want[~out])
    c.weights[docs % 3 == 1] = float("inf")
    _, dlogp = c.run()
    assert (dlogp[~c.mask] == 0).all()


@pytest.mark.parametrize("kl", [0.0, 0.1])
@pytest.mark.parametrize("lens", [[], [0], [0, 0, 0]])
def test_empty_batches_with_everything(cpt, cuda_device, lens, kl):
    """Documents without a token have a loss of 0, a reference and a mask given or not."""
    b = Batch(cpt, 3, 2, lens, 1)
    c = Case(cpt, b, kl=kl)
    terms, dlogp = c.run()
    assert (terms == 0).all() and dlogp.numel() == 0
