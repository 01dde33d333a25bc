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


DROPPED = [(64, BF16), (64, F32), (512, BF16), (640, BF16), (1132, F32)]


@pytest.mark.parametrize("C,dtype", DROPPED)
@pytest.mark.parametrize("pre", [False, True])
@pytest.mark.parametrize("gate", [0, 1, 2])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_what_was_dropped_does_not_matter(cpt, cuda_device, C, dtype, pre, gate, value):
    """Without a norm of its own the branch is elementwise: what stands in dropped elements of h, and of a gate that nothing
    else reads, changes no result."""
    b = Batch(cpt, 3, 2, [50, 31] + [1] * 60 + [0, 200], 1)
    c = base.Case(cpt, b, C, dtype, post=False, pre=pre, gate=gate, p=0.5, seed=1)
    dropped = c.drop() == 0
    plain = c.h.clone()
    b.flat(c.h)[b.real] = torch.where(dropped, value, b.pick(plain)).to(dtype)
    assert not torch.isfinite(b.pick(c.h)).all()
    keep = None if gate == 0 else c.gate.clone()
    if gate == 1:
        b.flat(c.gate)[b.real] = torch.where(dropped, value, b.pick(keep)).to(dtype)
    elif gate == 2:
        doc = b.doc[b.at]
        kept = torch.zeros(b.n, C, dtype=torch.float64, device="cuda").index_add_(0, doc, (~dropped).double())
        assert (kept[2:62] == 0).any()
        c.gate = torch.where(kept == 0, value, keep.double()).to(dtype)
        c.options["gate"] = c.gate
    y, n = c.forward()
    t = c.backward()
    c.h = plain
    if gate:
        c.gate = keep
    c.check_forward(y, n)
    c.check_backward(t)


@pytest.mark.parametrize("C,dtype", DROPPED)
@pytest.mark.parametrize("pre", [False, True])
@pytest.mark.parametrize("gate", [0, 1, 2])
def test_dropped_infinities_behind_a_norm(cpt, cuda_device, C, dtype, pre, gate):
    """A row with an infinite element has a norm of 0 in the others. Where the infinite one is dropped the row's branch is 0:
    it adds nothing to y or to any sum, and the others' gradients are 0."""
    b = Batch(cpt, 3, 2, [50, 31] + [1] * 60 + [0, 200], 1)
    c = base.Case(cpt, b, C, dtype, post=True, pre=pre, gate=gate, p=0.5, seed=2)
    dropped = c.drop() == 0
    rows = torch.arange(3, len(b.real), 7, device="cuda")
    h = b.pick(c.h)
    at = torch.zeros_like(dropped)
    at[rows] = dropped[rows] & (torch.rand(len(rows), C, device="cuda") < 0.2)
    at[rows[0]] = dropped[rows[0]]
    h[at] = float("inf")
    b.flat(c.h)[b.real] = h.to(dtype)
    y, n = c.forward()
    t = c.backward()
    wild = at.any(1)
    assert wild.sum() > 20
    b.flat(c.h)[b.real[wild]] = 0.0     # the same branch and sums; its own gradient differs
    c.check_forward(y, n)
    dh = b.flat(t["dh"])[b.real].double()
    assert (dh[wild][~at[wild]] == 0).all()
    c.check_backward({k: v for k, v in t.items() if k != "dh"})
    calm = base.residual_norm_backward(b.pick(c.h), None if c.y is None else b.pick(c.y), b.pick(c.dy), None if c.dn is None else b.pick(c.dn),
                                       c.gate64(), c.w64(c.post), c.w64(c.pre), c.options["scale"], c.drop(), base.EPS)["dh"]
    base.close(t["dh"].view(b.R, C)[b.real][~wild], *[v[~wild] for v in calm], "dh")


@pytest.mark.parametrize("C,dtype", DROPPED)
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_gates_of_dropped_columns_behind_a_norm(cpt, cuda_device, C, dtype, value):
    """A document's gate in a column that is dropped in all its tokens matters to nothing."""
    b = Batch(cpt, 1, 1, [1] * 300 + [40, 0, 2, 2], 1)
    c = base.Case(cpt, b, C, dtype, gate=2, p=0.5, seed=3)
    kept = torch.zeros(b.n, C, dtype=torch.float64, device="cuda").index_add_(0, b.doc[b.at], (c.drop() != 0).double())
    keep = c.gate
    c.options["gate"] = c.gate = torch.where(kept == 0, value, keep.double()).to(dtype)
    y, n = c.forward()
    t = c.backward()
    c.gate = keep
    c.check_forward(y, n)
    c.check_backward(t)


@pytest.mark.parametrize("C,dtype", DROPPED)
@pytest.mark.parametrize("pre", [False, True])
@pytest.mark.parametrize("gate", [0, 1, 2])
def test_gradient_of_a_dropped_infinity(cpt, cuda_device, C, dtype, pre, gate):
    """Behind a norm an infinite element of h makes its row's branch and its gradient 0, its own gradient too where it is dropped."""
    b = Batch(cpt, 3, 2, [50, 31, 7], 1)
    c = base.Case(cpt, b, C, dtype, post=True, pre=pre, gate=gate, p=0.5, seed=4)
    h = b.pick(c.h)
    at = c.drop() == 0
    at[::2] = False
    h[at] = -float("inf")
    b.flat(c.h)[b.real] = h.to(dtype)
    dh = b.flat(c.backward()["dh"])[b.real]
    assert torch.isfinite(dh).all() and (dh[1::2] == 0).all() and (dh[::2] != 0).any(1).all()
