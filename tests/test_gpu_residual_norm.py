"""The residual stream between two blocks and its gradient against 64-bit forms, with derived bounds."""
import itertools

import numpy as np
import pytest
import torch

from gpu_helpers import Guarded
from token_rows_ref import (U, Batch, close, factor, gen, residual_norm, residual_norm_backward)

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-5


class Case:
    """Inputs and options of both calls over one batch."""

    def __init__(self, cpt, b, C, dtype, post=True, pre=True, gate=0, p=0.0, scale=0.7, branch=True, seed=0, sigma=1.0):
        g = gen(seed + 17 * C)
        self.cpt, self.b, self.C, self.dtype, self.branch, self.p = cpt, b, C, dtype, branch, p
        self.x = b.randn(g, C, dtype=dtype, sigma=2.0 * sigma)
        self.h = b.randn(g, C, dtype=dtype, sigma=sigma) if branch else None
        self.y = b.randn(g, C, dtype=dtype, sigma=2.0 * sigma) if pre else None
        self.dy = b.randn(g, C, dtype=dtype)
        self.dn = b.randn(g, C, dtype=dtype) if pre else None
        w = lambda: 1.0 + 0.2 * torch.randn(C, device="cuda", generator=g)  # noqa: E731
        self.post, self.pre = w() if post else None, w() if pre else None
        self.gate_kind = gate
        self.gate = None
        if gate == 1:
            self.gate = b.randn(g, C, dtype=dtype)
        elif gate == 2:
            self.gate = torch.randn(b.n, C, device="cuda", generator=g).to(dtype)
        self.rng = torch.tensor([seed * 977 + 5, seed + 1], dtype=torch.int64, device="cuda") if p > 0 else None
        self.options = dict(post_weight=self.post, gate=self.gate, gate_per_document=gate == 2, scale=scale, p=p,
                            rng=self.rng, site=seed + 2, pre_weight=self.pre, eps=EPS, order=b.order)
        # padding rows hold what must not matter
        for t in (self.x, self.h, self.y, self.dy, self.dn, self.gate if gate == 1 else None):
            if t is not None:
                b.flat(t)[b.tokens < 0] = float("nan")

    def drop(self):
        if self.p == 0:
            return None
        return factor(int(self.rng[0]), int(self.rng[1]), self.options["site"], self.b.at.cpu().numpy(), self.C, self.p)

    def gate64(self):
        if self.gate_kind == 0:
            return None
        return self.b.pick(self.gate) if self.gate_kind == 1 else self.gate.double()[self.b.doc[self.b.at]]

    def w64(self, w):
        return None if w is None else w.double()

    def forward(self, inplace=False):
        like = lambda on: Guarded(tuple(self.x.shape), self.dtype) if on else None  # noqa: E731
        y, n = like(self.branch), like(self.pre is not None)
        x = self.x
        if inplace:
            y.t.copy_(x)
            x = y.t
        self.cpt.cpt_residual_norm(self.b.plan, x, self.h, y and y.t, n and n.t, **self.options)
        return y, n

    def backward(self, dy=True, need_h=True):
        b, C = self.b, self.C
        shape = tuple(self.dy.shape)
        out = {"dx": Guarded(shape, self.dtype)}
        if self.branch:
            out["dh"] = Guarded(shape, self.dtype)
        if self.gate_kind == 1:
            out["dgate"] = Guarded(shape, self.dtype)
        elif self.gate_kind == 2:
            out["dgate"] = Guarded((b.n, C), F32)
        if self.post is not None:
            out["dpost_weight"] = Guarded((C,), F32)
        if self.pre is not None:
            out["dpre_weight"] = Guarded((C,), F32)
        for o in out.values():
            o.t.fill_(float("nan"))
        t = {k: v.t for k, v in out.items()}
        need = self.cpt.cpt_residual_norm_backward_workspace_bytes(b.plan, C, self.dtype)
        work = Guarded((max(need, 256),), torch.uint8)
        work.t.fill_(0xFF)      # NaN, wherever it is read before it is written
        y = self.y if self.branch or self.y is not None else None
        self.cpt.cpt_residual_norm_backward(
            b.plan, self.h if need_h else None, y, self.dy if dy else None, self.dn, t["dx"], t.get("dh"),
            dgate=t.get("dgate"), dpost_weight=t.get("dpost_weight"), dpre_weight=t.get("dpre_weight"),
            workspace=work.t, **self.options)
        torch.cuda.synchronize()
        assert work.bands_intact() and all(o.bands_intact() for o in out.values())
        return t

    def check_forward(self, y, n):
        b, pick = self.b, self.b.pick
        want = residual_norm(pick(self.x), pick(self.h) if self.branch else None, self.gate64(), self.w64(self.post),
                             self.w64(self.pre), self.options["scale"], self.drop(), EPS)
        for got, exact, mag, what in ((y, want[0], want[1], "y"), (n, want[2], want[3], "n")):
            if got is None:
                continue
            close(self.b.flat(got.t)[b.real], exact, mag, what)
            assert b.padding_is_zero(got.t) and got.bands_intact()

    def check_backward(self, t, dy=True):
        b, pick = self.b, self.b.pick
        opt = lambda x: None if x is None else pick(x)  # noqa: E731
        scale = self.options["scale"]
        h = opt(self.h)
        want = residual_norm_backward(h, opt(self.y), pick(self.dy) if dy else None, opt(self.dn), self.gate64(),
                                      self.w64(self.post), self.w64(self.pre), scale, self.drop(), EPS)
        for k in ("dx", "dh") + (("dgate",) if self.gate_kind == 1 else ()):
            if k in t:
                close(b.flat(t[k])[b.real], *want[k], k)
                assert b.padding_is_zero(t[k]), k
        # sums: a term's own bound, and one rounding for every addition (tokens of a thread, parts, warps)
        def summed(terms, mag, count):
            return terms.sum(0), mag.sum(0) + (count + 64) * U * terms.abs().sum(0)

        for k, name in (("dpost", "dpost_weight"), ("dpre", "dpre_weight")):
            if name in t:
                close(t[name], *summed(*want[k], b.T), name)
        if self.gate_kind == 2:
            doc = b.doc[b.at]
            for d in range(b.n):
                m = doc == d
                close(t["dgate"][d], *summed(want["dgate"][0][m], want["dgate"][1][m], int(m.sum())), f"dgate {d}")


BATCHES = [(1, 1, [1]), (3, 8, [1, 0, 3]), (0, 2, [16, 24, 24]), (1, 4, [5, 90, 1, 0, 4]), (3, 3, [701, 0, 13, 1, 266])]
OPTIONS = [dict(post=q, pre=r, gate=g, p=p) for q, r, g, p in itertools.product((False, True), (False, True), (0, 1, 2), (0.0, 0.3))]


@pytest.mark.parametrize("kind,P,lens", BATCHES)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("order", [0, 1])
def test_every_combination_of_options(cpt, cuda_device, kind, P, lens, dtype, order):
    b = Batch(cpt, kind, P, lens, order)
    for i, o in enumerate(OPTIONS):
        c = Case(cpt, b, 72 if i % 2 else 320, dtype, seed=i, **o)
        c.check_forward(*c.forward())
        c.check_backward(c.backward())


# widths around every change of the rows' layout over threads: units of a part of a warp, a warp, two a lane, CTAs
@pytest.mark.parametrize("units", [1, 2, 3, 5, 8, 16, 17, 31, 32, 33, 47, 64, 65, 66, 95, 96, 97, 141, 160, 161, 256, 283, 320,
                                   321, 511, 512, 513, 640, 1023, 1024])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_every_width(cpt, cuda_device, units, dtype):
    b = Batch(cpt, 3, 2, [130, 41, 7], 1)
    C = units * (8 if dtype == BF16 else 4)
    for gate, p in ((2, 0.2), (1, 0.0)):
        c = Case(cpt, b, C, dtype, gate=gate, p=p, seed=units)
        c.check_forward(*c.forward())
        c.check_backward(c.backward())


@pytest.mark.parametrize("units", [1025, 1500, 1536, 2047, 2048])
def test_widest_float32_rows(cpt, cuda_device, units):
    b = Batch(cpt, 3, 2, [130, 41, 7], 1)
    c = Case(cpt, b, units * 4, F32, gate=2, p=0.2, seed=units)
    c.check_forward(*c.forward())
    c.check_backward(c.backward())


# beyond 1920 units the rows and the weights no longer fit beside each other; several rows for every team
@pytest.mark.parametrize("units", [1025, 1920, 1921, 2048])
@pytest.mark.parametrize("gate,p", [(1, 0.0), (1, 0.2), (2, 0.0)])
def test_widest_float32_rows_of_every_gate(cpt, cuda_device, units, gate, p):
    b = Batch(cpt, 3, 2, [330, 141, 7], 1)
    c = Case(cpt, b, units * 4, F32, gate=gate, p=p, seed=units)
    c.check_forward(*c.forward())
    c.check_backward(c.backward())


# many groups, documents inside one, over two, over many, ending at their borders
@pytest.mark.parametrize("kind,P,lens", [
    (1, 1, [20000]), (3, 4, [3000] * 5 + [1] * 500 + [0] * 40 + [9999]), (0, 2, [4] * 4000 + [4000]), (1, 8, [8] * 5000),
    (3, 2, [1] * 7777), (1, 1, [66] * 152), (1, 1, [1, 0, 0, 5000, 0, 1]),
])
@pytest.mark.parametrize("C,dtype", [(64, BF16), (640, BF16), (1132, F32), (4, F32)])
def test_documents_over_groups(cpt, cuda_device, kind, P, lens, C, dtype):
    b = Batch(cpt, kind, P, lens, 1)
    c = Case(cpt, b, C, dtype, gate=2, p=0.1, seed=3)
    c.check_forward(*c.forward())
    t = c.backward()
    # as check_backward, but the documents all at once
    want = residual_norm_backward(b.pick(c.h), b.pick(c.y), b.pick(c.dy), b.pick(c.dn), c.gate64(), c.w64(c.post),
                                  c.w64(c.pre), c.options["scale"], c.drop(), EPS)
    doc = b.doc[b.at]
    zero = torch.zeros(b.n, C, dtype=torch.float64, device="cuda")
    terms, mag = want["dgate"]
    exact = zero.clone().index_add_(0, doc, terms)
    size = zero.clone().index_add_(0, doc, terms.abs())
    length = torch.tensor(lens, device="cuda", dtype=torch.float64)[:, None]
    close(t["dgate"], exact, zero.clone().index_add_(0, doc, mag) + (length + 64) * U * size, "dgate")
    close(t["dpost_weight"], want["dpost"][0].sum(0),
          want["dpost"][1].sum(0) + (b.T + 64) * U * want["dpost"][0].abs().sum(0), "dpost")
    close(b.flat(t["dh"])[b.real], *want["dh"], "dh")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("C", [64, 640])
def test_first_norm_without_a_block(cpt, cuda_device, dtype, C):
    b = Batch(cpt, 3, 2, [33, 1], 1)
    c = Case(cpt, b, C, dtype, post=False, branch=False, scale=1.0)
    y, n = c.forward()
    assert y is None
    c.check_forward(y, n)
    c.check_backward(c.backward())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_without_a_gradient_of_the_stream(cpt, cuda_device, dtype):
    b = Batch(cpt, 0, 2, [64, 4], 1)
    c = Case(cpt, b, 264, dtype, gate=1, p=0.1)
    c.check_backward(c.backward(dy=False), dy=False)


def test_a_plain_branch_needs_no_h_in_its_gradient(cpt, cuda_device):
    b = Batch(cpt, 0, 2, [64, 4], 1)
    c = Case(cpt, b, 264, BF16, post=False, p=0.1)
    c.check_backward(c.backward(need_h=False))


@pytest.mark.parametrize("C,dtype", [(64, BF16), (640, BF16), (8192, F32)])
def test_in_place(cpt, cuda_device, C, dtype):
    b = Batch(cpt, 3, 2, [300, 41], 1)
    c = Case(cpt, b, C, dtype, gate=2, p=0.1)
    y, n = c.forward()
    y2, n2 = c.forward(inplace=True)
    assert torch.equal(y.t, y2.t) and torch.equal(n.t, n2.t)
    t = c.backward()
    d = c.dy.clone()
    rest = {k: torch.empty_like(v) for k, v in t.items() if k != "dx"}
    cpt.cpt_residual_norm_backward(b.plan, c.h, c.y, d, c.dn, d, rest["dh"], dgate=rest["dgate"],
                                   dpost_weight=rest["dpost_weight"], dpre_weight=rest["dpre_weight"], **c.options)
    assert torch.equal(d, t["dx"]) and all(torch.equal(rest[k], t[k]) for k in rest)


@pytest.mark.parametrize("C,dtype", [(64, BF16), (2560, BF16), (1132, F32)])
def test_the_same_bits_every_time(cpt, cuda_device, C, dtype):
    b = Batch(cpt, 3, 4, [2000, 1, 77, 3001], 1)
    c = Case(cpt, b, C, dtype, gate=2, p=0.1)
    first = c.backward()
    for _ in range(3):
        again = c.backward()
        assert all(torch.equal(first[k], again[k]) for k in first)


def test_the_same_tokens_in_every_layout(cpt, cuda_device):
    """Rows, and the sums over them, do not depend on the layout, the ranks or the row order."""
    lens, C = [64, 128, 32], 640
    g = gen(11)
    source = {k: torch.randn(224, C, device="cuda", generator=g).to(BF16) for k in ("x", "h", "y", "dy", "dn")}
    gate = torch.randn(3, C, device="cuda", generator=g).to(BF16)
    w = 1.0 + 0.2 * torch.randn(2, C, device="cuda", generator=g)
    seen = []
    for kind, P, order in [(1, 1, 0), (0, 2, 1), (0, 8, 1), (1, 4, 1), (3, 4, 1), (3, 3, 1)]:
        b = Batch(cpt, kind, P, lens, order)
        c = Case(cpt, b, C, BF16, gate=2, p=0.1, seed=4)
        for name, t in source.items():
            b.flat(getattr(c, name))[b.real] = t[b.at]
        c.gate.copy_(gate)
        c.post.copy_(w[0])
        c.pre.copy_(w[1])
        y, n = c.forward()
        t = c.backward()
        rows = []
        for x in (y.t, n.t, t["dx"], t["dh"]):
            v = torch.empty(b.T, C, dtype=BF16, device="cuda")
            v[b.at] = b.flat(x)[b.real]
            rows.append(v)
        seen.append(rows + [t["dgate"], t["dpost_weight"], t["dpre_weight"]])
    for rows in seen[1:]:
        assert all(torch.equal(a, r) for a, r in zip(seen[0], rows))


def test_gradient_against_differences(cpt, cuda_device):
    """The gradient call is the derivative of the forward call, along random directions in float32."""
    b = Batch(cpt, 3, 2, [40, 9], 1)
    for gate in (1, 2):
        c = Case(cpt, b, 96, F32, gate=gate, p=0.2, seed=gate, sigma=0.5)
        for t in (c.x, c.h, c.dy, c.dn) + ((c.gate,) if gate == 1 else ()):
            b.flat(t)[b.tokens < 0] = 0.0

        def value():
            y, n = c.forward()
            return (b.pick(y.t) * b.pick(c.dy)).sum().item() + (b.pick(n.t) * b.pick(c.dn)).sum().item(), y

        _, y = value()
        c.y = y.t.clone()
        g = c.backward()
        for name, grad in (("x", "dx"), ("h", "dh"), ("gate", "dgate"), ("post", "dpost_weight"), ("pre", "dpre_weight")):
            t = getattr(c, name)
            keep, v = t.clone(), torch.randn(t.shape, device="cuda", generator=gen(9))
            step = 2.0 ** -7
            vals = []
            for s in (1, -1):
                t.copy_(keep + s * step * v)
                vals.append(value()[0])
            t.copy_(keep)
            numeric = (vals[0] - vals[1]) / (2 * step)
            exact = (g[grad].double() * v.double()).sum().item()
            # outputs of size 1..4 over 49 x 96 elements carry 2^-24 of rounding each: some 1e-4 over the step; and
            # the third derivative, of the order of step^2, over as many elements
            assert abs(numeric - exact) < 2e-2 * max(1.0, abs(exact)), (name, numeric, exact)


def test_dropped_infinities_do_not_spread(cpt, cuda_device):
    b = Batch(cpt, 1, 1, [24], 1)
    c = Case(cpt, b, 64, F32, post=False, pre=False, gate=1, p=0.5)
    drop = c.drop()
    c.h.view(24, 64)[drop == 0] = float("inf")
    c.gate.view(24, 64)[drop == 0] = float("nan")
    y, _ = c.forward()
    t = c.backward()
    assert torch.isfinite(y.t).all() and all(torch.isfinite(v).all() for v in t.values())


def test_nan_stays_in_its_row(cpt, cuda_device):
    b = Batch(cpt, 3, 2, [50, 31], 1)
    for C in (64, 640):
        c = Case(cpt, b, C, BF16, p=0.1)
        row = int(b.real[20])
        b.flat(c.h)[row, 3] = float("nan")
        y, n = c.forward()
        for out in (y.t, n.t):
            bad = torch.isnan(b.flat(out)).any(1)
            assert bad[row] and bad.sum() == 1
        t = c.backward()
        bad = torch.isnan(b.flat(t["dh"])).any(1)
        assert bad[row] and bad.sum() == 1 and torch.isfinite(t["dx"]).all()


def test_zero_rows(cpt, cuda_device):
    b = Batch(cpt, 0, 2, [16], 1)
    c = Case(cpt, b, 64, F32)
    for t in (c.x, c.h, c.y):
        t.zero_()
    c.check_forward(*c.forward())
    c.check_backward(c.backward())


def test_empty_batch(cpt, cuda_device):
    b = Batch(cpt, 3, 2, [0, 0], 1)
    c = Case(cpt, b, 64, BF16, gate=2, p=0.1)
    c.forward()
    t = c.backward()
    assert (t["dgate"] == 0).all() and (t["dpost_weight"] == 0).all() and (t["dpre_weight"] == 0).all()


def test_a_row_shape_of_several_dimensions(cpt, cuda_device):
    b = Batch(cpt, 0, 2, [64], 1)
    c = Case(cpt, b, 320, BF16)
    y, n = c.forward()
    wide = lambda t: t.view(2, 32, 5, 64)  # noqa: E731
    y2, n2 = torch.empty_like(c.x), torch.empty_like(c.x)
    cpt.cpt_residual_norm(b.plan, wide(c.x), wide(c.h), wide(y2), wide(n2), **c.options)
    assert torch.equal(y.t, y2) and torch.equal(n.t, n2)
    assert np.isfinite(y2.float().cpu().numpy()).all()
