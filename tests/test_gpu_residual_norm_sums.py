"""The gradient's sums over tokens, exact: a token that is lost, or counted twice, changes them.

Every element is 1 or -1 and every norm is taken with eps = 3 over a power of two of columns, so that a row's mean square is 1 and its
statistic 1 / sqrt(4). Half of a row's dn times y is the negative of the other half, so the mean of the norm's gradient is 0. Then
all terms are multiples of 1/8 below 8 and no sum here needs more than 24 bits: the order of the additions does not matter, and
dx, dgate, dpost_weight and dpre_weight have to be equal to their 64-bit values. No term is 0 but those that were dropped.
"""
import numpy as np
import pytest
import torch

import test_gpu_residual_norm as base
from token_rows_ref import U, Batch, close, factor, gen, residual_norm_backward

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


class Signs(base.Case):
    """A case whose 64-bit results are exact in binary32."""

    def __init__(self, cpt, b, C, dtype, monkeypatch, gate, p, seed=0):
        monkeypatch.setattr(base, "EPS", 3.0)
        super().__init__(cpt, b, C, dtype, gate=gate, p=p, scale=1.0, seed=seed)
        g = gen(seed + 1)
        sign = lambda *s: torch.randint(0, 2, s, device="cuda", generator=g).to(F32) * 2 - 1  # noqa: E731
        R = len(b.real)
        rows = {"x": sign(R, C), "h": sign(R, C), "y": sign(R, C), "dy": sign(R, C)}
        pairs = sign(R, C // 2)
        self.post.copy_(1 + (sign(C) + 1) / 2)      # 1 or 2
        self.pre.fill_(1.0)
        rows["dn"] = torch.cat([pairs, -pairs], 1) * rows["y"]
        if gate == 1:
            rows["gate"] = sign(R, C)
        elif gate == 2:
            self.gate.copy_(sign(b.n, C))
        for name, t in rows.items():
            b.flat(getattr(self, name))[b.real] = t.to(dtype)

    def check(self):
        b, t = self.b, self.backward()
        want = residual_norm_backward(b.pick(self.h), b.pick(self.y), b.pick(self.dy), b.pick(self.dn), self.gate64(),
                                      self.w64(self.post), self.w64(self.pre), 1.0, self.drop(), 3.0)
        exact = lambda got, value, what: torch.testing.assert_close(got.double(), value, rtol=0, atol=0, msg=what)  # noqa: E731
        exact(b.flat(t["dx"])[b.real], want["dx"][0], "dx")
        exact(t["dpost_weight"], want["dpost"][0].sum(0), "dpost_weight")
        exact(t["dpre_weight"], want["dpre"][0].sum(0), "dpre_weight")
        if self.gate_kind == 1:
            exact(b.flat(t["dgate"])[b.real], want["dgate"][0], "dgate")
        elif self.gate_kind == 2:
            zero = torch.zeros(b.n, self.C, dtype=torch.float64, device="cuda")
            exact(t["dgate"], zero.index_add_(0, b.doc[b.at], want["dgate"][0]), "dgate")
        close(b.flat(t["dh"])[b.real], *want["dh"], "dh")


def test_the_statistic_is_exact(cpt, cuda_device):
    """What the others rest on: 1 / sqrt(1 + 3) of a row of signs is 1/2 in the kernels."""
    for C, dtype in ((64, F32), (1024, BF16), (2048, F32)):
        b = Batch(cpt, 1, 1, [33], 1)
        x = torch.randint(0, 2, (1, 33, C), device="cuda", generator=gen(1)).to(dtype) * 2 - 1
        n = torch.empty_like(x)
        cpt.cpt_residual_norm(b.plan, x, None, None, n, pre_weight=torch.ones(C, device="cuda"), eps=3.0)
        assert torch.equal(n, x / 2)


@pytest.mark.parametrize("kind,P,lens", [
    (1, 1, [20000]), (3, 4, [3000] * 5 + [1] * 500 + [0] * 40 + [9999]), (0, 2, [4] * 4000 + [4000]), (1, 8, [8] * 5000),
    (3, 2, [1] * 7777), (1, 1, [66] * 152), (1, 1, [1, 0, 0, 5000, 0, 1]), (3, 3, [609, 1, 607, 0, 0, 1216, 2]),
])
@pytest.mark.parametrize("C,dtype", [(16, F32), (64, BF16), (512, BF16), (1024, BF16), (2048, F32)])
def test_every_token_counts_once(cpt, cuda_device, monkeypatch, kind, P, lens, C, dtype):
    b = Batch(cpt, kind, P, lens, 1)
    for gate, p in ((0, 0.0), (1, 0.0), (2, 0.0), (2, 0.5)):
        Signs(cpt, b, C, dtype, monkeypatch, gate, p, seed=gate).check()


@pytest.mark.parametrize("T", [151, 152, 153, 607, 608, 609, 1215, 1216, 1217, 4863, 4864, 4865])
@pytest.mark.parametrize("C,dtype", [(64, BF16), (512, BF16), (1024, BF16), (4096, BF16), (2048, F32)])
def test_tokens_around_whole_rounds(cpt, cuda_device, monkeypatch, T, C, dtype):
    """One token more or fewer than the groups of all SMs take in whole rounds, a document's border among the last."""
    b = Batch(cpt, 1, 1, [T - 3, 2, 1], 1)
    for gate in (0, 2):
        Signs(cpt, b, C, dtype, monkeypatch, gate, 0.0, seed=T).check()


def test_gradient_of_rows_past_2_to_the_32(cpt, cuda_device):
    """1.1 million rows of 4096, zeros but for the first and the last, which lie past 2^32 elements (and 2^33 bytes): their own
    gradients, and the sums, against 64 bits. A sum has 80 terms and at most 64 more additions (of zeros) with a rounding."""
    T, C, last, scale, p = 1_100_003, 4096, 40, 0.5, 0.1
    b = Batch(cpt, 1, 1, [T - 20, 20], 1)
    g = gen(0)
    ends = torch.cat([torch.arange(last), torch.arange(T - last, T)]).cuda()
    some = {k: torch.randn(2 * last, C, device="cuda", generator=g).to(BF16) for k in ("h", "y", "dy", "dn")}
    t = {}
    for k, v in some.items():
        t[k] = torch.zeros(1, T, C, dtype=BF16, device="cuda")
        t[k][0, ends] = v
    w = 1 + 0.1 * torch.randn(2, C, device="cuda", generator=g)
    gate = torch.randn(2, C, device="cuda", generator=g).to(BF16)
    rng = torch.tensor([5, 6], dtype=torch.int64, device="cuda")
    dx, dh = torch.full_like(t["h"], 7.0), torch.full_like(t["h"], 7.0)
    dgate, dw = torch.full((2, C), 7.0, device="cuda"), torch.full((2, C), 7.0, device="cuda")
    cpt.cpt_residual_norm_backward(b.plan, t["h"], t["y"], t["dy"], t["dn"], dx, dh, post_weight=w[0], pre_weight=w[1], gate=gate,
                                   gate_per_document=True, scale=scale, p=p, rng=rng, site=1, eps=1e-5, dgate=dgate,
                                   dpost_weight=dw[0], dpre_weight=dw[1])
    doc = b.doc[ends]
    drop = factor(5, 6, 1, np.asarray(ends.cpu()), C, p)
    want = residual_norm_backward(*[some[k].double() for k in ("h", "y", "dy", "dn")], gate.double()[doc], w[0].double(), w[1].double(),
                                  scale, drop, 1e-5)
    close(dx[0, ends], *want["dx"], "dx")
    close(dh[0, ends], *want["dh"], "dh")
    for out in (dx, dh):
        assert out[0, last:-last].abs().max() == 0
    total = lambda terms, mag: (terms.sum(0), mag.sum(0) + 144 * U * terms.abs().sum(0))  # noqa: E731
    close(dw[0], *total(*want["dpost"]), "dpost_weight")
    close(dw[1], *total(*want["dpre"]), "dpre_weight")
    for d in range(2):
        close(dgate[d], *total(*[v[doc == d] for v in want["dgate"]]), f"dgate {d}")
