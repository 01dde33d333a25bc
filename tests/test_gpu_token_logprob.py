"""Log-probabilities of targets and their gradient against 64-bit forms, with derived bounds.

Bounds, in u = 2^-24. A weight 2^(c (x - m)) carries the roundings of the difference, of c and of their product, 3 u of the
exponent each, and 3 u of the instruction. Weighted by themselves exponents average to at most log2 of
the vocabulary (18), so the sum is off by 3 * 18 + 3 < 64 u, and by one u for each of the at most
100 additions, products and joins that a term goes through: l is off by 164 u and 2 u of itself.
"""
import math

import numpy as np
import pytest
import torch

from gpu_helpers import Guarded
from token_rows_ref import U, Batch, gen

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


class Case:
    def __init__(self, cpt, b, vocab, dtype, scale=1.0, pad=0, sigma=3.0, share=0.8, seed=0):
        self.cpt, self.b, self.vocab, self.dtype = cpt, b, vocab, dtype
        self.scale = float(np.float32(scale))
        per = 8 if dtype == BF16 else 4
        self.width = -(-vocab // per) * per + pad
        g = gen(seed + vocab)
        self.logits = b.randn(g, self.width, dtype=dtype, sigma=sigma)
        # what must not matter: padding rows and columns
        b.flat(self.logits)[:, vocab:] = float("nan")
        b.flat(self.logits)[b.tokens < 0] = float("nan")
        t = torch.randint(0, vocab, (b.T,), device="cuda", generator=g)
        none = torch.rand(b.T, device="cuda", generator=g) >= share
        odd = torch.randint(0, 3, (b.T,), device="cuda", generator=g)
        bad = torch.tensor([-1, -(2 ** 31), vocab], device="cuda")[odd]
        self.targets = torch.where(none, bad, t).to(torch.int32)
        self.has = ~none
        self.dlogp = torch.randn(b.T, device="cuda", generator=g)
        self.dlogp[torch.rand(b.T, device="cuda", generator=g) < 0.1] = 0.0

    def rows(self):
        """(row of every token with a target, its token)."""
        keep = self.has[self.b.at]
        return self.b.real[keep], self.b.at[keep]

    def forward(self):
        T = self.b.T
        logp, stats = Guarded((T,), F32), Guarded((T, 2), F32)
        logp.t.fill_(7.0)
        stats.t.fill_(7.0)
        self.cpt.cpt_token_logprob(self.b.plan, self.logits, self.targets, logp.t, stats.t, vocab=self.vocab,
                                   scale=self.scale, order=self.b.order)
        torch.cuda.synchronize()
        assert logp.bands_intact() and stats.bands_intact()
        return logp.t, stats.t

    def check_forward(self, logp, stats):
        q, t = self.rows()
        assert (logp[~self.has] == 0).all() and (stats[~self.has] == 0).all()
        for a in range(0, len(q), 256):
            x = self.b.flat(self.logits)[q[a:a + 256], :self.vocab].double()
            tt = t[a:a + 256]
            m = x.amax(1)
            l = torch.logsumexp((x - m[:, None]) * self.scale, 1)
            gap = (x.gather(1, self.targets[tt].long()[:, None]).squeeze(1) - m) * self.scale
            lb = 164 * U + 2 * U * l.abs()
            assert torch.equal(stats[tt, 0].double(), m)
            assert ((stats[tt, 1].double() - l).abs() <= lb).all()
            assert ((logp[tt].double() - (gap - l)).abs() <= lb + 3 * U * gap.abs() + U * (gap - l).abs()).all()

    def backward(self, stats, inplace=False):
        out = Guarded(tuple(self.logits.shape), self.dtype)
        src = self.logits
        if inplace:
            out.t.copy_(src)
            src = out.t
        else:
            out.t.fill_(7.0)
        self.cpt.cpt_token_logprob_backward(self.b.plan, src, self.targets, stats, self.dlogp, out.t, vocab=self.vocab,
                                            scale=self.scale, order=self.b.order)
        torch.cuda.synchronize()
        assert out.bands_intact()
        return out.t

    def check_backward(self, got, stats):
        b, V = self.b, self.vocab
        got = b.flat(got)
        q, t = self.rows()
        on = self.dlogp[t] != 0
        q, t = q[on], t[on]
        rest = torch.ones(b.R, dtype=torch.bool, device="cuda")
        rest[q] = False
        assert (got[rest] == 0).all() and (got[:, V:] == 0).all()
        c = self.scale / math.log(2)
        for a in range(0, len(q), 256):
            x = b.flat(self.logits)[q[a:a + 256], :V].double()
            tt = t[a:a + 256]
            st = stats[tt].double()
            w = torch.exp((x - st[:, :1]) * self.scale - st[:, 1:])
            f = (self.dlogp[tt].double() * self.scale)[:, None]
            one = torch.zeros_like(w).scatter_(1, self.targets[tt].long()[:, None], 1.0)
            exact = f * (one - w)
            # 4 u of the exponent's first part, 3 u of its second, ln 2 each, 3 u of the instruction, 3 u of products
            relative = math.log(2) * (4 * U * (x - st[:, :1]).abs() * c + 3 * U * st[:, 1:].abs() / math.log(2)) + 6 * U
            # (a weight of an exponent of -inf is 0 on either side)
            tol = f.abs() * (torch.where(w > 0, w * relative, 0.0) + 4 * U * one + 2.0 ** -120) + 2 * U * exact.abs()
            if self.dtype == BF16:
                tol = tol + 2.0 ** -8 * (exact.abs() + tol) + 2.0 ** -133   # half a step of the smallest numbers
            assert ((got[q[a:a + 256], :V].double() - exact).abs() <= tol).all()


BATCHES = [(1, 1, [1], 1), (3, 8, [1, 0, 3], 1), (0, 2, [16, 24, 24], 1), (1, 4, [5, 90, 1, 0, 4], 0),
           (3, 3, [101, 0, 13, 1, 66], 1), (3, 2, [17, 4], 0)]


@pytest.mark.parametrize("kind,P,lens,order", BATCHES)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("vocab,pad", [(1, 0), (2, 8), (7, 0), (8, 0), (9, 0), (31, 16), (255, 0), (256, 0), (1000, 24), (4099, 0),
                                       (50257, 40)])
def test_against_64_bits(cpt, cuda_device, kind, P, lens, order, dtype, vocab, pad):
    c = Case(cpt, Batch(cpt, kind, P, lens, order), vocab, dtype, scale=0.7 if vocab % 2 else 1.0, pad=pad)
    logp, stats = c.forward()
    c.check_forward(logp, stats)
    got = c.backward(stats)
    c.check_backward(got, stats)
    assert torch.equal(got, c.backward(stats, inplace=True))


# lengths of rows around every change of the work's division
@pytest.mark.parametrize("units", [1, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 512, 513, 1023, 1024, 1025, 2047,
                                   2048, 2049, 4095, 4096, 4097, 8192, 16384, 19648, 32768])
@pytest.mark.parametrize("tokens", [1, 3, 40, 700])
def test_every_row_length(cpt, cuda_device, units, tokens):
    for dtype, per in ((BF16, 8), (F32, 4)):
        c = Case(cpt, Batch(cpt, 1, 1, [tokens], 1), units * per - 1, dtype, share=0.9, seed=tokens)
        logp, stats = c.forward()
        c.check_forward(logp, stats)
        c.check_backward(c.backward(stats), stats)


@pytest.mark.parametrize("tokens,vocab", [(30000, 17), (5000, 500), (2000, 9001), (700, 157184)])
def test_many_tokens(cpt, cuda_device, tokens, vocab):
    c = Case(cpt, Batch(cpt, 3, 4, [tokens // 2, 0, 5, tokens - tokens // 2 - 5], 1), vocab, BF16)
    logp, stats = c.forward()
    c.check_forward(logp, stats)
    c.check_backward(c.backward(stats), stats)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("vocab", [40, 5000, 157184])
def test_masked_vocabulary_and_large_logits(cpt, cuda_device, dtype, vocab):
    """Columns at -inf or at the type's lowest value have no weight; logits of 10^4 lose nothing."""
    b = Batch(cpt, 1, 1, [24], 1)
    c = Case(cpt, b, vocab, dtype, share=1.0)
    x = c.logits.view(24, -1)
    x[:, :vocab] += 10000.0
    low = torch.finfo(dtype).min
    keep = torch.zeros(24, vocab, dtype=torch.bool, device="cuda")
    keep[torch.arange(24), c.targets.long()] = True
    keep[:, ::3] = True
    x[:12, :vocab][~keep[:12]] = float("-inf")
    x[12:, :vocab][~keep[12:]] = low
    # one logit alone, the first, the last
    x[0, :vocab] = float("-inf")
    x[0, c.targets[0]] = 3.0
    x[1, :vocab] = float("-inf")
    x[1, vocab - 1] = -2.0
    c.targets[1] = vocab - 1
    # a target that has no weight
    x[2, :vocab] = 1.0
    x[2, c.targets[2]] = float("-inf")
    logp, stats = c.forward()
    assert logp[0] == 0 and logp[1] == 0 and logp[2] == float("-inf")
    sound = torch.ones(24, dtype=torch.bool, device="cuda")
    sound[2] = False
    has = c.has
    c.has = has & sound
    kept_logp, kept_stats = logp.clone(), stats.clone()
    kept_logp[2], kept_stats[2] = 0, 0
    c.check_forward(kept_logp, kept_stats)
    c.has = has
    c.dlogp[:] = 1.0
    got = c.backward(stats)
    c.check_backward(got, stats)


@pytest.mark.parametrize("vocab", [40, 5000, 60000])
def test_nan_and_infinities_stay_in_their_row(cpt, cuda_device, vocab):
    b = Batch(cpt, 0, 2, [16, 8], 1)
    c = Case(cpt, b, vocab, BF16, share=1.0)
    x = c.logits.view(24, -1)
    rows = {2: float("nan"), 5: float("inf"), 9: float("-inf")}
    for r, v in rows.items():
        x[r, :vocab] = v if v == float("-inf") else x[r, :vocab]
        x[r, vocab // 2] = v
    logp, stats = c.forward()
    bad = torch.zeros(24, dtype=torch.bool, device="cuda")
    bad[b.tokens[list(rows)]] = True
    assert torch.equal(torch.isnan(logp), bad)
    # a gradient of 0 keeps such rows out of the gradient
    c.dlogp[bad] = 0.0
    c.check_backward(c.backward(stats), stats)


def test_gradient_against_differences(cpt, cuda_device):
    """Along random directions, in float32: step 2^-6, rounding of logp some 10 * 2^-24 over 2^-5, third derivatives of a
    log-sum at most 1 times the direction's cube."""
    b = Batch(cpt, 3, 2, [9, 4], 1)
    c = Case(cpt, b, 53, F32, scale=0.75, share=1.0)
    c.dlogp[:] = 1.0 + torch.arange(b.T, device="cuda") / 8
    logp, stats = c.forward()
    got = b.flat(c.backward(stats))[:, :53].double()
    keep = c.logits.clone()
    v = torch.randn(b.R, 53, device="cuda", generator=gen(5)).clamp(-2, 2)
    v[b.tokens < 0] = 0.0
    vals, step = [], 2.0 ** -6
    for s in (1, -1):
        b.flat(c.logits)[b.real, :53] = (b.flat(keep)[b.real, :53] + s * step * v[b.real])
        vals.append((c.forward()[0].double() * c.dlogp.double()).sum().item())
    numeric = (vals[0] - vals[1]) / (2 * step)
    exact = (got[b.real] * v[b.real].double()).sum().item()
    weight = c.dlogp.sum().item()
    assert abs(numeric - exact) <= weight * (200 * U / step + (2 * 0.75) ** 3 * step ** 2)


def test_the_same_bits_every_time_and_in_every_order(cpt, cuda_device):
    lens, V = [64, 32], 4099
    g = gen(3)
    x = torch.randn(96, 4104, device="cuda", generator=g).to(BF16)
    targets = torch.randint(0, V, (96,), device="cuda", generator=g).to(torch.int32)
    d = torch.randn(96, device="cuda", generator=g)
    seen = []
    for kind, P, order in [(1, 1, 0), (0, 2, 1), (3, 4, 1), (1, 3, 1)]:
        b = Batch(cpt, kind, P, lens, order)
        logits = torch.zeros(b.lead + (4104,), dtype=BF16, device="cuda")
        b.flat(logits)[b.real] = x[b.at]
        for _ in range(2):
            logp, stats, dx = torch.empty(96, device="cuda"), torch.empty(96, 2, device="cuda"), torch.empty_like(logits)
            cpt.cpt_token_logprob(b.plan, logits, targets, logp, stats, vocab=V, order=order)
            cpt.cpt_token_logprob_backward(b.plan, logits, targets, stats, d, dx, vocab=V, order=order)
            by_token = torch.empty(96, 4104, dtype=BF16, device="cuda")
            by_token[b.at] = b.flat(dx)[b.real]
            seen.append((logp, stats, by_token))
    for s in seen[1:]:
        assert all(torch.equal(a, r) for a, r in zip(seen[0], s))


def test_empty_batch(cpt, cuda_device):
    b = Batch(cpt, 3, 2, [0], 1)
    e = torch.empty(0, device="cuda")
    cpt.cpt_token_logprob(b.plan, torch.empty(2, 0, 16, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda"), e,
                          torch.empty(0, 2, device="cuda"))
    torch.cuda.synchronize()
