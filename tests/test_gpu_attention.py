"""Windowed attention with sinks and its gradient on the GPU, against dense
64-bit forms. The bounds of every error are derived in attention_ref."""
import math
import os
import re

import numpy as np
import pytest
import torch

import attention_ref as ref
from gpu_helpers import Guarded

pytestmark = pytest.mark.gpu


class Batch:
    """Inputs of one call in guarded buffers, and its outputs."""

    def __init__(self, cpt, layout, P, lens, Hq, Hk, D, window, sinks, seed=0, scale=None):
        self.cpt, self.P, self.window, self.sinks = cpt, P, window, sinks
        self.l2r, self.l2g, self.cu, self.cup = ref.local_rows(layout, P, lens)
        self.T, self.Tpad = int(self.cu[-1]), len(self.l2r)
        self.Hq, self.Hk, self.D = Hq, Hk, D
        self.scale = scale or D ** -0.5
        self.plan = cpt.cpt_plan_create(layout, P, self.cu.tolist(), self.T)
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(s, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
        self.q, self.dout = rnd(self.Tpad, Hq, D), rnd(self.Tpad, Hq, D)
        self.k, self.v = rnd(self.T, Hk, D), rnd(self.T, Hk, D)
        self.out = Guarded((self.Tpad, Hq, D), torch.bfloat16)
        self.lse = Guarded((Hq, self.Tpad), torch.float32)
        self.dq = Guarded((self.Tpad, Hq, D), torch.bfloat16)
        self.dk = [Guarded((self.Tpad, Hk, D), torch.bfloat16) for _ in range(P)]
        self.dv = [Guarded((self.Tpad, Hk, D), torch.bfloat16) for _ in range(P)]
        self.see = ref.visible(self.l2r, self.cu, self.T, window, sinks, "cuda")
        self.pad = torch.from_numpy(self.l2r < 0).cuda()

    def forward(self, stream=None):
        self.cpt.cpt_attention(self.plan, self.q, self.k, self.v, self.out.t, self.lse.t, self.scale, self.window,
                               self.sinks, stream=stream)

    def backward(self, workspace=None, stream=None):
        self.cpt.cpt_attention_backward(self.plan, self.q, self.k, self.v, self.out.t, self.lse.t, self.dout,
                                        self.dq.t, [x.t for x in self.dk], [x.t for x in self.dv], self.scale,
                                        self.window, self.sinks, workspace=workspace, stream=stream)

    def l2r_order(self):
        """Local rows in the order of the tokens they hold."""
        rows = np.flatnonzero(self.l2r >= 0)
        return torch.from_numpy(rows[np.argsort(self.l2r[rows])]).cuda()

    def workspace(self, extra=0):
        need = self.cpt.cpt_attention_backward_workspace_bytes(self.plan, self.Hq, self.Hk, self.D)
        return Guarded((need,), torch.uint8)

    def check_forward(self, q=None):
        assert self.out.bands_intact() and self.lse.bands_intact()
        out, lse, tol = ref.attention64(self.q if q is None else q, self.k, self.v, self.see, self.scale)
        got = self.out.t.double()
        assert torch.isfinite(got).all()
        assert ((got - out).abs() <= tol).all(), float(((got - out).abs() - tol).max())
        empty = lse == -math.inf
        assert torch.equal(self.lse.t == -math.inf, empty)
        diff = torch.where(empty, 0.0, (self.lse.t.double() - lse).abs())
        assert (diff <= ref.E32 + 2.0 ** -22 * lse.abs()).logical_or(empty).all(), float(diff.max())
        assert (got[empty.all(0)] == 0).all()

    def check_backward(self, q=None, dout=None, out=None):
        for x in [self.dq] + self.dk + self.dv:
            assert x.bands_intact()
        dq, tol, writers = ref.backward64(self.q if q is None else q, self.k, self.v,
                                          self.out.t if out is None else out,
                                          self.dout if dout is None else dout, self.see, self.scale, self.P)
        got = self.dq.t.double()
        assert torch.isfinite(got).all()
        assert ((got - dq).abs() <= tol).all(), float(((got - dq).abs() - tol).max())
        for r, pair in enumerate(writers):
            for name, buf, (want, tol) in zip(("dk", "dv"), (self.dk[r], self.dv[r]), pair):
                want, tol = (ref.to_padded(x, self.cu, self.cup, self.Tpad) for x in (want, tol))
                diff = (buf.t.double() - want).abs()
                assert torch.isfinite(diff).all(), (name, r)
                assert (diff <= tol).all(), (name, r, float((diff - tol).max()))


def both(cpt, *a, **kw):
    b = Batch(cpt, *a, **kw)
    b.forward()
    ws = b.workspace()
    b.backward(ws.t)
    torch.cuda.synchronize()
    assert ws.bands_intact()
    b.check_forward()
    b.check_backward()
    assert cpt.cpt_kernel_wait_timeouts() == 0
    return b


ODD = [1, 127, 128, 129, 0, 5, 300, 2, 0, 77]
EVEN = {P: [2 * P * m for m in (1, 17, 0, 40, 3)] for P in (1, 2, 3, 4, 8)}


@pytest.mark.parametrize("layout,P,lens", [
    (0, 4, [512]), (0, 2, EVEN[2]), (0, 8, EVEN[8]), (0, 1, [640]), (0, 3, EVEN[3]),
    (1, 1, ODD), (1, 4, ODD + [3]), (1, 3, [768]),
    (3, 1, ODD), (3, 4, ODD), (3, 8, [1, 1, 1, 3]), (3, 2, [701])])
@pytest.mark.parametrize("window,sinks", [(64, 4), (1 << 40, 0)])
def test_layouts(cpt, cuda_device, layout, P, lens, window, sinks):
    both(cpt, layout, P, lens, 2, 1, 64, window, sinks)


@pytest.mark.parametrize("window", [0, 1, 2, 127, 128, 129, 255, 400])
@pytest.mark.parametrize("sinks", [0, 1, 7, 128, 200])
def test_windows_and_sinks(cpt, cuda_device, window, sinks):
    both(cpt, 3, 2, [1, 390, 140, 260], 2, 2, 32, window, sinks, seed=window + sinks)


@pytest.mark.parametrize("Hq,Hk", [(1, 1), (3, 1), (4, 2), (6, 2), (5, 5), (8, 1)])
@pytest.mark.parametrize("D", [8, 64, 72, 128])
def test_heads(cpt, cuda_device, Hq, Hk, D):
    both(cpt, 3, 4, [150, 33, 301], Hq, Hk, D, 100, 3, seed=D + Hq)


@pytest.mark.parametrize("D", [16, 24, 32, 40, 48, 56, 80, 88, 96, 104, 112, 120])
def test_head_dims(cpt, cuda_device, D):
    both(cpt, 1, 2, [150, 34], 2, 1, D, 1000, 0, seed=D)


@pytest.mark.parametrize("layout,P,lens", [(3, 1, [1]), (3, 8, [1]), (1, 1, [0, 1, 0]), (3, 2, [0, 1, 1, 0]), (1, 8, [8])])
def test_shortest_batches(cpt, cuda_device, layout, P, lens):
    both(cpt, layout, P, lens, 2, 1, 64, 4, 1)


def test_empty_batch(cpt, cuda_device):
    plan = cpt.cpt_plan_create(1, 2, [0, 0], 0)
    z = torch.empty(0, 2, 64, device="cuda", dtype=torch.bfloat16)
    lse = torch.empty(2, 0, device="cuda")
    cpt.cpt_attention(plan, z, z, z, z, lse, 1.0, 4, 0)
    cpt.cpt_attention_backward(plan, z, z, z, z, lse, z, z, [z, z], [z, z], 1.0, 4, 0)
    torch.cuda.synchronize()


@pytest.mark.parametrize("window,sinks", [(300, 16), (4096, 0)])
def test_longer_documents(cpt, cuda_device, window, sinks):
    both(cpt, 0, 4, [2048, 1024], 2, 1, 128, window, sinks)
    both(cpt, 3, 3, [1999, 601, 450], 2, 2, 64, window, sinks)


@pytest.mark.parametrize("layout,P,lens,Hq,Hk,D,window,sinks", [
    (0, 1, [4096], 2, 1, 64, 64, 4),          # a tile of sinks that every row sees, among short ones
    (1, 2, [3000, 1096], 2, 1, 128, 70, 5),
    (0, 2, [4096], 1, 1, 128, 1 << 20, 0),    # the whole triangle of one head
    (3, 1, [3001], 4, 2, 80, 33, 130)])
def test_long_documents_with_few_heads(cpt, cuda_device, layout, P, lens, Hq, Hk, D, window, sinks):
    """Key tiles that many rows see are cut into parts; the sums of the parts are
    the same in every run."""
    b = both(cpt, layout, P, lens, Hq, Hk, D, window, sinks)
    first = [x.t.clone() for x in [b.dq] + b.dk + b.dv]
    ws = b.workspace()
    for _ in range(20):
        b.backward(ws.t)
    torch.cuda.synchronize()
    for x, y in zip([b.dq] + b.dk + b.dv, first):
        assert torch.equal(x.t, y)
    assert ws.bands_intact() and cpt.cpt_kernel_wait_timeouts() == 0


@pytest.mark.parametrize("layout,P,lens,Hq,Hk,D,window,sinks", [
    (0, 4, [32768], 8, 8, 128, 4096, 4),
    (1, 4, [20000, 3000, 777, 1, 9000, 22], 8, 2, 64, 1000, 5),
    (3, 3, [12000, 40, 9001], 6, 3, 80, 500, 0)])
def test_large_batches(cpt, cuda_device, layout, P, lens, Hq, Hk, D, window, sinks):
    """Batches that keep every SM busy for many tiles: the same bits in every run,
    whatever the workspace and the outputs held, and some rows and keys checked."""
    if layout == 1:
        lens = lens + [-sum(lens) % P]
    b = Batch(cpt, layout, P, lens, Hq, Hk, D, window, sinks)
    ws, first = b.workspace(), None
    for fill in (0x00, 0xFF, 0x7F, 0x3C):
        ws.t.fill_(fill)
        for x in [b.out, b.lse, b.dq] + b.dk + b.dv:
            x.t.view(torch.uint8).fill_(fill)
        b.forward()
        b.backward(ws.t)
        torch.cuda.synchronize()
        got = [x.t.clone() for x in [b.out, b.lse, b.dq] + b.dk + b.dv]
        first = first or got
        for x, y in zip(got, first):
            assert torch.equal(x, y)
    assert cpt.cpt_kernel_wait_timeouts() == 0
    rng = np.random.default_rng(3)
    rows = np.sort(rng.choice(np.flatnonzero(b.l2r >= 0), 96, replace=False))
    at = torch.from_numpy(rows).cuda()
    out, lse, tol, dq, dq_tol = ref.sampled_rows(b, rows)
    assert ((b.out.t[at].double() - out).abs() <= tol).all()
    assert ((b.lse.t[:, at].double() - lse).abs() <= ref.E32 + 2.0 ** -22 * lse.abs()).all()
    assert ((b.dq.t[at].double() - dq).abs() <= dq_tol).all()
    keys = np.unique(np.concatenate([rng.choice(b.T, 40), b.cu[:-1][np.diff(b.cu) > 0]]))
    for r, pair in enumerate(ref.sampled_keys(b, keys)):
        for buf, (want, bound) in zip((b.dk[r], b.dv[r]), pair):
            diff = (ref_raw(b, buf.t.double())[torch.from_numpy(keys).cuda()] - want).abs()
            assert (diff <= bound).all(), (r, float((diff - bound).max()))


@pytest.mark.parametrize("Hq,Hk", [(52, 26), (51, 17), (56, 7), (51, 51)])
@pytest.mark.parametrize("D,window,sinks", [
    (8, 100, 3), (48, 127, 0), (64, 1, 0), (64, 200, 130), (64, 1 << 31, 0), (72, 60, 2), (120, 129, 1), (128, 0, 4),
    (128, 90, 7), (128, 1 << 31, 0)])
def test_many_heads(cpt, cuda_device, Hq, Hk, D, window, sinks):
    """More query tiles than SMs: items of two heads, or of two tiles of one."""
    both(cpt, 3, 3, [1, 250, 130, 0, 7, 383], Hq, Hk, D, window, sinks)


@pytest.mark.parametrize("D", [16, 64, 80, 128])
@pytest.mark.parametrize("window,sinks", [(1 << 31, 0), (700, 5), (1, 300)])
def test_few_heads(cpt, cuda_device, D, window, sinks):
    """No more query tiles than SMs: an item's key tiles are shared out and joined, again and again the same."""
    b = both(cpt, 0, 2, [2048, 12, 1500], 2, 1, D, window, sinks)
    first = [x.t.clone() for x in (b.out, b.lse)]
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for i in range(20):
        flush.fill_(i)
        b.forward()
        torch.cuda.synchronize()
        assert torch.equal(b.out.t, first[0]) and torch.equal(b.lse.t, first[1])
    assert cpt.cpt_kernel_wait_timeouts() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [129, 257, 385])
def test_few_key_tiles_from_a_cold_cache(cpt, cuda_device, D, window):
    """Every row tile sees two, three or four key tiles, and what is loaded arrives late and out of
    order: no tile may make way for the next item's before it has been read."""
    b = Batch(cpt, 0, 1, [8192], 8, 4, D, window, 0)
    ws, first = b.workspace(), None
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")   # twice the L2 cache
    results = [b.out, b.lse, b.dq] + b.dk + b.dv
    for i in range(30):
        for x in results:
            x.t.view(torch.uint8).fill_(0xFF)
        flush.fill_(i)
        b.forward()
        flush.fill_(i)
        b.backward(ws.t)
        torch.cuda.synchronize()
        got = [x.t.clone() for x in results]
        first = first or got
        for x, y in zip(got, first):
            assert torch.equal(x, y), i
    assert cpt.cpt_kernel_wait_timeouts() == 0
    rows = np.arange(0, b.T, 67)
    at = torch.from_numpy(rows).cuda()
    out, lse, tol, dq, dq_tol = ref.sampled_rows(b, rows)
    assert ((b.out.t[at].double() - out).abs() <= tol).all()
    assert ((b.dq.t[at].double() - dq).abs() <= dq_tol).all()


@pytest.mark.parametrize("D", [64, 128])
def test_runs_of_rows_that_see_nothing(cpt, cuda_device, D):
    """Documents of one token leave the later ranks hundreds of padding rows in a run: row tiles
    that see nothing follow one another, between others that do."""
    lens = [1500] + [1] * 900 + [700] + [1] * 900
    b = Batch(cpt, 3, 4, lens, 12, 4, D, 300, 3)
    ws, first = b.workspace(), None
    results = [b.out, b.lse, b.dq] + b.dk + b.dv
    for _ in range(10):
        for x in results:
            x.t.view(torch.uint8).fill_(0xFF)
        b.forward()
        b.backward(ws.t)
        torch.cuda.synchronize()
        got = [x.t.clone() for x in results]
        first = first or got
        for x, y in zip(got, first):
            assert torch.equal(x, y)
    assert cpt.cpt_kernel_wait_timeouts() == 0
    empty = torch.from_numpy(np.flatnonzero(b.l2r < 0)).cuda()
    assert (b.out.t[empty] == 0).all() and (b.lse.t[:, empty] == -math.inf).all() and (b.dq.t[empty] == 0).all()
    rows = np.flatnonzero(b.l2r >= 0)[::41]
    at = torch.from_numpy(rows).cuda()
    out, lse, tol, dq, dq_tol = ref.sampled_rows(b, rows)
    assert ((b.out.t[at].double() - out).abs() <= tol).all()
    assert ((b.dq.t[at].double() - dq).abs() <= dq_tol).all()


def test_many_short_documents(cpt, cuda_device):
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(0, 40, 90)]
    both(cpt, 3, 4, lens, 2, 1, 64, 16, 2)
    lens[-1] += -sum(lens) % 4
    both(cpt, 1, 4, lens, 2, 1, 64, 1 << 31, 0)


@pytest.mark.parametrize("scale", [1e-3, 1.0, 4.0])
def test_scales(cpt, cuda_device, scale):
    # scores of up to some 100 * scale: the binary32 slack of a weight grows with them
    b = Batch(cpt, 0, 2, [256], 2, 1, 64, 100, 2, scale=scale)
    b.forward()
    b.backward()
    slack = max(1.0, 8 * scale)   # |s| grows by scale * sqrt(D) = 8 scale over unit scores
    e, ref.E32 = ref.E32, ref.E32 * slack
    try:
        b.check_forward()
        b.check_backward()
    finally:
        ref.E32 = e


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("score", [80.0, 88.5, 95.0])
def test_weights_that_leave_binary32(cpt, cuda_device, D, score):
    """Two late keys score 80 to 95 above all others: a weight relative to the first tile's, or only
    the sum of two, is past the largest binary32, with small V the product is not."""
    b = Batch(cpt, 0, 1, [512], 2, 1, D, 512, 0, scale=1.0)
    b.q.zero_()
    b.q[..., 0] = 8.0
    b.k.zero_()
    b.k[300:302, :, 0] = score / 8   # a bf16 value
    b.v.copy_((torch.rand(b.v.shape, device="cuda") / 8).to(torch.bfloat16))
    b.forward()
    out, v = b.out.t.reshape(b.Tpad, 2, D)[b.l2r_order()].double(), b.v[:, 0].double()
    mean = torch.cumsum(v, 0) / torch.arange(1, 513, device="cuda")[:, None]
    late = (v[300] + v[301]) / 2
    # equal weights; from key 300 on the others weigh exp(-80) at most. Weights and out are rounded, and sums of
    # n binary32 terms are off by n E at most
    for want, rows in ((mean[:300], out[:300]), (v[300:301], out[300:301]), (late.expand(211, D), out[301:])):
        assert ((rows - want[:, None]).abs() <= (2 * ref.U + 512 * 2.0 ** -24) * want[:, None].abs()).all()
    lse = b.lse.t[:, b.l2r_order()].double()
    assert ((lse[:, 301:] - score - math.log(2)).abs() <= 1e-4).all()   # 2^-22 of 95, and the exponentials
    b.backward()
    assert b.dq.t.isfinite().all() and all(x.t.isfinite().all() for x in b.dk + b.dv)


def test_first_row_of_every_document_copies_v(cpt, cuda_device):
    """A row that sees one key alone has out = v, bit for bit."""
    b = Batch(cpt, 3, 4, [1, 50, 129, 3], 2, 1, 64, 1, 0)
    b.forward()
    real = ~b.pad
    want = b.v[torch.from_numpy(b.l2r).cuda()[real]].repeat_interleave(2, 1)
    assert torch.equal(b.out.t[real], want)


def test_gradients_against_differences(cpt, cuda_device):
    """Directional derivatives of sum(out * dout) by central differences of the
    64-bit form agree with the kernels' gradients."""
    b = both(cpt, 3, 2, [60, 33, 140], 4, 2, 64, 50, 2)
    g = torch.Generator(device="cuda").manual_seed(9)
    dk = sum(ref_raw(b, x.t.double()) for x in b.dk)
    dv = sum(ref_raw(b, x.t.double()) for x in b.dv)
    do = torch.where(b.pad[:, None, None], 0.0, b.dout.double())
    for name, grad in (("q", b.dq.t.double()), ("k", dk), ("v", dv)):
        x = getattr(b, name).double()
        d = torch.randn(x.shape, device="cuda", generator=g, dtype=torch.float64)
        h = 1e-4
        f = []
        for sgn in (1, -1):
            args = {n: getattr(b, n).double() for n in "qkv"}
            args[name] = x + sgn * h * d
            out, _, _ = ref.attention64(args["q"], args["k"], args["v"], b.see, b.scale)
            f.append((out * do).sum())
        want = (f[0] - f[1]) / (2 * h)
        got = (grad * d).sum()
        # every element of the gradient is off by a few roundings (independent signs); the
        # difference's own error is of order h^2
        assert abs(want - got) <= 8 * ref.U * (grad * d).square().sum().sqrt() + 1e-4 * abs(want) + 1e-2, name


def ref_raw(b, x):
    """Padded global rows back in raw order."""
    at = np.arange(b.T) + np.repeat(b.cup[:-1] - b.cu[:-1], np.diff(b.cu))
    return x[torch.from_numpy(at).cuda()]


# few tiles of query rows, or enough of them for the kernel of two tiles (two heads that share keys, or not)
@pytest.mark.parametrize("heads", [(2, 1), (40, 20), (44, 44)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("D", [64, 128])
def test_infinities_and_nan_stay_where_they_are_seen(cpt, cuda_device, bad, D, heads):
    """K and V rows of one document, a key past its window and the last key
    of a document hold NaN or infinities: rows that do not see them are as if
    they were finite, in both directions."""
    lens, W, S = [100, 90, 260], 70, 2
    b = Batch(cpt, 3, 2, lens, *heads, D, W, S)
    spoiled = [99, 120, 190 + 40]          # raw tokens: last of document 0, inside 1, past sinks of 2
    k, v = b.k, b.v
    b.k, b.v = k.clone(), v.clone()
    b.k[spoiled] = bad
    b.v[spoiled] = bad
    hit = b.see[:, spoiled].any(1)
    assert hit.any() and (~hit).any()
    b.forward()
    want, lse, tol = ref.attention64(b.q, k, v, b.see, b.scale)
    real = ~hit & ~b.pad
    assert ((b.out.t.double() - want).abs() <= tol)[~hit].all()
    assert ((b.lse.t.double() - lse).abs()[:, real] <= ref.E32 + 2.0 ** -22 * lse.abs()[:, real]).all()
    # the gradient: rows that saw none of it, and keys that no such row sees
    b.out.t.copy_(want)
    b.lse.t.copy_(lse)
    b.backward()
    dq, tol, writers = ref.backward64(b.q, k, v, b.out.t, b.dout, b.see, b.scale, 2)
    assert ((b.dq.t.double() - dq).abs() <= tol)[~hit].all()
    free = ~b.see[hit].any(0)
    free[spoiled] = False
    assert free.any()
    for r, pair in enumerate(writers):
        for buf, (want, tol) in zip((b.dk[r], b.dv[r]), pair):
            assert ((ref_raw(b, buf.t.double()) - want).abs() <= tol)[free].all()


@pytest.mark.parametrize("heads", [(4, 2), (40, 20), (39, 39)])
@pytest.mark.parametrize("D", [64, 128])
def test_garbage_in_padding_rows_is_not_used(cpt, cuda_device, D, heads):
    b = Batch(cpt, 3, 4, [3, 1, 150, 47, 9], *heads, D, 60, 2)
    q, dout = b.q.clone(), b.dout.clone()
    q[b.pad] = 0
    dout[b.pad] = 0
    b.q[b.pad] = float("nan")
    b.dout[b.pad] = float("inf")
    b.forward()
    b.check_forward(q=q)
    assert (b.out.t[b.pad] == 0).all() and (b.lse.t[:, b.pad] == -math.inf).all()
    out = b.out.t.clone()
    b.out.t[b.pad] = float("nan")
    b.lse.t[:, b.pad] = float("nan")
    b.backward()
    b.check_backward(q=q, dout=dout, out=out)
    assert (b.dq.t[b.pad] == 0).all()


def test_repeated_calls_give_the_same_bits(cpt, cuda_device):
    b = Batch(cpt, 3, 4, [700, 33, 900, 1], 4, 2, 128, 500, 5)
    b.forward()
    b.backward()
    first = [x.t.clone() for x in [b.out, b.lse, b.dq] + b.dk + b.dv]
    for _ in range(3):
        for x in [b.out, b.lse, b.dq] + b.dk + b.dv:
            x.t.fill_(7.0)
        b.forward()
        b.backward()
        for x, y in zip([b.out, b.lse, b.dq] + b.dk + b.dv, first):
            assert torch.equal(x.t, y)


def test_streams_and_graphs(cpt, cuda_device):
    """On another stream, captured and replayed, two graphs at once with a
    workspace each."""
    batches = [Batch(cpt, 3, 4, [300, 33, 129], 4, 2, 64, 100, 3, seed=s) for s in (1, 2)]
    wants = []
    for b in batches:
        b.forward()
        b.backward()
        wants.append([x.t.clone() for x in [b.out, b.lse, b.dq] + b.dk + b.dv])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in batches]
    spaces = [b.workspace() for b in batches]

    def clear():
        for b in batches:
            for x in [b.out, b.lse, b.dq] + b.dk + b.dv:
                x.t.zero_()
        torch.cuda.synchronize()

    def check():
        torch.cuda.synchronize()
        for b, want in zip(batches, wants):
            for x, y in zip([b.out, b.lse, b.dq] + b.dk + b.dv, want):
                assert torch.equal(x.t, y)

    clear()
    for b, s, w in zip(batches, streams, spaces):
        b.forward(stream=s)
        b.backward(w.t, stream=s)
    check()
    graphs = []
    for b, w in zip(batches, spaces):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            b.forward()
            b.backward(w.t)
        graphs.append(graph)
    for _ in range(2):
        clear()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        check()


def test_calls_in_a_row_and_on_two_streams(cpt, cuda_device):
    """Inputs and outputs change hands between calls without a synchronisation, on one stream and
    on two at once: the same bits as with the device waited for after every step."""
    shapes = [(0, 4, [4096], 6, 6, 128, 1500, 4), (1, 4, [1000, 3, 2005, 988], 8, 2, 64, 300, 2)]
    batches = [Batch(cpt, *s) for s in shapes]
    spaces = [b.workspace() for b in batches]
    inputs = [[(torch.randn_like(b.q), torch.randn_like(b.k), torch.randn_like(b.dout)) for _ in range(6)]
              for b in batches]

    def run(wait, streams):
        got = [[], []]
        for i in range(6):
            for b, w, s, given, res in zip(batches, spaces, streams, inputs, got):
                with torch.cuda.stream(s):
                    for to, x in zip((b.q, b.k, b.dout), given[i]):
                        to.copy_(x)
                    for step in (b.forward, lambda: b.backward(w.t)):
                        step()
                        if wait:
                            torch.cuda.synchronize()
                    res.append([x.t.clone() for x in [b.out, b.lse, b.dq] + b.dk + b.dv])
                    b.out.t.zero_()
                    b.lse.t.zero_()
        torch.cuda.synchronize()
        return got

    torch.cuda.synchronize()
    one = torch.cuda.Stream()
    want = run(True, [one, one])
    for streams in ([one, one], [one, torch.cuda.Stream()], [torch.cuda.default_stream()] * 2):
        for b, x, y in zip(batches, run(False, streams), want):
            for i, (u, v) in enumerate(zip(x, y)):
                for s, t in zip(u, v):
                    assert torch.equal(s, t), i
    assert cpt.cpt_kernel_wait_timeouts() == 0


def test_refusals_on_the_device(cpt, cuda_device):
    b = Batch(cpt, 0, 2, [64], 2, 1, 64, 16, 0)
    ok = dict(q=b.q, k=b.k, v=b.v, out=b.out.t, lse=b.lse.t, scale=1.0, window=4, sinks=0)

    def status(**kw):
        with pytest.raises(cpt.CptError) as e:
            cpt.cpt_attention(b.plan, **{**ok, **kw})
        return e.value.status

    f = lambda t: t.float()  # noqa: E731
    assert status(q=f(b.q), k=f(b.k), v=f(b.v), out=f(b.out.t)) == cpt.CPT_ERR_UNSUPPORTED
    assert status(scale=0.0) == cpt.CPT_ERR_INVALID_ARG
    assert status(scale=-1.0) == cpt.CPT_ERR_INVALID_ARG
    assert status(scale=float("nan")) == cpt.CPT_ERR_INVALID_ARG
    assert status(window=-1) == cpt.CPT_ERR_INVALID_ARG
    assert status(sinks=-1) == cpt.CPT_ERR_INVALID_ARG
    assert status(out=b.q) == cpt.CPT_ERR_ALIAS
    assert status(k=b.k.cpu()) == cpt.CPT_ERR_DEVICE
    ws = b.workspace().t

    def back(**kw):
        a = dict(q=b.q, k=b.k, v=b.v, out=b.out.t, lse=b.lse.t, dout=b.dout, dq=b.dq.t,
                 dk_writers=[x.t for x in b.dk], dv_writers=[x.t for x in b.dv], scale=1.0, window=4, sinks=0,
                 workspace=ws)
        with pytest.raises(cpt.CptError) as e:
            cpt.cpt_attention_backward(b.plan, **{**a, **kw})
        return e.value.status

    assert back(workspace=ws[:-1]) == cpt.CPT_ERR_WORKSPACE
    assert back(workspace=ws[16:]) == cpt.CPT_ERR_WORKSPACE
    assert back(dq=b.q) == cpt.CPT_ERR_ALIAS
    assert back(dv_writers=[b.dv[0].t, b.dk[1].t]) == cpt.CPT_ERR_ALIAS
    assert back(window=-1) == cpt.CPT_ERR_INVALID_ARG
    torch.cuda.synchronize()


def test_a_whole_step(cpt, cuda_device):
    """Rotate, attend, differentiate, return and turn back, as a step uses the
    calls, against autograd in 64 bits over the whole documents."""
    lens, P, Hq, Hk, D, W, S = [130, 0, 57, 300], 4, 4, 2, 64, 90, 3
    b = Batch(cpt, 3, P, lens, Hq, Hk, D, W, S)
    T, Tpad = b.T, b.Tpad
    g = torch.Generator(device="cuda").manual_seed(4)
    freq, axis = [10000.0 ** (-i / 32) for i in range(32)], [i * 3 // 32 for i in range(32)]
    pos = torch.randint(0, 5000, (3, T), dtype=torch.int32, device="cuda", generator=g)
    q0, k0 = (torch.randn(T, h, D, device="cuda", generator=g).to(torch.bfloat16) for h in (Hq, Hk))
    rot = cpt.cpt_rotary_create(D, freq, axis, 3)
    kr = torch.empty_like(k0)
    cpt.cpt_rotary_apply(rot, b.plan, [q0], [b.q], pos)
    cpt.cpt_rotary_apply(rot, b.plan, [k0], [kr], pos, cpt.CPT_ORDER_GLOBAL, cpt.CPT_ORDER_GLOBAL)
    b.k = kr
    b.forward()
    b.check_forward()
    b.backward()
    b.check_backward()
    own = [[torch.empty(Tpad // P, Hk, D, device="cuda", dtype=torch.bfloat16) for _ in range(P)] for _ in range(2)]
    cpt.cpt_grad_return(b.plan, [x.t for x in b.dk], [x.t for x in b.dv], own[0], own[1])
    gq, gk = torch.empty_like(q0), torch.empty_like(k0)
    gv = torch.empty_like(k0)
    dko, dvo = torch.cat(own[0]), torch.cat(own[1])
    L, G = cpt.CPT_ORDER_LOCAL, cpt.CPT_ORDER_GLOBAL
    cpt.cpt_rotary_apply(rot, b.plan, [b.dq.t, dko], [gq, gk], pos, L, G, True)
    cpt.cpt_restore(b.plan, [dvo], [gv])

    x = [t.double().cpu().requires_grad_() for t in (q0, k0, b.v)]
    theta = torch.stack([pos[a].double().cpu() * f for a, f in zip(axis, freq)], 1)[:, None, :]
    turn = torch.polar(torch.ones_like(theta), theta)

    def rotate(t):
        z = torch.complex(t[..., :32], t[..., 32:]) * turn
        return torch.cat([z.real, z.imag], -1)

    see = ref.visible(np.arange(T), b.cu, T, W, S, "cpu")
    s = torch.einsum("ihd,jhd->hij", rotate(x[0]), rotate(x[1]).repeat_interleave(Hq // Hk, 1)) * b.scale
    p = torch.softmax(s.masked_fill(~see, -math.inf), -1)
    out = torch.einsum("hij,jhd->ihd", p, x[2].repeat_interleave(Hq // Hk, 1))
    real = torch.from_numpy(b.l2r[b.l2r >= 0])
    do = torch.zeros(T, Hq, D, dtype=torch.float64)
    do[real] = b.dout.double().cpu()[torch.from_numpy(b.l2r >= 0)]
    (out * do).sum().backward()
    got_out = torch.empty(T, Hq, D, dtype=torch.float64)
    got_out[real] = b.out.t.double().cpu()[torch.from_numpy(b.l2r >= 0)]
    # by norms: rotated q and k, p or ds, the output, the sum and the rotation back are rounded
    # to bf16 once each, at most U of their values
    for got, want in ((got_out, out.detach()), (gq, x[0].grad), (gk, x[1].grad), (gv, x[2].grad)):
        rel = (got.double().cpu() - want).norm() / want.norm()
        assert rel <= 6 * ref.U, float(rel)


def test_readme_example_of_the_layer(cpt, cuda_device):
    """The README's second example runs as written, after its first; rows checked against 64 bits."""
    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")) as f:
        text = f.read()
    env = {}
    for kind in ("python", "py"):
        exec(compile(re.search(rf"```{kind}\n(.*?)```", text, flags=re.S).group(1), "README.md", "exec"), env)
    torch.cuda.synchronize()
    S, H, KV, D = env["S"], env["H"], env["KV"], env["D"]
    l2g = torch.empty(S, dtype=torch.int32, device="cuda")
    cpt.cpt_index_map(env["plan"], l2g, None)
    freq = torch.tensor([10000.0 ** (-i / 64) for i in range(64)], dtype=torch.float64, device="cuda")

    def turn(x, at):
        theta = at.double()[:, None, None] * freq
        z = torch.complex(x[..., :64].double(), x[..., 64:].double()) * torch.polar(torch.ones_like(theta), theta)
        return torch.cat([z.real, z.imag], -1)

    for row in (0, 1, 40000, 131071, 262143):
        i = int(l2g[row])
        keys = torch.arange(S, device="cuda")
        keys = keys[(keys <= i) & ((i - keys < env["window"]) | (keys < env["sinks"]))]
        q = turn(env["q"][i:i + 1], torch.tensor([i], device="cuda"))[0]
        k = turn(env["k"][keys], keys).repeat_interleave(H // KV, 1)
        p = torch.softmax(torch.einsum("hd,jhd->hj", q, k) * env["scale"], 1)
        want = torch.einsum("hj,jhd->hd", p, env["v"][keys].double().repeat_interleave(H // KV, 1))
        # by norms: rotated q and k move the scores, and p and out are rounded, by at most U each
        got = env["out"].view(S, H, D)[row].double()
        assert (got - want).norm() <= 6 * ref.U * want.norm(), row
    # the turn back undoes the turn: the same norms, up to the two roundings
    a, b = env["dq"].double().norm(), env["dq_global"].double().norm()
    assert abs(a - b) <= 2 * ref.U * a
    assert env["dk_turned"].isfinite().all() and env["dv"].isfinite().all()
