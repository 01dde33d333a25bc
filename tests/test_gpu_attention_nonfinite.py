"""Infinities and NaN in the attention layer: which outputs they reach, and what
such a call costs."""
import math

import pytest
import torch

import attention_ref as ref
from test_gpu_attention import Batch, ref_raw

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")
HEADS = [(2, 1), (40, 20)]      # few query tiles, or many


def _batch(cpt, heads, D=64):
    return Batch(cpt, 3, 2, [100, 90, 260], *heads, D, 70, 2)


def _same_but(got, want, tol, nan):
    """NaN exactly where `nan` holds, within the bound elsewhere."""
    assert torch.equal(got.isnan(), nan)
    assert ((got - want).abs() <= tol)[~nan].all()


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("where", ["q", "k", "v", "dout"])
def test_nan_reaches_what_sees_it(cpt, cuda_device, where, heads):
    """One NaN (element 5 of one head's row) reaches exactly the outputs that the formulas carry it to."""
    b = _batch(cpt, heads)
    clean = {n: getattr(b, n).clone() for n in ("q", "k", "v", "dout")}
    token = 150                                       # inside document 1
    row = int((torch.from_numpy(b.l2r) == token).nonzero()[0, 0])
    at = token if where in "kv" else row
    getattr(b, where)[at, 0, 5] = NAN
    b.forward()
    b.backward()
    out, lse, tol = ref.attention64(clean["q"], clean["k"], clean["v"], b.see, b.scale)
    dq, dq_tol, writers = ref.backward64(clean["q"], clean["k"], clean["v"], out, clean["dout"], b.see, b.scale, b.P)
    G = b.Hq // b.Hk
    heads_hit = torch.zeros(b.Hq, dtype=torch.bool, device="cuda")
    heads_hit[:G if where in "kv" else 1] = True
    rows_hit = b.see[:, token] if where in "kv" else torch.arange(b.Tpad, device="cuda") == row
    hit = rows_hit[:, None] & heads_hit[None]        # (row, head) that meets the NaN
    one = torch.zeros(b.D, dtype=torch.bool, device="cuda")
    one[5] = True
    none = torch.zeros_like(hit)
    whole = {"q": hit, "k": hit, "v": none, "dout": none}[where]        # all of out, and lse
    part = {"q": none, "k": none, "v": hit, "dout": none}[where]        # element 5 of out
    nan_out = whole[..., None] | (part[..., None] & one)
    _same_but(b.out.t.double(), out, tol, nan_out)
    assert torch.equal(b.lse.t.isnan(), whole.t())
    ok = ~whole.t() & (lse != -math.inf)
    assert ((b.lse.t.double() - lse).abs() <= ref.E32 + 2.0 ** -22 * lse.abs())[ok].all()
    # dq: delta or the weights of the row are NaN. The kernel's delta comes from its own out, the
    # bound's from the exact one: they differ by the rounding of out
    slack = 2 * ref.U * (clean["dout"].double().abs() * out.abs()).sum(-1, keepdim=True)
    mag = b.scale * clean["k"].double().abs().amax()
    _same_but(b.dq.t.double(), dq, dq_tol + slack * mag, hit[..., None].expand(-1, -1, b.D))
    Tp = b.Tpad // b.P
    for r, ((dk, _), (dv, dv_tol)) in enumerate(writers):
        rows = slice(r * Tp, (r + 1) * Tp)
        # keys of the hit rows of this rank, by kv head
        keys = (b.see[rows].t().double() @ hit[rows].double()) > 0                 # [T, Hq]
        keys = keys.reshape(b.T, b.Hk, G).any(-1)
        got_k, got_v = ref_raw(b, b.dk[r].t.double()), ref_raw(b, b.dv[r].t.double())
        assert torch.equal(got_k.isnan(), keys[..., None].expand(-1, -1, b.D))
        nan_v = {"q": keys[..., None].expand(-1, -1, b.D), "k": keys[..., None].expand(-1, -1, b.D),
                 "v": torch.zeros_like(got_v, dtype=torch.bool), "dout": keys[..., None] & one}[where]
        _same_but(got_v, dv, dv_tol, nan_v)
        rest = ~keys[..., None].expand(-1, -1, b.D)
        assert got_k[rest].isfinite().all()
        assert ((got_k - dk).abs() <= 16 * ref.U * dk.abs().amax())[rest].all()
    assert cpt.cpt_kernel_wait_timeouts() == 0


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("bad", [INF, -INF])
def test_infinity_in_v(cpt, cuda_device, bad, heads):
    b = _batch(cpt, heads)
    clean = b.v.clone()
    b.v[150, 0, 5] = bad
    b.forward()
    out, lse, tol = ref.attention64(b.q, b.k, clean, b.see, b.scale)
    got = b.out.t.double()
    hit = b.see[:, 150][:, None] & (torch.arange(b.Hq, device="cuda") < b.Hq // b.Hk)[None]
    assert (got[hit][:, 5] == bad).all()          # weights are above zero, the rest is finite
    got[..., 5] = torch.where(hit, out[..., 5], got[..., 5])
    assert ((got - out).abs() <= tol).all()
    ok = lse != -math.inf
    assert ((b.lse.t.double() - lse).abs() <= ref.E32 + 2.0 ** -22 * lse.abs())[ok].all()


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("bad", [INF, -INF])
def test_infinity_in_k(cpt, cuda_device, bad, heads):
    """A score of +inf makes a row NaN, one of -inf hides the key."""
    b = _batch(cpt, heads)
    clean = b.k.clone()
    b.k[150, 0, 5] = bad
    b.forward()
    hit = b.see[:, 150][:, None] & (torch.arange(b.Hq, device="cuda") < b.Hq // b.Hk)[None]
    up = (b.q[..., 5].double() * bad) > 0
    see = b.see[None].repeat(b.Hq, 1, 1)
    see[:, :, 150] &= ~(hit & ~up).t()
    out, lse, tol = ref.attention64(b.q, clean, b.v, see, b.scale)
    nan = hit & up
    _same_but(b.out.t.double(), out, tol, nan[..., None].expand(-1, -1, b.D))
    assert torch.equal(b.lse.t.isnan(), nan.t())
    ok = ~nan.t() & (lse != -math.inf)
    assert ((b.lse.t.double() - lse).abs() <= ref.E32 + 2.0 ** -22 * lse.abs())[ok].all()


def _ms(call):
    times = []
    for _ in range(4):
        a, z = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        call()
        z.record()
        z.synchronize()
        times.append(a.elapsed_time(z))
    return min(times[1:])


class Long(Batch):
    """One long document under the whole triangle, without the dense masks."""

    def __init__(self, cpt, T=16384, H=4, D=64):
        self.cpt, self.P, self.window, self.sinks, self.scale = cpt, 4, T, 0, D ** -0.5
        self.plan = cpt.cpt_plan_create(0, 4, [0, T], T)
        self.T = self.Tpad = T
        self.Hq = self.Hk = H
        self.D = D
        bf = dict(device="cuda", dtype=torch.bfloat16)
        self.q, self.dout, self.k, self.v = (torch.randn(T, H, D, **bf) for _ in range(4))

        class Plain:
            def __init__(self, t):
                self.t = t

        self.out, self.dq = (Plain(torch.empty(T, H, D, **bf)) for _ in range(2))
        self.lse = Plain(torch.empty(H, T, device="cuda"))
        self.dk, self.dv = ([Plain(torch.empty(T, H, D, **bf)) for _ in range(4)] for _ in range(2))


@pytest.mark.parametrize("where,at", [("k", 0), ("q", 8191), ("v", 0), ("dout", 8191), ("all", 0)])
def test_a_step_with_nan_is_no_slower_by_much(cpt, cuda_device, where, at):
    """A NaN (a row of Q or dO, the first K, one element of the first V, the first row of all four) that reaches
    every row behind or every key before: an output that is NaN whatever else comes is not computed again key
    by key. Held to four times the time of the call without (and half a millisecond); computed again, these calls took
    24 to 1000 times it. (Rows that share a tile of 128 keys with a hidden NaN in V are computed again, slowly: not here.)"""
    b = Long(cpt)
    ws = torch.empty(cpt.cpt_attention_backward_workspace_bytes(b.plan, b.Hq, b.Hk, b.D), dtype=torch.uint8,
                     device="cuda")

    def back():
        b.backward(ws)

    forward, backward = _ms(b.forward), _ms(back)
    if where == "all":
        for x in (b.q, b.k, b.v, b.dout):
            x[at] = NAN
    elif where == "v":
        b.v[at, :, 5] = NAN
    else:
        getattr(b, where)[at] = NAN
    slow_forward, slow_backward = _ms(b.forward), _ms(back)
    print(f"{where} {at}: forward {forward:.3f} -> {slow_forward:.3f} ms, backward {backward:.3f} -> {slow_backward:.3f}")
    assert slow_forward <= 4 * forward + 0.5
    assert slow_backward <= 4 * backward + 0.5
