"""The calls on token rows together, as a training step makes them; in graphs, on streams, over 2^32 elements; and their
refusals through the C entries."""
import ctypes
import os
import re
import subprocess
import sys

import numpy as np
import pytest
import torch

from token_rows_ref import U, Batch, close, factor, gen, residual_norm

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


class Step:
    """Two blocks' ends, the logits of a small vocabulary, a policy loss and everything back, in float32."""

    def __init__(self, cpt, b, C=96, V=113, seed=0):
        g = gen(seed)
        r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
        self.cpt, self.b, self.C, self.V = cpt, b, C, V
        lead = b.lead
        self.x, self.h = r(*lead, C), [r(*lead, C) for _ in range(2)]
        self.gate = r(b.n, C)
        self.post, self.pre = [1 + 0.1 * r(C) for _ in range(2)], [1 + 0.1 * r(C) for _ in range(2)]
        self.head = torch.zeros(C, 120, device="cuda")
        self.head[:, :V] = r(C, V) / C ** 0.5
        targets = torch.randint(0, V, (b.T,), device="cuda", generator=g).to(torch.int32)
        ends = torch.tensor(np.cumsum(b.lens)[np.asarray(b.lens) > 0] - 1, device="cuda")
        targets[ends] = -1                         # a document's last token has none
        self.targets, self.mask = targets, targets >= 0
        self.adv = r(b.n)
        self.old, self.ref = -4.7 + 0.2 * r(b.T), -4.7 + 0.2 * r(b.T)
        self.rng = torch.tensor([99 + seed, 0], dtype=torch.int64, device="cuda")
        e = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
        self.y, self.n = [e(*lead, C) for _ in range(2)], [e(*lead, C) for _ in range(2)]
        self.logits, self.dlogits = e(*lead, 120), e(*lead, 120)
        self.logp, self.stats, self.terms, self.dlogp = e(b.T), e(b.T, 2), e(b.n, 4), e(b.T)
        self.dn, self.dx = e(*lead, C), [e(*lead, C) for _ in range(2)]
        self.dh, self.dgate = [e(*lead, C) for _ in range(2)], e(b.n, C)
        self.dpost, self.dpre = [e(C) for _ in range(2)], [e(C) for _ in range(2)]
        need = cpt.cpt_residual_norm_backward_workspace_bytes(b.plan, C, F32)
        self.work = torch.empty(max(256, need), dtype=torch.uint8, device="cuda")

    def options(self, i):
        o = dict(post_weight=self.post[i], pre_weight=self.pre[i], scale=0.8, p=0.2, rng=self.rng, site=i, order=self.b.order)
        return dict(o, gate=self.gate, gate_per_document=True) if i == 1 else o

    def run(self):
        cpt, plan, order = self.cpt, self.b.plan, self.b.order
        cpt.cpt_residual_norm(plan, self.x, self.h[0], self.y[0], self.n[0], **self.options(0))
        cpt.cpt_residual_norm(plan, self.y[0], self.h[1], self.y[1], self.n[1], **self.options(1))
        torch.matmul(self.n[1], self.head, out=self.logits)
        cpt.cpt_token_logprob(plan, self.logits, self.targets, self.logp, self.stats, vocab=self.V, order=order)
        cpt.cpt_policy_loss(plan, self.logp, self.old, self.adv, self.terms, self.dlogp, logp_ref=self.ref, mask=self.mask,
                            clip_low=0.3, clip_high=0.4, kl_coef=0.1)
        cpt.cpt_token_logprob_backward(plan, self.logits, self.targets, self.stats, self.dlogp, self.dlogits, vocab=self.V,
                                       order=order)
        torch.matmul(self.dlogits, self.head.t(), out=self.dn)
        cpt.cpt_residual_norm_backward(plan, self.h[1], self.y[1], None, self.dn, self.dx[1], self.dh[1], dgate=self.dgate,
                                       dpost_weight=self.dpost[1], dpre_weight=self.dpre[1], workspace=self.work,
                                       **self.options(1))
        # nothing but the stream goes back from the first block's norm here
        self.dn.zero_()
        cpt.cpt_residual_norm_backward(plan, self.h[0], self.y[0], self.dx[1], self.dn, self.dx[0], self.dh[0],
                                       dpost_weight=self.dpost[0], dpre_weight=self.dpre[0], workspace=self.work,
                                       **self.options(0))

    def results(self):
        return [self.terms, self.dlogp, self.dgate] + self.dx + self.dh + self.dpost + self.dpre + self.y + self.n

    def reference(self):
        """The same in float64 with autograd, on real tokens in global order."""
        b, C = self.b, self.C
        tok = lambda t: torch.zeros(b.T, C, dtype=torch.float64, device="cuda").index_copy_(0, b.at, b.pick(t)).requires_grad_(True)  # noqa: E731
        x, h = tok(self.x), [tok(t) for t in self.h]
        gate = self.gate.double().requires_grad_(True)
        post, pre = ([w.double().requires_grad_(True) for w in ws] for ws in (self.post, self.pre))
        seed, step = (int(v) for v in self.rng)
        y = x
        for i in range(2):
            u = h[i] / torch.sqrt(h[i].square().mean(1, keepdim=True) + 1e-6) * post[i]
            if i == 1:
                u = u * gate[b.doc]
            y = y + 0.8 * u * factor(seed, step, i, np.arange(b.T), C, 0.2)
        n = y / torch.sqrt(y.square().mean(1, keepdim=True) + 1e-6) * pre[1]
        z = (n @ self.head.double())[:, :self.V]
        m = self.mask
        logp = torch.log_softmax(z, 1)[torch.arange(b.T, device="cuda"), self.targets.clamp(min=0).long()]
        A = self.adv.double()[b.doc]
        ratio = torch.exp(logp - self.old.double())
        gap = self.ref.double() - logp
        each = -torch.minimum(ratio * A, ratio.clamp(0.7, 1.4) * A) + 0.1 * (torch.exp(gap) - gap - 1)
        count = torch.zeros(b.n, dtype=torch.float64, device="cuda").index_add_(0, b.doc, m.double())
        loss = torch.zeros(b.n, dtype=torch.float64, device="cuda").index_add(0, b.doc, torch.where(m, each, 0.0)) / count.clamp(min=1)
        grads = torch.autograd.grad(loss.sum() / b.n, [x, h[0], h[1], gate, post[0], post[1], pre[1]])
        return loss.detach(), grads


@pytest.mark.parametrize("kind,P,order", [(3, 4, 1), (1, 2, 1), (3, 3, 0)])
def test_a_step_against_autograd(cpt, cuda_device, kind, P, order):
    b = Batch(cpt, kind, P, [37, 0, 12, 1, 100], order)
    s = Step(cpt, b)
    s.run()
    loss, grads = s.reference()
    # Every value on the way is off by some 100 u of the terms it is made of (the bounds of the calls' own tests), and six
    # stages follow one another: 1000 u of a gradient's norm, and as much for the matrix products in binary32
    tol = 2000 * U
    assert ((s.terms[:, 0].double() - loss).abs() <= tol * (1 + loss.abs())).all()
    got = [b.pick(s.dx[0]), b.pick(s.dh[0]), b.pick(s.dh[1]), s.dgate, s.dpost[0], s.dpost[1], s.dpre[1]]
    for g, want, name in zip(got, grads, ("x", "h0", "h1", "gate", "post0", "post1", "pre1")):
        w = want[b.at] if want.shape[0] == b.T and name in ("x", "h0", "h1") else want
        assert (g.double() - w).norm() <= tol * w.norm(), name
    assert (s.dpre[0] == 0).all()
    assert cpt.cpt_kernel_wait_timeouts() == 0


def test_a_captured_step_draws_anew(cpt, cuda_device):
    """Replays equal eager runs at every step of the generator, while another graph of the same calls is replayed too."""
    b = Batch(cpt, 3, 4, [300, 0, 41, 700], 1)
    steps = [Step(cpt, b, C=640, seed=i) for i in range(2)]
    graphs, side = [], torch.cuda.Stream()
    for s in steps:
        s.run()
        torch.cuda.synchronize()
        s.rng[1] = 0
        g = torch.cuda.CUDAGraph()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=side):
            s.rng[1] += 1
            s.run()
        graphs.append(g)
    eager = [Step(cpt, b, C=640, seed=i) for i in range(2)]
    seen = []
    for step in (1, 2, 3):
        for g in graphs:
            g.replay()
        for e, s in zip(eager, steps):
            e.rng[1] = step
            e.run()
            torch.cuda.synchronize()
            assert all(torch.equal(a, r) for a, r in zip(e.results(), s.results()))
        seen.append(steps[0].y[0].clone())
    assert not torch.equal(seen[0], seen[1]) and not torch.equal(seen[1], seen[2])


def test_captured_clusters(cpt, cuda_device):
    """The calls that split a row or a document over a cluster, recorded and replayed with new inputs."""
    b = Batch(cpt, 1, 1, [9000, 3], 1)
    logp, old, adv = (torch.zeros(n, device="cuda") for n in (b.T, b.T, 2))
    terms, d = torch.empty(2, 4, device="cuda"), torch.empty(b.T, device="cuda")
    few = Batch(cpt, 1, 1, [6], 1)
    x, targets = torch.zeros(1, 6, 40000, device="cuda"), torch.arange(6, device="cuda", dtype=torch.int32)
    lp, stats = torch.empty(6, device="cuda"), torch.empty(6, 2, device="cuda")

    def calls():
        cpt.cpt_policy_loss(b.plan, logp, old, adv, terms, d)
        cpt.cpt_token_logprob(few.plan, x, targets, lp, stats)

    calls()
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=side):
        calls()
    for seed in (1, 2):
        r = gen(seed)
        for t in (logp, old, adv, x):
            t.copy_(torch.randn(t.shape, device="cuda", generator=r) * 0.3)
        g.replay()
        got = [t.clone() for t in (terms, d, lp, stats)]
        calls()
        assert all(torch.equal(a, w) for a, w in zip(got, (terms, d, lp, stats)))


FRESH = """
import torch
from context_attention_token_gb300 import cpt
plan = cpt.cpt_plan_create(3, 2, [0, 37, 50], 50)
rows = plan.padded_tokens // 2
x, h, n, dx, dh = (torch.ones(2, rows, 640, device="cuda") for _ in range(5))
w, dw = torch.ones(2, 640, device="cuda"), torch.empty(2, 640, device="cuda")
gate, dgate = torch.ones(2, 640, device="cuda"), torch.empty(2, 640, device="cuda")
o = dict(post_weight=w[0], pre_weight=w[1], gate=gate, gate_per_document=True)
work = torch.empty(cpt.cpt_residual_norm_backward_workspace_bytes(plan, 640, torch.float32), dtype=torch.uint8, device="cuda")
torch.cuda.synchronize()
g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
s.wait_stream(torch.cuda.current_stream())
with torch.cuda.graph(g, stream=s):
    cpt.cpt_residual_norm(plan, x, h, x, n, **o)
    cpt.cpt_residual_norm_backward(plan, h, x, None, n, dx, dh, dgate=dgate, dpost_weight=dw[0], dpre_weight=dw[1],
                                   workspace=work, **o)
g.replay()
torch.cuda.synchronize()
assert torch.isfinite(dw).all() and torch.isfinite(dgate).all()
print("ok")
"""


def test_first_calls_of_a_process_inside_a_capture(cpt, cuda_device):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FRESH], capture_output=True, text=True, timeout=300, cwd=root,
                       env=dict(os.environ, PYTHONPATH=root))
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr[-2000:]


def test_two_streams_at_once(cpt, cuda_device):
    b = Batch(cpt, 0, 4, [8 * 400, 8 * 13], 1)
    steps = [Step(cpt, b, C=1280, seed=i) for i in range(2)]
    for s in steps:
        s.run()
    torch.cuda.synchronize()
    want = [[t.clone() for t in s.results()] for s in steps]
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(5):
        for s, st in zip(steps, streams):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                s.run()
    torch.cuda.synchronize()
    for s, w in zip(steps, want):
        assert all(torch.equal(a, r) for a, r in zip(s.results(), w))


def test_a_stream_of_ones_own(cpt, cuda_device):
    """With `stream` the call goes there, whatever torch's current stream is."""
    b = Batch(cpt, 1, 1, [64], 1)
    s = Step(cpt, b)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    cpt.cpt_residual_norm(b.plan, s.x, s.h[0], s.y[0], s.n[0], stream=st, **s.options(0))
    cpt.cpt_residual_norm_backward(b.plan, s.h[0], s.y[0], s.x, s.n[0], s.dx[0], s.dh[0], dpost_weight=s.dpost[0],
                                   dpre_weight=s.dpre[0], workspace=s.work, stream=st, **s.options(0))
    st.synchronize()
    assert all(torch.isfinite(t).all() for t in (s.y[0], s.n[0], s.dx[0], s.dh[0]))


def test_readme_example(cpt, cuda_device):
    """The README's third example runs as written after its first; some rows against 64 bits."""
    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")) as f:
        text = f.read()
    first = re.search(r"```python\n(.*?)```", text, flags=re.S).group(1)
    example = re.findall(r"```py\n(.*?)```", text, flags=re.S)[1]
    env = {}
    exec(compile(first[:first.index("q = ")], "README.md", "exec"), env)
    before, after = example[:example.index("cpt.cpt_residual_norm(")], example[example.index("cpt.cpt_residual_norm("):]
    exec(compile(before, "README.md", "exec"), env)
    x0 = env["x"].clone()
    exec(compile(after, "README.md", "exec"), env)
    torch.cuda.synchronize()
    P, S, C = env["P"], env["S"], env["C"]
    l2g = torch.empty(S, dtype=torch.int32, device="cuda")
    cpt.cpt_index_map(env["plan"], l2g, None)
    rows = torch.arange(0, S, S // 50, device="cuda")
    at = lambda t: t.reshape(S, -1)[rows].double()  # noqa: E731
    drop = factor(1234, 0, 7, l2g[rows].cpu().numpy(), C, 0.1)
    want = residual_norm(at(x0), at(env["h"]), None, env["w_post"].double(), env["w_pre"].double(), 0.5, drop, 1e-6)
    close(env["x"].reshape(S, -1)[rows], want[0], want[1], "y")
    close(env["n"].reshape(S, -1)[rows], want[2], want[3], "n")
    # the gradient of the logits of a row adds up to nothing: each of its columns is off by half a step of bf16, 2^-8, and
    # the weights' own 300 u
    d = env["logits"].reshape(S, -1)[rows, :env["V"]].double()
    assert (d.sum(1).abs() <= (2.0 ** -8 + 300 * U) * d.abs().sum(1)).all()
    assert all(torch.isfinite(env[k]).all() for k in ("terms", "dlogp", "dx", "dh", "dw_post", "dw_pre"))


# ---------------------------------------------------------------- more than 2^32 elements

def test_rows_past_2_to_the_32(cpt, cuda_device):
    """1.1 million rows of 4096: the last rows lie past 2^32 elements (and 2^33 bytes)."""
    T, C, last = 1_100_003, 4096, 40
    b = Batch(cpt, 1, 1, [T - 20, 20], 1)
    g = gen(0)
    full = lambda: torch.zeros(1, T, C, dtype=BF16, device="cuda")  # noqa: E731
    x, h, y, n = full(), full(), full(), full()
    for t in (x, h):
        t[0, -last:] = torch.randn(last, C, device="cuda", generator=g).to(BF16)
        t[0, :last] = torch.randn(last, C, device="cuda", generator=g).to(BF16)
    w = 1 + 0.1 * torch.randn(2, C, device="cuda", generator=g)
    gate = torch.randn(2, C, device="cuda", generator=g).to(BF16)
    rng = torch.tensor([5, 6], dtype=torch.int64, device="cuda")
    o = dict(post_weight=w[0], pre_weight=w[1], gate=gate, gate_per_document=True, scale=0.5, p=0.1, rng=rng, site=1, eps=1e-5)
    cpt.cpt_residual_norm(b.plan, x, h, y, n, **o)
    for rows in (slice(0, last), slice(T - last, T)):
        at = np.arange(T)[rows]
        want = residual_norm(x[0, rows].double(), h[0, rows].double(), gate.double()[b.doc[rows]], w[0].double(), w[1].double(),
                             0.5, factor(5, 6, 1, at, C, 0.1), 1e-5)
        close(y[0, rows], want[0], want[1], "y")
        close(n[0, rows], want[2], want[3], "n")
    # the gradient of rows that are zeros is that of the stream alone; a document's gate has the last rows' sums
    dx, dh, dgate, dw = x, n, torch.empty(2, C, device="cuda"), torch.empty(2, C, device="cuda")
    dn = full()
    dn[0, -last:] = torch.randn(last, C, device="cuda", generator=g).to(BF16)
    dx = full()
    dh2 = full()
    cpt.cpt_residual_norm_backward(b.plan, h, y, None, dn, dx, dh2, dgate=dgate, dpost_weight=dw[0], dpre_weight=dw[1], **o)
    assert torch.isfinite(dgate).all() and torch.isfinite(dw).all()
    assert (dx[0, last:-last].abs().amax() == 0) and (dx[0, -last:] != 0).any(1).all() and (dh2[0, -last:] != 0).any(1).all()
    del dn, dx, dh2, n, y, x
    cpt.cpt_dropout(b.plan, h, h, 0.1, rng, 3)
    kept = (h[0, -last:] != 0).cpu().numpy()
    assert np.array_equal(kept, (factor(5, 6, 3, np.arange(T - last, T), C, 0.1) > 0).cpu().numpy())


def test_logits_past_2_to_the_32(cpt, cuda_device):
    T, V, last = 27500, 157184, 8
    b = Batch(cpt, 1, 1, [T], 1)
    x = torch.zeros(1, T, V, dtype=BF16, device="cuda")
    x[0, -last:] = torch.randn(last, V, device="cuda", generator=gen(1)).to(BF16)
    targets = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    targets[-last:] = V - 1 - torch.arange(last, device="cuda", dtype=torch.int32)
    logp, stats, d = torch.empty(T, device="cuda"), torch.empty(T, 2, device="cuda"), torch.ones(T, device="cuda")
    cpt.cpt_token_logprob(b.plan, x, targets, logp, stats)
    want = torch.log_softmax(x[0, -last:].double(), 1)
    got = logp[-last:].double() - want[torch.arange(last), targets[-last:].long()]
    assert got.abs().max() <= 200 * U * 16 and (logp[:-last] == 0).all()
    keep = x[0, -last:].clone()
    cpt.cpt_token_logprob_backward(b.plan, x, targets, stats, d, x)          # in place
    one = torch.zeros(last, V, dtype=torch.float64, device="cuda").scatter_(1, targets[-last:].long()[:, None], 1.0)
    exact = one - torch.softmax(keep.double(), 1)
    # half a step of bf16, and the weight's own 300 u of test_gpu_token_logprob's derivation
    assert ((x[0, -last:].double() - exact).abs() <= (2.0 ** -8 + 300 * U) * exact.abs() + 1e-30).all()
    assert x[0, -last - 5:-last].abs().max() == 0


# ---------------------------------------------------------------- refusals

def _p(t):
    return None if t is None else t.data_ptr()


class Residual:
    def __init__(self, cpt, T=32, C=64):
        self.cpt, self.C = cpt, C
        self.plan = cpt.cpt_plan_create(0, 2, [0, T], T)
        z = lambda *s, v=7.0: torch.full(s, v, device="cuda")  # noqa: E731
        self.x, self.h, self.dn = (torch.randn(T, C, device="cuda") for _ in range(3))
        self.w = torch.ones(4, C, device="cuda")
        self.gate = torch.randn(T, C, device="cuda")
        self.rng = torch.zeros(2, dtype=torch.int64, device="cuda")
        self.outs = [z(T, C) for _ in range(3)] + [z(C) for _ in range(2)]
        self.need = cpt.cpt_residual_norm_backward_workspace_bytes(self.plan, C, F32)
        self.work = torch.empty(self.need, dtype=torch.uint8, device="cuda")
        self.stream = torch.cuda.current_stream().cuda_stream

    def options(self, **kw):
        o = dict(post_weight=_p(self.w[0]), pre_weight=_p(self.w[1]), gate=_p(self.gate), gate_kind=1, scale=1.0, eps=1e-6, p=0.1,
                 rng=_p(self.rng), site=0)
        o.update(kw)
        return self.cpt._Residual(*[o[n] for n, _ in self.cpt._Residual._fields_])

    def forward(self, given=None, **kw):
        a = dict(plan=self.plan.handle, x=_p(self.x), h=_p(self.h), y=_p(self.outs[0]), n=_p(self.outs[1]), row=self.C, dtype=0,
                 order=1, options=ctypes.byref(given if given is not None else self.options()), stream=self.stream)
        assert set(kw) <= set(a)
        return self.cpt._lib.cpt_residual_norm(*{**a, **kw}.values())

    def backward(self, given=None, **kw):
        o = self.outs
        a = dict(plan=self.plan.handle, h=_p(self.h), y=_p(self.x), dy=None, dn=_p(self.dn), dx=_p(o[0]), dh=_p(o[1]), dgate=_p(o[2]),
                 dpost=_p(o[3]), dpre=_p(o[4]), row=self.C, dtype=0, order=1,
                 options=ctypes.byref(given if given is not None else self.options()), work=_p(self.work),
                 bytes=self.need, stream=self.stream)
        assert set(kw) <= set(a)
        return self.cpt._lib.cpt_residual_norm_backward(*{**a, **kw}.values())


def test_residual_norm_refuses(cpt, cuda_device):
    r = Residual(cpt)
    A, U_, L, X, W, D = (cpt.CPT_ERR_INVALID_ARG, cpt.CPT_ERR_UNSUPPORTED, cpt.CPT_ERR_ALIGNMENT, cpt.CPT_ERR_ALIAS,
                         cpt.CPT_ERR_WORKSPACE, cpt.CPT_ERR_DEVICE)
    o, host = r.options, torch.zeros(32, 64)
    shared = [
        (dict(plan=None), None, A), (dict(row=0), None, A), (dict(row=-4), None, A), (dict(row=63), None, L),
        (dict(row=8196), None, U_), (dict(dtype=2), None, A), (dict(order=2), None, A), (dict(order=-1), None, A),
        (dict(options=None), None, A), ({}, o(gate_kind=3), A), ({}, o(gate_kind=0), A), ({}, o(gate=None), A),
        ({}, o(scale=float("inf")), A), ({}, o(scale=float("nan")), A), ({}, o(eps=-1e-9), A), ({}, o(eps=float("nan")), A),
        ({}, o(p=-0.1), A), ({}, o(p=1.1), A), ({}, o(p=float("nan")), A), ({}, o(rng=None), A),
        ({}, o(post_weight=_p(r.w) + 4), L), ({}, o(pre_weight=_p(r.w) + 8), L), ({}, o(gate=_p(r.gate) + 4), L),
        ({}, o(rng=_p(r.rng) + 4), L), ({}, o(post_weight=_p(host)), D), ({}, o(gate=_p(host)), D),
    ]
    first = [
        (dict(x=None), None, A), (dict(h=None), None, A), (dict(y=None), None, A), (dict(n=None), None, A),
        (dict(h=None, y=None), None, A),                                   # a post norm without a block
        (dict(h=None, y=None, n=None), o(post_weight=None, pre_weight=None, gate=None, gate_kind=0, p=0.0), A),
        ({}, o(pre_weight=None), A),                                       # n without its weight
        (dict(x=_p(r.x) + 8), None, L), (dict(y=_p(r.outs[0]) + 4), None, L), (dict(x=_p(host)), None, D),
        (dict(y=_p(r.h)), None, X), (dict(n=_p(r.x)), None, X), (dict(n=_p(r.outs[0])), None, X), (dict(y=_p(r.x) + 256), None, X),
        (dict(n=_p(r.gate)), None, X), (dict(y=r.plan.workspace.data_ptr()), None, X),
    ]
    for kw, options, want in shared + first:
        assert r.forward(options, **kw) == want, (kw, want)
    back = [
        (dict(h=None), None, A), (dict(y=None), None, A), (dict(dn=None), None, A), (dict(dx=None), None, A), (dict(dh=None), None, A),
        (dict(dgate=None), None, A), (dict(dpost=None), None, A), (dict(dpre=None), None, A), ({}, o(pre_weight=None), A),
        (dict(y=None, dn=None, dpre=None), o(pre_weight=None), A),         # no gradient comes in
        (dict(work=None), None, W), (dict(bytes=r.need - 1), None, W), (dict(work=_p(r.work) + 16), None, W),
        (dict(dx=_p(r.h)), None, X), (dict(dh=_p(r.dn)), None, X), (dict(dgate=_p(r.outs[0])), None, X), (dict(dpost=_p(r.w)), None, X),
        (dict(dpre=_p(r.outs[3])), None, X), (dict(dh=_p(r.work)), None, X), (dict(dy=_p(r.outs[1])), None, X),
        (dict(dx=_p(r.outs[0]) + 4), None, L), (dict(dpost=_p(r.outs[3]) + 4), None, L), (dict(dn=_p(host)), None, D),
    ]
    for kw, options, want in shared + back:
        assert r.backward(options, **kw) == want, (kw, want)
    torch.cuda.synchronize()
    assert all((t == 7.0).all() for t in r.outs)
    assert r.forward() == 0 and r.backward() == 0
    torch.cuda.synchronize()
    assert not any((t == 7.0).any() for t in r.outs)
    assert cpt.cpt_residual_norm_backward_workspace_bytes(r.plan, 8196, F32) == 0
    assert cpt.cpt_residual_norm_backward_workspace_bytes(r.plan, 63, F32) == 0
    assert cpt.cpt_residual_norm_backward_workspace_bytes(r.plan, 64, torch.float16) == 0


def test_dropout_refuses(cpt, cuda_device):
    T, C = 32, 64
    plan = cpt.cpt_plan_create(0, 2, [0, T], T)
    x, y = torch.randn(T, C, device="cuda"), torch.full((T, C), 7.0, device="cuda")
    rng = torch.zeros(2, dtype=torch.int64, device="cuda")
    ok = dict(plan=plan.handle, src=_p(x), dst=_p(y), row=C, dtype=0, order=1, p=0.5, rng=_p(rng), site=0,
              stream=torch.cuda.current_stream().cuda_stream)
    A, L, X, D = cpt.CPT_ERR_INVALID_ARG, cpt.CPT_ERR_ALIGNMENT, cpt.CPT_ERR_ALIAS, cpt.CPT_ERR_DEVICE
    bad = [
        (dict(plan=None), A), (dict(src=None), A), (dict(dst=None), A), (dict(row=0), A), (dict(row=62), L), (dict(row=1 << 40), A),
        (dict(dtype=5), A), (dict(order=3), A), (dict(p=-1e-9), A), (dict(p=1.0000001), A), (dict(p=float("nan")), A), (dict(rng=None), A),
        (dict(src=_p(x) + 4), L), (dict(dst=_p(y) + 8), L), (dict(rng=_p(rng) + 4), L), (dict(src=_p(torch.zeros(T, C))), D),
        (dict(rng=_p(torch.zeros(2, dtype=torch.int64))), D), (dict(dst=_p(x) + 256), X), (dict(rng=_p(y)), X),
        (dict(dst=plan.workspace.data_ptr()), X),
    ]
    for kw, want in bad:
        assert cpt._lib.cpt_dropout(*{**ok, **kw}.values()) == want, kw
    torch.cuda.synchronize()
    assert (y == 7.0).all()
    assert cpt._lib.cpt_dropout(*ok.values()) == 0
    assert cpt._lib.cpt_dropout(*{**ok, "p": 0.0, "rng": None}.values()) == 0


def test_logprob_refuses(cpt, cuda_device):
    T, V = 32, 64
    plan = cpt.cpt_plan_create(0, 2, [0, T], T)
    x, dx = torch.randn(T, V, device="cuda"), torch.full((T, V), 7.0, device="cuda")
    t = torch.zeros(T, dtype=torch.int32, device="cuda")
    logp, stats, d = torch.full((T,), 7.0, device="cuda"), torch.full((T, 2), 7.0, device="cuda"), torch.ones(T, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    shape = dict(vocab=60, padded=V, dtype=0, order=1, scale=1.0, stream=st)
    fwd = dict(plan=plan.handle, logits=_p(x), targets=_p(t), logp=_p(logp), stats=_p(stats), **shape)
    back = dict(plan=plan.handle, logits=_p(x), targets=_p(t), stats=_p(stats), dlogp=_p(d), dlogits=_p(dx), **shape)
    A, L, X, D = cpt.CPT_ERR_INVALID_ARG, cpt.CPT_ERR_ALIGNMENT, cpt.CPT_ERR_ALIAS, cpt.CPT_ERR_DEVICE
    both = [
        (dict(plan=None), A), (dict(logits=None), A), (dict(targets=None), A), (dict(stats=None), A), (dict(vocab=0), A),
        (dict(vocab=-1), A), (dict(vocab=65), A), (dict(padded=0), A), (dict(padded=63, vocab=1), L), (dict(dtype=-1), A),
        (dict(order=2), A), (dict(scale=0.0), A), (dict(scale=-1.0), A), (dict(scale=float("inf")), A), (dict(scale=float("nan")), A),
        (dict(logits=_p(x) + 4), L), (dict(targets=_p(t) + 2), L), (dict(stats=_p(stats) + 4), L), (dict(logits=_p(torch.zeros(T, V))), D),
    ]
    for kw, want in both + [(dict(logp=None), A), (dict(logp=_p(x)), X), (dict(stats=_p(logp) - _p(logp) % 8), X), (dict(logp=_p(t)), X)]:
        assert cpt._lib.cpt_token_logprob(*{**fwd, **kw}.values()) == want, kw
    for kw, want in both + [(dict(dlogp=None), A), (dict(dlogits=None), A), (dict(dlogits=_p(x) + 256), X), (dict(dlogits=_p(stats)), X if _p(stats) % 16 == 0 else L),
                            (dict(dlogits=_p(dx) + 4), L)]:
        assert cpt._lib.cpt_token_logprob_backward(*{**back, **kw}.values()) == want, kw
    torch.cuda.synchronize()
    assert (logp == 7.0).all() and (stats == 7.0).all() and (dx == 7.0).all()
    assert cpt._lib.cpt_token_logprob(*fwd.values()) == 0 and cpt._lib.cpt_token_logprob_backward(*back.values()) == 0


def test_policy_loss_refuses(cpt, cuda_device):
    T = 32
    plan = cpt.cpt_plan_create(0, 2, [0, 16, T], T)
    f = [torch.randn(T, device="cuda") for _ in range(3)]
    adv, w = torch.ones(2, device="cuda"), torch.ones(2, device="cuda")
    mask = torch.ones(T, dtype=torch.uint8, device="cuda")
    terms, d = torch.full((2, 4), 7.0, device="cuda"), torch.full((T,), 7.0, device="cuda")
    ok = dict(plan=plan.handle, logp=_p(f[0]), old=_p(f[1]), ref=_p(f[2]), mask=_p(mask), adv=_p(adv), w=_p(w), low=0.2, high=0.2,
              kl=0.1, terms=_p(terms), dlogp=_p(d), stream=torch.cuda.current_stream().cuda_stream)
    A, L, X, D = cpt.CPT_ERR_INVALID_ARG, cpt.CPT_ERR_ALIGNMENT, cpt.CPT_ERR_ALIAS, cpt.CPT_ERR_DEVICE
    nan = float("nan")
    bad = [
        (dict(plan=None), A), (dict(logp=None), A), (dict(old=None), A), (dict(ref=None), A), (dict(adv=None), A), (dict(terms=None), A),
        (dict(dlogp=None), A), (dict(low=-0.1), A), (dict(low=1.1), A), (dict(low=nan), A), (dict(high=-0.1), A), (dict(high=nan), A),
        (dict(high=float("inf")), A), (dict(kl=-1.0), A), (dict(kl=nan), A), (dict(kl=float("inf")), A), (dict(logp=_p(f[0]) + 2), L),
        (dict(terms=_p(terms) + 4), L), (dict(mask=_p(torch.zeros(T, dtype=torch.uint8))), D), (dict(dlogp=_p(f[0])), X), (dict(dlogp=_p(f[2])), X),
        (dict(dlogp=_p(mask)), X), (dict(terms=_p(f[1])), X), (dict(dlogp=_p(terms)), X),
    ]
    for kw, want in bad:
        assert cpt._lib.cpt_policy_loss(*{**ok, **kw}.values()) == want, kw
    torch.cuda.synchronize()
    assert (terms == 7.0).all() and (d == 7.0).all()
    assert cpt._lib.cpt_policy_loss(*ok.values()) == 0
    assert cpt._lib.cpt_policy_loss(*{**ok, "ref": None, "kl": 0.0, "mask": None, "w": None}.values()) == 0
