"""The operators around the context-parallel attention layer, as measured.

What a training step does with token rows outside of attention and of matrix
products, wherever it has to know which token and which document a row is:

  dropout                 dropout whose mask is a function of the token, not of the
                          row, so that it is the same in either row order and
                          for any number of ranks, and is never stored;
  residual_norm           the end of one block and the beginning of the next:
                          y = x + scale * dropout(gate * norm(h)), n = norm(y);
  residual_norm_backward  its gradient, with those of weights and of gates that
                          all tokens of a document share;
  token_logprob           the logarithm of the probability that rank-local logits
                          give to every token's target;
  token_logprob_backward  its gradient, the logits';
  policy_loss             a clipped policy loss with a KL term over the plan's
                          documents, and its gradient.

`run` computes them in plain torch (own = False) or calls the library.
"""
import math
import random

import numpy as np
import torch

own = False

LAYOUTS = {"swap": 0, "packed": 1, "padded": 3}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # latency: the smallest packed batch of this repository's tests
        {"name": "dropout_tiny", "op": "dropout", "layout": "swap", "P": 2, "T": 64, "median": 16, "C": 16,
         "order": "local", "p": 0.1, "dtype": "f32"},
        # dropout of the embeddings of a packed batch, documents of any length
        {"name": "dropout_packed_docs", "op": "dropout", "layout": "padded", "P": 4, "T": 131071, "median": 2048,
         "C": 2048, "order": "local", "p": 0.1, "dtype": "bf16"},
        # latency: a block of a small model
        {"name": "residual_norm_tiny", "op": "residual_norm", "layout": "swap", "P": 2, "T": 64, "median": 16, "C": 64,
         "order": "local", "post": True, "pre": True, "gate": "none", "p": 0.0, "dtype": "bf16"},
        # one long causal sequence at 20 heads of 128: norms on both sides of the block, dropout
        {"name": "residual_norm_long", "op": "residual_norm", "layout": "swap", "P": 4, "T": 262144, "median": 0,
         "C": 2560, "order": "local", "post": True, "pre": True, "gate": "none", "p": 0.1, "dtype": "bf16"},
        # the gradient of a float32 block of odd width, a gate of every token's own
        {"name": "residual_norm_backward_odd_f32", "op": "residual_norm_backward", "layout": "padded", "P": 3,
         "T": 20011, "median": 700, "C": 1132, "order": "local", "post": True, "pre": True, "gate": "token", "p": 0.05,
         "dtype": "f32"},
        # the gradient of a packed batch whose documents each have a gate, as a conditioned model's do
        {"name": "residual_norm_backward_docs", "op": "residual_norm_backward", "layout": "padded", "P": 4, "T": 131071,
         "median": 2048, "C": 2560, "order": "local", "post": True, "pre": True, "gate": "document", "p": 0.1,
         "dtype": "bf16"},
        # scoring a short answer: few rows, the whole vocabulary
        {"name": "logprob_few_rows", "op": "token_logprob", "layout": "swap", "P": 2, "T": 64, "median": 16,
         "vocab": 157184, "order": "local", "scale": 1.0, "prompt": 0.3, "dtype": "bf16"},
        # a training micro-batch's logits, rank by rank
        {"name": "logprob_batch", "op": "token_logprob", "layout": "padded", "P": 4, "T": 8191, "median": 2048,
         "vocab": 157184, "order": "local", "scale": 1.0, "prompt": 0.0, "dtype": "bf16"},
        # the gradient of a small float32 vocabulary of odd size, prompts without a target
        {"name": "logprob_backward_small_f32", "op": "token_logprob_backward", "layout": "packed", "P": 2, "T": 4096,
         "median": 256, "vocab": 4099, "order": "global", "scale": 0.7, "prompt": 0.4, "dtype": "f32"},
        # the gradient of a training micro-batch's logits
        {"name": "logprob_backward_batch", "op": "token_logprob_backward", "layout": "padded", "P": 4, "T": 8191,
         "median": 2048, "vocab": 157184, "order": "local", "scale": 1.0, "prompt": 0.0, "dtype": "bf16"},
        # latency: a few sampled answers
        {"name": "policy_loss_tiny", "op": "policy_loss", "layout": "swap", "P": 2, "T": 512, "median": 64,
         "prompt": 0.3, "reference": True},
        # a large batch of answers of any length
        {"name": "policy_loss_docs", "op": "policy_loss", "layout": "padded", "P": 4, "T": 262139, "median": 2048,
         "prompt": 0.3, "reference": True},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["dropout", "residual_norm", "residual_norm", "residual_norm_backward",
                         "residual_norm_backward", "token_logprob", "token_logprob_backward", "policy_loss"])
        layout = rng.choice(["swap", "packed", "padded"])
        P = rng.choice([1, 2, 3, 4, 8])
        T = _log_uniform(rng, 1, 65536 if op.startswith("token") else 262144)
        T -= T % (1 if layout == "padded" else P if layout == "packed" else 2 * P)
        if T < 1:
            continue
        c = {"op": op, "layout": layout, "P": P, "T": T, "median": rng.choice([0, _log_uniform(rng, 8, 8192)])}
        dtype = rng.choice(["bf16", "bf16", "f32"])
        if op == "policy_loss":
            c.update(prompt=rng.choice([0.0, 0.3, 0.9]), reference=rng.random() < 0.7)
            if _answers(c).any():
                return c
            continue
        if op.startswith("token"):
            V = _log_uniform(rng, 16, 200000)
            c.update(vocab=V, order=rng.choice(["local", "global"]), scale=rng.choice([1.0, 1.0, 0.7, 1.5]),
                     prompt=rng.choice([0.0, 0.3, 0.9]), dtype=dtype)
            if T * V * (2 if dtype == "bf16" else 4) <= 8191 * 157184 * 2 and _answers(c).any():
                return c
            continue
        C = 8 * _log_uniform(rng, 2, 1024)
        c.update(C=C, order=rng.choice(["local", "local", "global"]), dtype=dtype)
        if op == "dropout":
            c.update(p=rng.choice([0.1, 0.1, 0.05, 0.5, 0.25]))
        elif rng.random() < 0.1:    # a model's first norm: there is no block yet
            c.update(post=False, pre=True, gate="first", p=0.0)
        else:
            post = rng.random() < 0.7
            gate = rng.choice(["none", "none", "token", "document"])
            c.update(post=post, pre=rng.random() < 0.8, gate=gate, p=rng.choice([0.0, 0.1, 0.05, 0.3]))
        most = 262144 * 2560 if op == "residual_norm" else 131071 * 2560 if op != "dropout" else 131071 * 2048
        if T * C * (2 if dtype == "bf16" else 4) <= 2 * most:
            return c


# ---------------------------------------------------------------- layouts (host)

def _lengths(case):
    """Document lengths of a batch: one document, or lognormal lengths around the median."""
    T, P, median = case["T"], case["P"], case["median"]
    multiple = 2 * P if case["layout"] == "swap" else 1
    if median == 0 or median >= T:
        return [T]
    rng = np.random.default_rng([T, median, P])
    lens, left = [], T
    while left > 0:
        x = int(min(max(round(math.exp(rng.normal(math.log(median), 1.0))), median // 8, 1), 16 * median))
        x = min(-(-x // multiple) * multiple, left)
        lens.append(x)
        left -= x
    return lens


def _layout(case):
    """Raw token of every local row, rank-major (-1: a padding row), and the raw boundaries."""
    P, kind = case["P"], case["layout"]
    lens = np.array(_lengths(case), dtype=np.int64)
    cu = np.concatenate([[0], np.cumsum(lens)])
    if kind == "packed":
        return np.arange(case["T"], dtype=np.int64), cu
    pad = -(-lens // (2 * P)) * (2 * P)
    l2r = []
    for r in range(P):
        for i in range(len(lens)):
            m = pad[i] // (2 * P)
            u = np.concatenate([np.arange(r * m, (r + 1) * m), np.arange((2 * P - 1 - r) * m, (2 * P - r) * m)])
            l2r.append(np.where(u < lens[i], cu[i] + u, -1))
    return np.concatenate(l2r), cu


def _rows(case):
    """Raw token of every row of the case's token tensors (-1: padding)."""
    l2r, cu = _layout(case)
    return (l2r if case.get("order") == "local" else np.arange(case["T"], dtype=np.int64)), cu


def _padded_vocab(case):
    """Columns of a row of logits: whole groups of 16 bytes, as a padded embedding table has."""
    return -(-case["vocab"] // 8) * 8


def _answers(case):
    """Tokens that are scored: those behind each document's prompt, but for its last one."""
    _, cu = _layout(case)
    rng = np.random.default_rng([case["T"], case["P"], 5])
    take = np.zeros(case["T"], dtype=bool)
    for a, b in zip(cu[:-1], cu[1:]):
        prompt = int((b - a) * min(1.0, 2 * case["prompt"] * rng.random()))
        take[a + prompt:b - 1] = True
    return take


def work(case):
    op, T = case["op"], case["T"]
    if op == "policy_loss":
        n, k = len(_lengths(case)), int(_answers(case).sum())
        return {"bytes": 5 * T + k * (12 if case["reference"] else 8) + 20 * n, "flops": 20 * k}
    e = 2 if case["dtype"] == "bf16" else 4
    rows, cu = _rows(case)
    R, n = len(rows), len(cu) - 1
    if op == "dropout":
        return {"bytes": (T + R) * case["C"] * e, "flops": T * case["C"]}
    if op.startswith("token"):
        V, W, k = case["vocab"], _padded_vocab(case), int(_answers(case).sum())
        if op == "token_logprob":
            return {"bytes": k * V * e + 16 * T, "flops": 5 * k * V}
        return {"bytes": k * V * e + R * W * e + 16 * T, "flops": 5 * k * V}
    C, first = case["C"], case["gate"] == "first"
    gate = {"token": 1, "none": 0, "first": 0, "document": 0}[case["gate"]]
    gate_doc = n * C * e if case["gate"] == "document" else 0
    if op == "residual_norm":
        reads, writes = 1 + (not first) + gate, (not first) + case["pre"]
        return {"bytes": (T * reads + R * writes) * C * e + gate_doc, "flops": 14 * T * C}
    reads = 1 + 2 * case["pre"] + (case["post"] or case["gate"] in ("token", "document")) + gate
    writes = 1 + (not first) + gate
    return {"bytes": (T * reads + R * writes) * C * e + 3 * gate_doc, "flops": 30 * T * C}


# ---------------------------------------------------------------- inputs

EPS = 1e-6


def _normal(shape, dtype, g, sigma=1.0, mean=0.0):
    t = torch.randn(shape, dtype=torch.float32, device="cuda", generator=g)
    return t.mul_(sigma).add_(mean).to(dtype)


def _inputs(case, seed):
    """What the program has in hand: no plan, nothing of the library."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 29)
    op, T, P = case["op"], case["T"], case["P"]
    rows, cu = _rows(case)
    R = len(rows)
    doc = np.repeat(np.arange(len(cu) - 1), np.diff(cu))
    s = {"case": case, "R": R, "n": len(cu) - 1, "cu": cu}
    s["tokens"] = torch.from_numpy(rows).cuda()                 # raw token of every row
    s["doc"] = torch.from_numpy(doc).cuda()                     # document of every raw token
    lead = (P, R // P) if case.get("order") == "local" else (R,)
    if op == "policy_loss":
        s["logp"] = _normal((T,), torch.float32, g).abs_().mul_(-1.5)
        s["old"] = s["logp"] + _normal((T,), torch.float32, g, 0.1)
        s["ref"] = s["logp"] + _normal((T,), torch.float32, g, 0.2) if case["reference"] else None
        s["advantages"] = _normal((s["n"],), torch.float32, g)
        s["mask"] = torch.from_numpy(_answers(case)).cuda()
        s["weights"] = torch.full((s["n"],), 1.0 / s["n"], device="cuda")
        s["clip"], s["kl"] = (0.2, 0.28), 0.04 if case["reference"] else 0.0
        s["terms"] = torch.empty((s["n"], 4), device="cuda")
        s["dlogp"] = torch.empty((T,), device="cuda")
        return s
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    if op.startswith("token"):
        V, W = case["vocab"], _padded_vocab(case)
        x = torch.empty(lead + (W,), dtype=dt, device="cuda")
        flat = x.view(R, W)
        for a in range(0, R, 1024):     # in pieces: a whole binary32 copy is not needed
            flat[a:a + 1024] = _normal((min(1024, R - a), W), dt, g, 2.5)
        take = torch.from_numpy(_answers(case)).cuda()
        target = torch.randint(0, V, (T,), device="cuda", generator=g)
        # a trained model gives most targets a large logit
        real = torch.nonzero(s["tokens"] >= 0).squeeze(1)
        up = torch.rand((len(real),), device="cuda", generator=g) * 12.0
        flat[real, target[s["tokens"][real]]] = up.to(dt)
        s["logits"], s["take"] = x, take
        s["targets"] = torch.where(take, target, -1).to(torch.int32)
        s["logp"] = torch.empty((T,), device="cuda")
        s["stats"] = torch.empty((T, 2), device="cuda")
        if op == "token_logprob_backward":
            s["logp"], s["stats"] = _token_logprob(s)
            s["dlogp"] = torch.where(take, _normal((T,), torch.float32, g, 1.0 / T), 0.0)
            s["dlogits"] = torch.empty_like(x)
        return s
    C = case["C"]
    s["rng"] = torch.randint(0, 1 << 62, (2,), dtype=torch.int64, device="cuda", generator=g)
    s["site"] = seed % 97
    if op == "dropout":
        s["x"] = _normal(lead + (C,), dt, g)
        s["out"] = torch.empty_like(s["x"])
        return s
    back, first = op == "residual_norm_backward", case["gate"] == "first"
    s["scale"] = 1.0 if first else 0.7
    s["x"] = None if back else _normal(lead + (C,), dt, g, 2.0)
    s["h"] = None if first else _normal(lead + (C,), dt, g, 0.8)
    s["post_weight"] = _normal((C,), torch.float32, g, 0.1, 1.0) if case["post"] else None
    s["pre_weight"] = _normal((C,), torch.float32, g, 0.1, 1.0) if case["pre"] else None
    shape = {"token": lead + (C,), "document": (s["n"], C)}.get(case["gate"])
    s["gate"] = _normal(shape, dt, g, 0.5, 0.5) if shape else None
    if not back:
        s["y"] = None if first else torch.empty_like(s["x"])
        s["normed"] = torch.empty_like(s["x"]) if case["pre"] else None
        return s
    s["y"] = _normal(lead + (C,), dt, g, 2.0) if case["pre"] else None
    s["dy"], s["dn"] = _normal(lead + (C,), dt, g), _normal(lead + (C,), dt, g) if case["pre"] else None
    s["dx"] = torch.empty_like(s["dy"])
    s["dh"] = None if first else torch.empty_like(s["dy"])
    s["dgate"] = None if s["gate"] is None else torch.empty(
        shape, dtype=dt if case["gate"] == "token" else torch.float32, device="cuda")
    for w in ("post_weight", "pre_weight"):
        s["d" + w] = None if s[w] is None else torch.empty((C,), device="cuda")
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        from context_attention_token_gb300 import cpt

        s["plan"] = cpt.cpt_plan_create(LAYOUTS[case["layout"]], case["P"], s["cu"].tolist(), case["T"])
        if case["op"] == "residual_norm_backward":
            need = cpt.cpt_residual_norm_backward_workspace_bytes(s["plan"], case["C"], s["dy"].dtype)
            s["workspace"] = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------- plain forms

def _bits(state, tokens, columns):
    """16 random bits for every row's token and column: ten rounds of Philox-4x32 of (group of 8 columns, token,
    step, site) under the seed."""
    low = 0xFFFFFFFF
    seed, step = state["rng"][0], state["rng"][1]
    k0, k1 = seed & low, (seed >> 32) & low
    groups = torch.arange(-(-columns // 8), device="cuda")
    c0 = groups[None, :].expand(len(tokens), -1)
    c1 = tokens[:, None].expand(-1, len(groups))
    c2 = (step & low).expand_as(c0)
    c3 = torch.full_like(c0, state["site"])
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & low) ^ c1 ^ k0, b & low, ((a >> 32) & low) ^ c3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack([c0, c1, c2, c3], -1)
    return torch.stack([words & 0xFFFF, words >> 16], -1).reshape(len(tokens), -1)[:, :columns]


def _kept(p):
    """Of 2^16 values of the bits, those that keep an element."""
    return int(math.floor((1.0 - p) * 65536 + 0.5))


def _keep(state, tokens, columns, p):
    """Truth values in pieces: the generator's words are 64 bits wide here."""
    step = max(1, 2 ** 27 // columns)
    return torch.cat([_bits(state, t, columns) < _kept(p) for t in torch.split(tokens, step)])


def _dropped(x, keep, p):
    return torch.where(keep, x * (65536.0 / _kept(p)), 0.0)


def _dropout(s):
    c = s["case"]
    x, t = s["x"].reshape(s["R"], c["C"]).float(), s["tokens"]
    z = _dropped(x, _keep(s, t.clamp(min=0), c["C"], c["p"]), c["p"])
    return torch.where((t >= 0)[:, None], z, 0.0).to(s["x"].dtype).reshape(s["x"].shape)


def _rsqrt_of_mean(x):
    return torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)


def _gate_rows(s, at):
    """The gate of every row, or None."""
    if s["gate"] is None:
        return None
    if s["case"]["gate"] == "token":
        return s["gate"].reshape(s["R"], -1).float()
    return s["gate"].float()[s["doc"][at]]


def _residual_norm(s):
    c, R, t = s["case"], s["R"], s["tokens"]
    C, p, real, at = c["C"], c["p"], (t >= 0)[:, None], t.clamp(min=0)
    y = s["x"].reshape(R, C).float()
    out = []
    if s["h"] is not None:
        u = s["h"].reshape(R, C).float()
        if c["post"]:
            u = u * _rsqrt_of_mean(u) * s["post_weight"]
        gate = _gate_rows(s, at)
        if gate is not None:
            u = u * gate
        if p > 0:
            u = _dropped(u, _keep(s, at, C, p), p)
        y = torch.where(real, y + u * s["scale"], 0.0)
        out.append(y.to(s["x"].dtype).reshape(s["x"].shape))
    if c["pre"]:
        n = torch.where(real, y * _rsqrt_of_mean(y) * s["pre_weight"], 0.0)
        out.append(n.to(s["x"].dtype).reshape(s["x"].shape))
    return out


def _column_sum(x):
    return x.sum(0, dtype=torch.float64).float()


def _residual_norm_backward(s):
    c, R, t, dt = s["case"], s["R"], s["tokens"], s["dy"].dtype
    C, p, at = c["C"], c["p"], t.clamp(min=0)
    real = (t >= 0)[:, None]

    def rows(x):
        return torch.where(real, x.reshape(R, C).float(), 0.0)

    def back(x, like):
        return torch.where(real, x, 0.0).to(like.dtype).reshape(like.shape)

    d = rows(s["dy"])
    res = {}
    if c["pre"]:
        y, dn = rows(s["y"]), rows(s["dn"])
        r = _rsqrt_of_mean(y)
        y = y * r
        res["dpre_weight"] = _column_sum(dn * y)
        dn = dn * s["pre_weight"]
        d = d + r * (dn - y * (dn * y).mean(-1, keepdim=True))
        del y, dn
    res["dx"] = back(d, s["dy"])
    if s["h"] is None:
        return res
    d = d * s["scale"]
    if p > 0:
        d = _dropped(d, _keep(s, at, C, p), p)
    h = rows(s["h"])
    if c["post"]:
        r = _rsqrt_of_mean(h)
        h = h * r
    gate = _gate_rows(s, at)
    if gate is not None:
        z = d * h * s["post_weight"] if c["post"] else d * h
        if c["gate"] == "token":
            res["dgate"] = back(z, s["gate"])
        else:
            sums = torch.zeros((s["n"], C), dtype=torch.float64, device="cuda")
            doc = s["doc"][at]
            for a in range(0, R, 32768):
                sums.index_add_(0, doc[a:a + 32768], z[a:a + 32768].double())
            res["dgate"] = sums.float()
        d = d * gate
    if c["post"]:
        res["dpost_weight"] = _column_sum(d * h)
        d = d * s["post_weight"]
        d = r * (d - h * (d * h).mean(-1, keepdim=True))
    res["dh"] = back(d, s["dy"])
    return res


def _scored_rows(s):
    """Rows whose token has a target, in pieces, with the tokens."""
    t = s["tokens"]
    q = torch.nonzero((t >= 0) & s["take"][t.clamp(min=0)]).squeeze(1)
    return [(x, t[x]) for x in torch.split(q, max(1, 2 ** 29 // s["case"]["vocab"]))]


def _token_logprob(s):
    """The target's logarithm of a probability; the largest logit and the logarithm of the sum of the weights."""
    c = s["case"]
    V, R = c["vocab"], s["R"]
    logits = s["logits"].view(R, -1)
    logp, stats = torch.zeros((c["T"],), device="cuda"), torch.zeros((c["T"], 2), device="cuda")
    for q, t in _scored_rows(s):
        x = logits[q, :V].float()
        m = x.amax(-1, keepdim=True)
        x = (x - m) * c["scale"]
        l = torch.log(torch.exp(x).sum(-1))
        logp[t] = x.gather(1, s["targets"][t].long()[:, None]).squeeze(1) - l
        stats[t] = torch.stack([m.squeeze(1), l], 1)
    return logp, stats


def _token_logprob_backward(s):
    c = s["case"]
    V, R = c["vocab"], s["R"]
    logits = s["logits"].view(R, -1)
    out = torch.zeros_like(logits)
    for q, t in _scored_rows(s):
        x = logits[q, :V].float()
        p = torch.exp((x - s["stats"][t, 0:1]) * c["scale"] - s["stats"][t, 1:2])
        p = -p
        p[torch.arange(len(q), device="cuda"), s["targets"][t].long()] += 1.0
        out[q, :V] = (p * (s["dlogp"][t][:, None] * c["scale"])).to(out.dtype)
    return out.view(s["logits"].shape)


def _kl(d):
    """exp(d) - 1 - d, from its series where the terms cancel."""
    near = d * d * (0.5 + d * (1 / 6 + d * (1 / 24 + d * (1 / 120 + d * (1 / 720 + d * (1 / 5040 + d / 40320))))))
    return torch.where(d.abs() < 0.5, near, torch.expm1(d) - d)


def _policy_loss(s):
    n, doc, mask = s["n"], s["doc"], s["mask"]
    lo, hi = s["clip"]
    a = s["advantages"][doc]
    # which side of a border a ratio lies on is settled in 64 bits
    d64 = s["logp"].double() - s["old"].double()
    above, below = d64 > math.log1p(hi), d64 < math.log1p(-lo)
    ratio = torch.exp(d64.float())
    flat = (above & (a > 0)) | (below & (a < 0))
    loss = -a * torch.where(flat, torch.where(above, 1.0 + hi, 1.0 - lo), ratio)
    grad = torch.where(flat, 0.0, -a * ratio)
    kl = torch.zeros_like(loss)
    if s["ref"] is not None:
        d = (s["ref"].double() - s["logp"].double()).float()
        kl = _kl(d)
        grad = grad - s["kl"] * torch.expm1(d)

    def mean(x):
        z = torch.zeros(n, dtype=torch.float64, device="cuda")
        return z.index_add_(0, doc, torch.where(mask, x, 0.0).double())

    count = mean(torch.ones_like(loss))
    some = count.clamp(min=1.0)
    policy, kl, clipped = mean(loss) / some, mean(kl) / some, mean(flat.float()) / some
    terms = torch.stack([policy + s["kl"] * kl, kl, clipped, count], 1).float()
    return terms, torch.where(mask, grad * (s["weights"] / some).float()[doc], 0.0)


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"dropout": _dropout, "residual_norm": _residual_norm, "residual_norm_backward": _residual_norm_backward,
                "token_logprob": _token_logprob, "token_logprob_backward": _token_logprob_backward,
                "policy_loss": _policy_loss}[c["op"]](s)
    from context_attention_token_gb300 import cpt

    op = c["op"]
    if op == "policy_loss":
        cpt.cpt_policy_loss(s["plan"], s["logp"], s["old"], s["advantages"], s["terms"], s["dlogp"], logp_ref=s["ref"],
                            mask=s["mask"], weights=s["weights"], clip_low=s["clip"][0], clip_high=s["clip"][1],
                            kl_coef=s["kl"])
        return s["terms"], s["dlogp"]
    order = cpt.CPT_ORDER_LOCAL if c["order"] == "local" else cpt.CPT_ORDER_GLOBAL
    if op == "dropout":
        cpt.cpt_dropout(s["plan"], s["x"], s["out"], c["p"], s["rng"], s["site"], order=order)
        return s["out"]
    if op == "token_logprob":
        cpt.cpt_token_logprob(s["plan"], s["logits"], s["targets"], s["logp"], s["stats"], vocab=c["vocab"],
                              scale=c["scale"], order=order)
        return s["logp"], s["stats"]
    if op == "token_logprob_backward":
        cpt.cpt_token_logprob_backward(s["plan"], s["logits"], s["targets"], s["stats"], s["dlogp"], s["dlogits"],
                                       vocab=c["vocab"], scale=c["scale"], order=order)
        return s["dlogits"]
    shared = dict(post_weight=s["post_weight"], gate=s["gate"], gate_per_document=c["gate"] == "document",
                  scale=s["scale"], p=c["p"], rng=s["rng"] if c["p"] > 0 else None, site=s["site"],
                  pre_weight=s["pre_weight"], eps=EPS, order=order)
    if op == "residual_norm":
        cpt.cpt_residual_norm(s["plan"], s["x"], s["h"], s["y"], s["normed"], **shared)
        return [x for x in (s["y"], s["normed"]) if x is not None]
    cpt.cpt_residual_norm_backward(s["plan"], s["h"], s["y"], s["dy"], s["dn"], s["dx"], s["dh"], dgate=s["dgate"],
                                   dpost_weight=s["dpost_weight"], dpre_weight=s["dpre_weight"],
                                   workspace=s["workspace"], **shared)
    names = ("dx", "dh", "dgate", "dpost_weight", "dpre_weight")
    return {k: s[k] for k in names if s[k] is not None}


# ---------------------------------------------------------------- 64 bits, from the definitions

def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "policy_loss":
        return _exact_policy(s)
    if op.startswith("token"):
        return _exact_logprob(s)
    return _exact_rows(s)


def _mulhi(a, m):
    """The high word of a 32 by 32-bit product, from 16-bit halves."""
    a0, a1, m0, m1 = a & 0xFFFF, a >> 16, m & 0xFFFF, m >> 16
    mid = a1 * m0 + ((a0 * m0) >> 16)
    return a1 * m1 + (mid >> 16) + (((mid & 0xFFFF) + a0 * m1) >> 16)


def _factor(s, tokens, p):
    """1 / (share that is kept) where an element is kept, 0 where it is dropped, [tokens, C]."""
    C = s["case"]["C"]
    kept = round((1.0 - p) * 65536)
    seed, step = (int(v) % (1 << 64) for v in s["rng"].tolist())
    key = [seed % (1 << 32), seed >> 32]
    g, tok = torch.meshgrid(torch.arange((C + 7) // 8, device="cuda"), tokens, indexing="ij")
    w = [g, tok, torch.full_like(g, step % (1 << 32)), torch.full_like(g, s["site"])]
    for i in range(10):
        k = [(key[0] + i * 0x9E3779B9) % (1 << 32), (key[1] + i * 0xBB67AE85) % (1 << 32)]
        w = [_mulhi(w[2], 0xCD9E8D57) ^ w[1] ^ k[0], (w[2] * 0xCD9E8D57) & 0xFFFFFFFF,
             _mulhi(w[0], 0xD2511F53) ^ w[3] ^ k[1], (w[0] * 0xD2511F53) & 0xFFFFFFFF]
    f = torch.empty((len(tokens), g.shape[0], 8), dtype=torch.float64, device="cuda")
    for j in range(8):
        v = (w[j // 2] >> (16 * (j % 2))) & 0xFFFF
        f[:, :, j] = (v < kept).double().t()
    return f.reshape(len(tokens), -1)[:, :C] * (65536.0 / kept)


def _exact_rows(s):
    c = s["case"]
    C, R, p, op = c["C"], s["R"], c["p"], c["op"]
    real = torch.nonzero(s["tokens"] >= 0).squeeze(1)
    wide = {k: None if s.get(k) is None else torch.zeros((R, C), dtype=torch.float64, device="cuda")
            for k in ("out", "y", "normed", "dx", "dh")}
    if op == "residual_norm_backward":
        wide["y"] = None
    sums = {}
    per_doc = c.get("gate") == "document"
    if s.get("dgate") is not None:
        wide["dgate"] = torch.zeros((s["n"] if per_doc else R, C), dtype=torch.float64, device="cuda")

    def norm(x, w):
        return x / torch.sqrt(x.square().mean(1, keepdim=True) + EPS) * w

    for q in torch.split(real, max(1, 2 ** 25 // C)):
        t = s["tokens"][q]
        doc = s["doc"][t]
        pick = {k: None if s.get(k) is None else s[k].reshape(R, C)[q].double() for k in ("x", "h", "y", "dy", "dn")
                if not (op == "residual_norm" and k == "y")}
        drop = _factor(s, t, p) if p > 0 else 1.0
        if op == "dropout":
            wide["out"][q] = pick["x"] * drop
            continue
        w1, w2 = (None if s[k] is None else s[k].double().requires_grad_(True) for k in ("post_weight", "pre_weight"))
        gate = None if s["gate"] is None else s["gate"].double()[doc] if per_doc else s["gate"].reshape(R, C)[q].double()
        if gate is not None:
            gate.requires_grad_(True)

        def branch(h):
            z = h if w1 is None else norm(h, w1)
            z = z if gate is None else z * gate
            return s["scale"] * z * drop

        if op == "residual_norm":
            with torch.no_grad():
                y = pick["x"] if pick["h"] is None else pick["x"] + branch(pick["h"])
                if wide["y"] is not None:
                    wide["y"][q] = y
                if w2 is not None:
                    wide["normed"][q] = norm(y, w2)
            continue
        d = pick["dy"]
        if w2 is not None:
            y = pick["y"].requires_grad_(True)
            gy, gw = torch.autograd.grad((norm(y, w2) * pick["dn"]).sum(), (y, w2))
            d = d + gy
            sums["dpre_weight"] = sums.get("dpre_weight", 0.0) + gw
        wide["dx"][q] = d
        if pick["h"] is None:
            continue
        h = pick["h"].requires_grad_(True)
        leaves = [h] + [x for x in (gate, w1) if x is not None]
        got = list(torch.autograd.grad((branch(h) * d).sum(), leaves))
        wide["dh"][q] = got.pop(0)
        if gate is not None:
            if per_doc:
                wide["dgate"].index_add_(0, doc, got.pop(0))
            else:
                wide["dgate"][q] = got.pop(0)
        if w1 is not None:
            sums["dpost_weight"] = sums.get("dpost_weight", 0.0) + got.pop(0)
    if op == "dropout":
        return wide["out"].reshape(s["out"].shape)
    if op == "residual_norm":
        return [wide[k].reshape(s["x"].shape) for k in ("y", "normed") if wide[k] is not None]
    res = {k: wide[k].reshape(s["dy"].shape) for k in ("dx", "dh") if wide[k] is not None}
    if s["dgate"] is not None:
        res["dgate"] = wide["dgate"].reshape(s["dgate"].shape)
    res.update(sums)
    return {k: res[k] for k in ("dx", "dh", "dgate", "dpost_weight", "dpre_weight") if k in res}


def _exact_logprob(s):
    c = s["case"]
    V, R, T = c["vocab"], s["R"], c["T"]
    x = s["logits"].reshape(R, -1)
    row_of = torch.full((T,), -1, dtype=torch.int64, device="cuda")
    has = s["tokens"] >= 0
    row_of[s["tokens"][has]] = torch.nonzero(has).squeeze(1)
    scored = torch.nonzero(s["targets"] >= 0).squeeze(1)
    back = c["op"] == "token_logprob_backward"
    if back:
        out = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
    logp = torch.zeros((T,), dtype=torch.float64, device="cuda")
    stats = torch.zeros((T, 2), dtype=torch.float64, device="cuda")
    for t in torch.split(scored, max(1, 2 ** 26 // V)):
        z = x[row_of[t]][:, :V].double()
        lse = torch.logsumexp(z * c["scale"], 1)
        at = s["targets"][t].long()
        if back:
            g = -torch.exp(z * c["scale"] - lse[:, None])
            g.scatter_add_(1, at[:, None], torch.ones_like(lse)[:, None])
            out[row_of[t], :V] = g * (c["scale"] * s["dlogp"][t].double())[:, None]
            continue
        top = z.max(1).values
        logp[t] = c["scale"] * z[torch.arange(len(t), device="cuda"), at] - lse
        stats[t, 0], stats[t, 1] = top, lse - c["scale"] * top
    if back:
        return out.reshape(s["logits"].shape)
    return logp, stats


def _exact_policy(s):
    lo, hi = s["clip"]
    lp = s["logp"].double().requires_grad_(True)
    old, adv, doc = s["old"].double(), s["advantages"].double(), s["doc"]
    on = s["mask"].double()
    count = torch.zeros(s["n"], dtype=torch.float64, device="cuda").index_add_(0, doc, on)
    share = on / count.clamp(min=1.0)[doc]
    ratio = torch.exp(lp - old)
    free, held = ratio * adv[doc], ratio.clamp(1.0 - lo, 1.0 + hi) * adv[doc]
    each = -torch.minimum(free, held)
    kl = torch.zeros_like(each)
    if s["ref"] is not None:
        gap = s["ref"].double() - lp
        kl = torch.exp(gap) - gap - 1.0
        each = each + s["kl"] * kl

    def per_doc(v):
        return torch.zeros(s["n"], dtype=torch.float64, device="cuda").index_add(0, doc, v * share)

    loss = per_doc(each)
    dlogp, = torch.autograd.grad((loss * s["weights"].double()).sum(), lp)
    terms = torch.stack([loss, per_doc(kl), per_doc((held < free).double()), count], 1).detach()
    return terms, dlogp
