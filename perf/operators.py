"""The context-parallel attention layer's operators, as measured.

Three operators stand between the Q/K/V reorder and the owner-gradient return:

  rotary              rotary positions with several axes (time, height, width),
                      applied while the tokens move between global order and
                      rank-local order, and its gradient (the inverse rotation
                      on the way back);
  attention           causal attention over packed documents with a sliding
                      window and a few first tokens of each document that stay
                      visible; queries in rank-local order, keys and values in
                      global order;
  attention_backward  its gradient: dQ in rank-local order, and every rank's
                      dK and dV in that writer's global slot, which is what the
                      gradient return sums.

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
        {"name": "rotary_tiny", "op": "rotary", "order": "partition", "inverse": False, "layout": "swap", "P": 2,
         "T": 64, "median": 16, "heads": 2, "kv": 2, "D": 8, "axes": 1, "pairs": 4, "interleaved": False, "dtype": "f32"},
        # images and text in one batch, documents of any length: Q and K rotated into rank-local order
        {"name": "rotary_partition_packed_docs", "op": "rotary", "order": "partition", "inverse": False,
         "layout": "padded", "P": 4, "T": 131071, "median": 2048, "heads": 16, "kv": 16, "D": 128, "axes": 3,
         "pairs": 64, "interleaved": False, "dtype": "bf16"},
        # the gradients of Q and K of one long causal sequence, turned back where they lie
        {"name": "rotary_gradient_long", "op": "rotary", "order": "local", "inverse": True, "layout": "swap", "P": 4,
         "T": 262144, "median": 0, "heads": 20, "kv": 20, "D": 128, "axes": 3, "pairs": 64, "interleaved": False,
         "dtype": "bf16"},
        # a partial rotation of float32 heads of odd size, returned to global order
        {"name": "rotary_restore_partial_f32", "op": "rotary", "order": "restore", "inverse": True, "layout": "padded",
         "P": 3, "T": 20011, "median": 700, "heads": 6, "kv": 2, "D": 72, "axes": 2, "pairs": 18, "interleaved": True,
         "dtype": "f32"},
        # latency: a few short documents
        {"name": "attention_tiny", "op": "attention", "layout": "swap", "P": 2, "T": 128, "median": 32, "heads": 2,
         "kv": 1, "D": 64, "window": 32, "sinks": 2, "dtype": "bf16"},
        # one document of ordinary length, window and sinks
        {"name": "attention_document", "op": "attention", "layout": "swap", "P": 4, "T": 32768, "median": 0, "heads": 8,
         "kv": 8, "D": 128, "window": 4096, "sinks": 4, "dtype": "bf16"},
        # a packed batch of documents of any length, grouped heads, heads of 80
        {"name": "attention_packed_docs", "op": "attention", "layout": "padded", "P": 4, "T": 65521, "median": 2048,
         "heads": 16, "kv": 4, "D": 80, "window": 1000, "sinks": 5, "dtype": "bf16"},
        # the longest sequence, a window of 2048
        {"name": "attention_long", "op": "attention", "layout": "swap", "P": 4, "T": 262144, "median": 0, "heads": 20,
         "kv": 20, "D": 128, "window": 2048, "sinks": 16, "dtype": "bf16"},
        # latency of a gradient: a few short documents
        {"name": "backward_tiny", "op": "attention_backward", "layout": "swap", "P": 2, "T": 128, "median": 32,
         "heads": 2, "kv": 1, "D": 64, "window": 32, "sinks": 2, "dtype": "bf16"},
        # the whole causal triangle: a window as long as the document
        {"name": "backward_full_causal", "op": "attention_backward", "layout": "swap", "P": 4, "T": 8192, "median": 0,
         "heads": 16, "kv": 16, "D": 128, "window": 8192, "sinks": 0, "dtype": "bf16"},
        # a packed batch in equal chunks, grouped heads of 64
        {"name": "backward_packed_docs", "op": "attention_backward", "layout": "packed", "P": 4, "T": 65536,
         "median": 2048, "heads": 16, "kv": 4, "D": 64, "window": 1000, "sinks": 5, "dtype": "bf16"},
        # one long document, window and sinks
        {"name": "backward_document", "op": "attention_backward", "layout": "swap", "P": 4, "T": 32768, "median": 0,
         "heads": 20, "kv": 20, "D": 128, "window": 4096, "sinks": 4, "dtype": "bf16"},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "attention", "attention", "attention_backward", "attention_backward"])
    while True:
        layout = rng.choice(["swap", "packed", "padded"])
        P = rng.choice([1, 2, 3, 4, 8])
        T = _log_uniform(rng, 64, 262144 if op == "rotary" else 131072)
        T -= T % (1 if layout == "padded" else P if layout == "packed" else 2 * P)
        kv = rng.choice([1, 2, 4, 5, 8])
        heads = kv * rng.choice([1, 1, 2, 3, 4])
        c = {"op": op, "layout": layout, "P": P, "T": T, "median": rng.choice([0, _log_uniform(rng, 64, 8192)]),
             "heads": heads, "kv": kv}
        if op == "rotary":
            D = rng.choice([16, 64, 72, 80, 96, 128, 256])
            pairs = rng.choice([D // 2, D // 2, D // 4])
            order = rng.choice(["partition", "restore", "local", "global"])
            dtype = rng.choice(["bf16", "bf16", "f32"])
            c.update(order=order, inverse=rng.random() < 0.5, D=D, axes=rng.choice([1, 2, 3, 4]), pairs=pairs,
                     interleaved=rng.random() < 0.3, dtype=dtype)
            if T > 0 and T * (heads + kv) * D * (2 if dtype == "bf16" else 4) <= 262144 * 40 * 128 * 2:
                return c
            continue
        D = rng.choice([32, 64, 64, 80, 96, 128, 128, 128])
        window = _log_uniform(rng, 16, 16384)
        c.update(D=D, window=window, sinks=rng.choice([0, 0, 1, 4, 16, 100]), dtype="bf16")
        if T <= 0 or T * heads * D > 65536 * 16 * 128:
            continue
        if T * heads * min(T, window) <= 32768 * 16 * 4096:
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
    """Raw row of every local row, rank-major (-1: a padding row), the global
    position of every local row, the raw boundaries and the global ones."""
    P, kind = case["P"], case["layout"]
    lens = np.array(_lengths(case), dtype=np.int64)
    cu = np.concatenate([[0], np.cumsum(lens)])
    if kind == "packed":
        at = np.arange(case["T"], dtype=np.int64)
        return at, at, cu, cu
    pad = -(-lens // (2 * P)) * (2 * P)
    cup = np.concatenate([[0], np.cumsum(pad)])
    l2r, l2g = [], []
    for r in range(P):
        for i in range(len(lens)):
            m = pad[i] // (2 * P)
            u = np.concatenate([np.arange(r * m, (r + 1) * m), np.arange((2 * P - 1 - r) * m, (2 * P - r) * m)])
            l2g.append(cup[i] + u)
            l2r.append(np.where(u < lens[i], cu[i] + u, -1))
    return np.concatenate(l2r), np.concatenate(l2g), cu, cup


def _runs(case):
    """(first local row, first raw row, rows, first raw row of the document,
    rank) of every run of rows that are neighbours both ways."""
    l2r, _, cu, _ = _layout(case)
    Tp = len(l2r) // case["P"]
    doc = np.searchsorted(cu, l2r, side="right") - 1
    new = np.ones(len(l2r), dtype=bool)
    new[1:] = (l2r[1:] != l2r[:-1] + 1) | (doc[1:] != doc[:-1])
    new[::max(Tp, 1)] = True
    at = np.flatnonzero(new)
    n = np.diff(np.append(at, len(l2r)))
    keep = l2r[at] >= 0
    at, n = at[keep], n[keep]
    return np.stack([at, l2r[at], n, cu[doc[at]], at // Tp], 1)


def _blocks(case):
    """The runs cut into blocks of at most B rows, with the keys of each."""
    runs = _runs(case)
    W, S = case["window"], case["sinks"]
    B = int(min(256, -(-int(runs[:, 2].max()) // 16) * 16))
    parts = []
    for q0, g0, n, kb, r in runs.tolist():
        for b in range(0, n, B):
            g = g0 + b
            parts.append((q0 + b, g, min(B, n - b), kb, r, max(kb, g - W + 1)))
    parts = np.array(parts, dtype=np.int64)
    keys = int((parts[:, 1] + parts[:, 2] - parts[:, 5]).max())
    return parts, B, keys, S


def _pairs(case):
    """Query-key pairs that are visible."""
    W, S, total = case["window"], case["sinks"], 0
    for L in _lengths(case):
        u = np.arange(L, dtype=np.int64) + 1
        total += int(np.minimum(u, W).sum() + np.minimum(S, np.maximum(u - W, 0)).sum())
    return total


def _sizes(case):
    l2r, _, _, _ = _layout(case)
    return len(l2r)


def work(case):
    Tpad, T, D, H, Hk = _sizes(case), case["T"], case["D"], case["heads"], case["kv"]
    if case["op"] == "rotary":
        e = 2 if case["dtype"] == "bf16" else 4
        rows = {"partition": (T, Tpad), "restore": (T, T), "local": (T, Tpad), "global": (T, T)}[case["order"]]
        return {"bytes": sum(rows) * (H + Hk) * D * e + 4 * T * case["axes"], "flops": 6 * T * (H + Hk) * case["pairs"]}
    q, k, pairs = 2 * Tpad * H * D, 2 * T * Hk * D, _pairs(case)
    if case["op"] == "attention":
        return {"bytes": 2 * q + 2 * k + 4 * H * Tpad, "flops": 4 * D * H * pairs}
    return {"bytes": 4 * q + 2 * k + 4 * H * Tpad + 2 * case["P"] * 2 * Tpad * Hk * D, "flops": 10 * D * H * pairs}


# ---------------------------------------------------------------- inputs

def _normal(shape, dtype, g, sigma=1.0):
    t = torch.randn(shape, dtype=torch.float32, device="cuda", generator=g)
    return (t if sigma == 1.0 else t.mul_(sigma)).to(dtype)


def _inv_freq(case):
    n = case["pairs"]
    return [10000.0 ** (-i / n) for i in range(n)]


def _axis_of_pair(case):
    n, a = case["pairs"], case["axes"]
    return [i * a // n for i in range(n)]


def _positions(case, g):
    """Positions of every raw token: time runs on, height and width lie in a
    frame of some hundred patches a side."""
    T, dev = case["T"], "cuda"
    base = torch.randint(0, 1 << 16, (1,), device=dev, generator=g)
    rows = [torch.arange(T, device=dev) + base]
    rows += [torch.randint(0, 300, (T,), device=dev, generator=g) for _ in range(case["axes"] - 1)]
    return torch.stack(rows).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 17)
    T, P, H, Hk, D = case["T"], case["P"], case["heads"], case["kv"], case["D"]
    l2r, l2g, cu, cup = _layout(case)
    Tpad = len(l2r)
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    s = {"case": case, "Tpad": Tpad}
    if own:
        from context_attention_token_gb300 import cpt

        s["plan"] = cpt.cpt_plan_create(LAYOUTS[case["layout"]], P, cu.tolist(), T)
    if case["op"] == "rotary":
        local = (P, Tpad // P)
        src, dst = {"partition": ((T,), local), "restore": (local, (T,)), "local": (local, local),
                    "global": ((T,), (T,))}[case["order"]]
        s["src"] = [_normal(src + (h, D), dt, g) for h in (H, Hk)]
        s["dst"] = [torch.empty(dst + (h, D), dtype=dt, device="cuda") for h in (H, Hk)]
        s["positions"] = _positions(case, g)
        s["inv_freq"], s["axis"] = _inv_freq(case), _axis_of_pair(case)
        s["freq"] = torch.tensor(s["inv_freq"], dtype=torch.float64, device="cuda")
        s["axis_at"] = torch.tensor(s["axis"], device="cuda")
        s["l2r"] = torch.from_numpy(l2r).cuda()
        if own:
            s["rotary"] = cpt.cpt_rotary_create(D, s["inv_freq"], s["axis"], case["axes"],
                                                cpt.CPT_ROTARY_INTERLEAVED if case["interleaved"] else cpt.CPT_ROTARY_HALF)
        return s
    s["q"] = _normal((P, Tpad // P, H, D), dt, g)
    s["k"], s["v"] = (_normal((T, Hk, D), dt, g) for _ in range(2))
    parts, s["B"], s["keys"], _ = _blocks(case)
    s["parts"] = torch.from_numpy(parts).cuda()
    s["raw_to_global"] = torch.from_numpy(
        np.arange(T, dtype=np.int64) + np.repeat(cup[:-1] - cu[:-1], np.diff(cu))).cuda()
    s["scale"] = D ** -0.5
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((H, Tpad), dtype=torch.float32, device="cuda")
    if case["op"] == "attention_backward":
        s["dout"] = _normal((P, Tpad // P, H, D), dt, g)
        out, lse = _attention(s)
        s["out"].copy_(out)
        s["lse"].copy_(lse)
        del out, lse
        s["dq"] = torch.empty_like(s["q"])
        s["dk"], s["dv"] = (torch.empty((P, Tpad, Hk, D), dtype=dt, device="cuda") for _ in range(2))
        if own:
            need = cpt.cpt_attention_backward_workspace_bytes(s["plan"], H, Hk, D)
            s["workspace"] = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------- plain forms

def _rotary(s):
    c = s["case"]
    n, D, order = c["pairs"], c["D"], c["order"]
    angle = s["positions"].double()[s["axis_at"]].t() * s["freq"]  # [T, n]
    cos = torch.cos(angle).float()
    sin = torch.sin(angle).float() * (-1.0 if c["inverse"] else 1.0)
    l2r, Tpad = s["l2r"], s["Tpad"]
    real = (l2r >= 0)[:, None, None]
    at = l2r.clamp(min=0)
    if order in ("partition", "local"):
        cos, sin = cos[at], sin[at]
    cos, sin = cos[:, None, :], sin[:, None, :]
    out = []
    for x, y in zip(s["src"], s["dst"]):
        x = x.reshape((-1,) + x.shape[-2:])
        if order == "partition":
            x = x[at]
        elif order == "restore":
            back = torch.empty(c["T"] + 1, dtype=torch.int64, device="cuda")
            back[torch.where(l2r >= 0, l2r, c["T"])] = torch.arange(Tpad, device="cuda")
            x = x[back[:-1]]
        x = x.float()
        a, b = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if c["interleaved"] else (x[..., :n], x[..., n:2 * n])
        u, v = a * cos - b * sin, a * sin + b * cos
        z = torch.stack([u, v], -1).flatten(-2) if c["interleaved"] else torch.cat([u, v], -1)
        z = torch.cat([z, x[..., 2 * n:]], -1)
        if order in ("partition", "local"):
            z = torch.where(real, z, 0.0)
        out.append(z.to(y.dtype).reshape(y.shape))
    return out


def _scores(s, part, q, k):
    """Rows, keys, and the masked scores of some blocks of queries."""
    c, B = s["case"], s["B"]
    W, S = c["window"], c["sinks"]
    q0, g0, n, kb, _, lo = (x[:, None] for x in part.unbind(1))
    b = torch.arange(B, device="cuda")
    g = (g0 + b)[:, :, None]
    rows = torch.where(b < n, q0 + b, s["Tpad"])
    sink = kb + torch.arange(S, device="cuda")
    key = lo + torch.arange(s["keys"], device="cuda")
    last = g0 + n
    idx = torch.cat([torch.where(sink < lo, sink, last), key], 1)
    j = idx[:, None, :]
    see = (j <= g) & ((j > g - W) | (j < (kb + S)[:, :, None])) & (b < n)[:, :, None] & (j < last[:, :, None])
    idx = torch.where(idx < last, idx, lo)
    nb, H, Hk, D = len(part), c["heads"], c["kv"], c["D"]
    G = H // Hk
    qb = q[rows].reshape(nb, B, Hk, G, D).permute(0, 2, 3, 1, 4).reshape(nb, Hk, G * B, D)
    kb_ = k[idx].transpose(1, 2)
    sc = (qb @ kb_.transpose(2, 3)).mul_(s["scale"]).reshape(nb, Hk, G, B, -1)
    sc.masked_fill_(~see[:, None, None], -math.inf)
    m = sc.amax(-1, keepdim=True)
    m = torch.where(m > -math.inf, m, 0.0)
    p = sc.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    return rows, idx, qb, kb_, p, m, l


def _groups(s):
    """The blocks in groups whose scores stay below some 2 GB."""
    c = s["case"]
    step = max(1, int(2 ** 29 // (c["heads"] * s["B"] * (s["keys"] + c["sinks"]))))
    return torch.split(s["parts"], step)


def _with_dummy(x, rows):
    x = x.reshape((rows,) + x.shape[-2:]).float()
    return torch.cat([x, x.new_zeros((1,) + x.shape[1:])])


def _attention(s):
    c, Tpad = s["case"], s["Tpad"]
    H, Hk, D, B = c["heads"], c["kv"], c["D"], s["B"]
    q, k, v = _with_dummy(s["q"], Tpad), s["k"].float(), s["v"].float()
    out = torch.zeros((Tpad + 1, H, D), device="cuda")
    lse = torch.full((Tpad + 1, H), -math.inf, device="cuda")
    for part in _groups(s):
        rows, idx, _, _, p, m, l = _scores(s, part, q, k)
        nb = len(part)
        o = p.reshape(nb, Hk, -1, idx.shape[1]) @ v[idx].transpose(1, 2)
        o = o.reshape(nb, Hk, -1, B, D) / torch.where(l > 0, l, 1.0)
        out[rows] = o.permute(0, 3, 1, 2, 4).reshape(nb, B, H, D)
        lse[rows] = (m + torch.log(l)).squeeze(-1).permute(0, 3, 1, 2).reshape(nb, B, H)
    return out[:-1].to(s["out"].dtype).reshape(s["out"].shape), lse[:-1].t().contiguous()


def _attention_backward(s):
    c, Tpad = s["case"], s["Tpad"]
    P, T, H, Hk, D, B = c["P"], c["T"], c["heads"], c["kv"], c["D"], s["B"]
    q, do = _with_dummy(s["q"], Tpad), _with_dummy(s["dout"], Tpad)
    k, v = s["k"].float(), s["v"].float()
    dq = torch.zeros((Tpad + 1, H, D), device="cuda")
    dk, dv = (torch.zeros((P * Tpad, Hk, D), device="cuda") for _ in range(2))
    for part in _groups(s):
        rows, idx, qb, kb, p, _, l = _scores(s, part, q, k)
        nb = len(part)
        p = p.div_(torch.where(l > 0, l, 1.0)).reshape(nb, Hk, -1, idx.shape[1])
        dob = do[rows].reshape(nb, B, Hk, H // Hk, D).permute(0, 2, 3, 1, 4).reshape(nb, Hk, -1, D)
        dp = dob @ v[idx].transpose(1, 2).transpose(2, 3)
        ds = (dp.sub_((p * dp).sum(-1, keepdim=True))).mul_(p).mul_(s["scale"])
        dq[rows] = (ds @ kb).reshape(nb, Hk, -1, B, D).permute(0, 3, 1, 2, 4).reshape(nb, B, H, D)
        at = (part[:, 4:5] * Tpad + s["raw_to_global"][idx]).reshape(-1)
        dk.index_add_(0, at, (ds.transpose(2, 3) @ qb).transpose(1, 2).reshape(-1, Hk, D))
        dv.index_add_(0, at, (p.transpose(2, 3) @ dob).transpose(1, 2).reshape(-1, Hk, D))
    dt = s["dq"].dtype
    return dq[:-1].to(dt).reshape(s["dq"].shape), dk.to(dt).reshape(s["dk"].shape), dv.to(dt).reshape(s["dv"].shape)


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"rotary": _rotary, "attention": _attention, "attention_backward": _attention_backward}[c["op"]](s)
    from context_attention_token_gb300 import cpt

    if c["op"] == "rotary":
        src, dst = {"partition": (cpt.CPT_ORDER_GLOBAL, cpt.CPT_ORDER_LOCAL),
                    "restore": (cpt.CPT_ORDER_LOCAL, cpt.CPT_ORDER_GLOBAL),
                    "local": (cpt.CPT_ORDER_LOCAL, cpt.CPT_ORDER_LOCAL),
                    "global": (cpt.CPT_ORDER_GLOBAL, cpt.CPT_ORDER_GLOBAL)}[c["order"]]
        cpt.cpt_rotary_apply(s["rotary"], s["plan"], s["src"], s["dst"], s["positions"], src, dst, c["inverse"])
        return s["dst"]
    if c["op"] == "attention":
        cpt.cpt_attention(s["plan"], s["q"], s["k"], s["v"], s["out"], s["lse"], s["scale"], c["window"], c["sinks"])
        return s["out"], s["lse"]
    cpt.cpt_attention_backward(s["plan"], s["q"], s["k"], s["v"], s["out"], s["lse"], s["dout"], s["dq"], s["dk"],
                               s["dv"], s["scale"], c["window"], c["sinks"], workspace=s["workspace"])
    return s["dq"], s["dk"], s["dv"]


# ---------------------------------------------------------------- 64 bits, from the definitions

def exact(case, seed):
    if case["op"] != "rotary" and 10 * case["D"] * case["heads"] * _pairs(case) > 4e12:
        return None
    s = prepare(case, seed)
    P, T, D, H, Hk = case["P"], case["T"], case["D"], case["heads"], case["kv"]
    l2r, l2g, cu, cup = _layout(case)
    Tpad = len(l2r)
    if case["op"] == "rotary":
        return _exact_rotary(case, s, l2r, Tpad)
    G, W, S = H // Hk, case["window"], case["sinks"]
    q = s["q"].reshape(Tpad, Hk, G, D).double()
    k, v = s["k"].double(), s["v"].double()
    back = case["op"] == "attention_backward"
    out = torch.zeros((Tpad, Hk, G, D), dtype=torch.float64, device="cuda")
    lse = torch.full((Tpad, Hk, G), -math.inf, dtype=torch.float64, device="cuda")
    if back:
        do = s["dout"].reshape(Tpad, Hk, G, D).double()
        dk, dv = (torch.zeros((P, Tpad, Hk, D), dtype=torch.float64, device="cuda") for _ in range(2))
    doc = np.searchsorted(cu, l2r, side="right") - 1
    doc[l2r < 0] = -1
    cuts = np.flatnonzero(np.diff(doc)) + 1
    for rows in np.split(np.arange(Tpad), np.union1d(cuts, np.arange(0, Tpad, max(1, Tpad // P)))):
        if len(rows) == 0 or doc[rows[0]] < 0:
            continue
        d = doc[rows[0]]
        r = rows[0] // (Tpad // P)
        for a in range(0, len(rows), 512):
            qi = rows[a:a + 512]
            u = l2r[qi] - cu[d]
            # every key that some row of the piece sees, by brute force over the document
            near = np.zeros(u.max() + 1, dtype=bool)
            near[:S] = True
            for x, y in ((x[0], x[-1]) for x in np.split(u, np.flatnonzero(np.diff(u) != 1) + 1)):
                near[max(0, x - W + 1):y + 1] = True
            kj = np.flatnonzero(near)
            ut, jt = torch.from_numpy(u).cuda()[:, None], torch.from_numpy(kj).cuda()[None, :]
            hide = (jt > ut) | ((ut - jt >= W) & (jt >= S))
            qt, kt = torch.from_numpy(qi).cuda(), torch.from_numpy(kj).cuda()
            K, V = k[cu[d] + kt], v[cu[d] + kt]
            z = torch.einsum("ihgd,jhd->hgij", q[qt], K) * s["scale"]
            z[:, :, hide] = -math.inf
            ls = torch.logsumexp(z, -1)
            p = torch.exp(z - ls[..., None])
            if not back:
                out[qt] = torch.einsum("hgij,jhd->ihgd", p, V)
                lse[qt] = ls.permute(2, 0, 1)
                continue
            dp = torch.einsum("ihgd,jhd->hgij", do[qt], V)
            ds = p * (dp - (p * dp).sum(-1, keepdim=True))
            out[qt] = torch.einsum("hgij,jhd->ihgd", ds, K) * s["scale"]
            at = cup[d] + kt
            dk[r, at] += torch.einsum("hgij,ihgd->jhd", ds, q[qt]) * s["scale"]
            dv[r, at] += torch.einsum("hgij,ihgd->jhd", p, do[qt])
    if back:
        return out.reshape(s["dq"].shape), dk, dv
    return out.reshape(s["out"].shape), lse.reshape(Tpad, H).t().contiguous()


def _exact_rotary(case, s, l2r, Tpad):
    n, sign = case["pairs"], -1.0 if case["inverse"] else 1.0
    pos = s["positions"].cpu().numpy().astype(np.float64)
    theta = np.stack([pos[a] * f for a, f in zip(s["axis"], s["inv_freq"])], 1)
    turn = torch.from_numpy(np.cos(theta) + 1j * sign * np.sin(theta)).cuda()[:, None, :]
    T, D, order = case["T"], case["D"], case["order"]
    real = torch.from_numpy(np.flatnonzero(l2r >= 0)).cuda()
    raw = torch.from_numpy(l2r[l2r >= 0]).cuda()
    got = []
    for x, y in zip(s["src"], s["dst"]):
        x = x.reshape(-1, y.shape[-2], D).double()
        tokens = torch.zeros((T,) + tuple(x.shape[1:]), dtype=torch.float64, device="cuda")
        if order in ("partition", "global"):
            tokens.copy_(x)
        else:
            tokens[raw] = x[real]
        w = tokens[..., :2 * n]
        z = torch.complex(w[..., 0::2].contiguous(), w[..., 1::2].contiguous()) if case["interleaved"] else \
            torch.complex(w[..., :n].contiguous(), w[..., n:].contiguous())
        z = z * turn
        if case["interleaved"]:
            tokens[..., 0:2 * n:2], tokens[..., 1:2 * n:2] = z.real, z.imag
        else:
            tokens[..., :n], tokens[..., n:2 * n] = z.real, z.imag
        if order in ("partition", "local"):
            res = torch.zeros((Tpad,) + tuple(x.shape[1:]), dtype=torch.float64, device="cuda")
            res[real] = tokens[raw]
            tokens = res
        got.append(tokens.reshape(y.shape))
    return got
