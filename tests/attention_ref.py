"""Plain 64-bit forms of the attention layer's operators, by brute force over
dense masks, and the error bounds that follow from the kernels' roundings.

Bounds. u = 2^-8 is the largest relative error of one rounding to bf16
(half a step). The kernels round the softmax weights p and the score
gradients ds to bf16 before they multiply (u times the sum of the absolute
products) and every output once (u times its value). The rest is binary32:
a score is a sum of at most 128 products, off by at most 128 * 2^-24 of the
sum of their absolute values, which for the inputs here (unit normals,
scale D^-1/2) stays below 2^-14; exponentials, sums and divisions add a few
2^-22. E32 = 2^-13 covers the relative error of a weight from all of them.
"""
import math

import numpy as np
import torch

U = 2.0 ** -8
E32 = 2.0 ** -13

SWAP, PACKED, PADDED = 0, 1, 3


def local_rows(layout, P, lens):
    """(l2r, l2g, cu, cup): raw token and (padded) global position of every
    local row, raw and padded boundaries."""
    lens = np.asarray(lens, dtype=np.int64)
    cu = np.concatenate([[0], np.cumsum(lens)])
    if layout == PACKED:
        at = np.arange(cu[-1])
        return at, at, cu, cu
    unit = 2 * P
    pad = (lens + unit - 1) // unit * unit
    if layout == SWAP:
        assert (pad == lens).all()
    cup = np.concatenate([[0], np.cumsum(pad)])
    l2r, l2g = [], []
    for r in range(P):
        for i, L in enumerate(lens):
            m = int(pad[i]) // unit
            for c in (r, unit - 1 - r):
                for u in range(c * m, (c + 1) * m):
                    l2g.append(cup[i] + u)
                    l2r.append(cu[i] + u if u < L else -1)
    return np.array(l2r, dtype=np.int64), np.array(l2g, dtype=np.int64), cu, cup


def visible(l2r, cu, T, window, sinks, device):
    """[Tpad, T] mask: whether a local row sees a raw token."""
    doc_of = np.repeat(np.arange(len(cu) - 1), np.diff(cu))
    pos = np.arange(T) - cu[doc_of] if T else np.zeros(0)
    g = np.maximum(l2r, 0)
    doc = torch.from_numpy(doc_of).to(device)
    u = torch.from_numpy(pos).to(device)
    gd, gu = doc[torch.from_numpy(g).to(device)], u[torch.from_numpy(g).to(device)]
    real = torch.from_numpy(l2r >= 0).to(device)
    d = gu[:, None] - u[None, :]
    return real[:, None] & (gd[:, None] == doc[None, :]) & (d >= 0) & ((d < window) | (u[None, :] < sinks))


def _masked(see, x):
    return torch.where(see, x, torch.zeros((), dtype=x.dtype, device=x.device))


def _weights(q, k, see, scale, G):
    """Scores and softmax weights [Hq, Tpad, T] in float64, zeros where hidden;
    log-sum-exp [Hq, Tpad]. What is hidden is never multiplied."""
    kk = k.double().repeat_interleave(G, 1)
    s = torch.einsum("ihd,jhd->hij", q.double(), kk) * scale
    s = torch.where(see, s, torch.full((), -math.inf, dtype=s.dtype, device=s.device))
    lse = torch.logsumexp(s, -1)
    p = torch.where(see, torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)[..., None]), 0.0)
    return p, lse


def attention64(q, k, v, see, scale):
    """out [Tpad, Hq, D], lse [Hq, Tpad] and the bound of out's error."""
    G = q.shape[1] // k.shape[1]
    p, lse = _weights(q, k, see, scale, G)
    vv = v.double().repeat_interleave(G, 1)
    out = torch.einsum("hij,jhd->ihd", p, vv)
    mag = torch.einsum("hij,jhd->ihd", p, vv.abs())
    return out, lse, (U + 2 * E32) * mag + U * (1 + U) * out.abs() + 1e-30


def backward64(q, k, v, out, dout, see, scale, P):
    """dq [Tpad, Hq, D] with the bound of its error, and for every rank the
    pairs (gradient, bound) of dk and dv, [T, Hkv, D] in raw order. delta comes
    from the given out, as the call defines it."""
    Tpad, Hq, D = q.shape
    G = Hq // k.shape[1]
    p, _ = _weights(q, k, see, scale, G)
    kk, vv = k.double().repeat_interleave(G, 1), v.double().repeat_interleave(G, 1)
    qd, do = q.double(), dout.double()
    delta = (do * out.double()).sum(-1).t()                        # [Hq, Tpad]
    dp = torch.einsum("ihd,jhd->hij", do, vv)
    mag_dp = torch.einsum("ihd,jhd->hij", do.abs(), vv.abs())
    mag_delta = (do * out.double()).abs().sum(-1).t()
    ds = _masked(see, p * (dp - delta[..., None])) * scale
    # ds: rounded once; p, dp and delta carry their binary32 errors
    err = _masked(see, p * (mag_dp + mag_delta[..., None])) * scale * 2 * E32 + U * ds.abs()
    dq = torch.einsum("hij,jhd->ihd", ds, kk)
    dq_tol = torch.einsum("hij,jhd->ihd", err, kk.abs()) + U * (1 + U) * dq.abs() + 1e-30
    return dq, dq_tol, _writers(p, ds, err, qd, do, P, G, Tpad)


def _writers(p, ds, err, qd, do, P, G, Tpad):
    Hq, _, T = p.shape
    D = qd.shape[-1]
    Tp = Tpad // P
    res = []
    for r in range(P):
        rows = slice(r * Tp, (r + 1) * Tp)
        one = []
        for w, e, x in ((ds, err, qd), (p, p * (U + 2 * E32), do)):
            g = torch.einsum("hij,ihd->jhd", w[:, rows], x[rows]).reshape(T, Hq // G, G, D).sum(2)
            m = torch.einsum("hij,ihd->jhd", e[:, rows], x[rows].abs()).reshape(T, Hq // G, G, D).sum(2)
            one.append((g, m + U * (1 + U) * g.abs() + 1e-30))
        res.append(one)
    return res


def sampled_rows(b, rows):
    """out, lse and dq of some local rows against all keys, with their bounds
    (the rows' own masks; lse and delta from b.out, b.lse)."""
    see = visible(b.l2r[rows], b.cu, b.T, b.window, b.sinks, "cuda")
    at = torch.from_numpy(rows).cuda()
    out, lse, tol = attention64(b.q[at], b.k, b.v, see, b.scale)
    dq, dq_tol, _ = backward64(b.q[at], b.k, b.v, b.out.t[at], b.dout[at], see, b.scale, 1)
    return out, lse, tol, dq, dq_tol


def sampled_keys(b, keys):
    """For every rank (dk, bound, dv, bound) of some raw keys, from the rows'
    log-sum-exp in b.lse and the outputs in b.out."""
    G, Tp = b.Hq // b.Hk, b.Tpad // b.P
    at = torch.from_numpy(keys).cuda()
    kk, vv = (x[at].double().repeat_interleave(G, 1) for x in (b.k, b.v))
    res = []
    for r in range(b.P):
        rows = slice(r * Tp, (r + 1) * Tp)
        q, do, o = b.q[rows].double(), b.dout[rows].double(), b.out.t[rows].double()
        see = visible_keys(b, rows, keys)
        s = torch.einsum("ihd,jhd->hij", q, kk) * b.scale
        p = torch.where(see, torch.exp(s - b.lse.t[:, rows, None].double()), 0.0)
        dp = torch.einsum("ihd,jhd->hij", do, vv)
        delta = (do * o).sum(-1).t()[..., None]
        mag = torch.einsum("ihd,jhd->hij", do.abs(), vv.abs()) + (do * o).abs().sum(-1).t()[..., None]
        ds = torch.where(see, p * (dp - delta), 0.0) * b.scale
        err = torch.where(see, p * mag, 0.0) * b.scale * 2 * E32 + U * ds.abs()
        one = []
        for w, e, x in ((ds, err, q), (p, p * (U + 2 * E32), do)):
            g = torch.einsum("hij,ihd->jhd", w, x).reshape(len(keys), b.Hk, G, b.D).sum(2)
            m = torch.einsum("hij,ihd->jhd", e, x.abs()).reshape(len(keys), b.Hk, G, b.D).sum(2)
            one.append((g, m + U * (1 + U) * g.abs() + 1e-30))
        res.append(one)
    return res


def visible_keys(b, rows, keys):
    l2r = b.l2r[rows]
    doc = np.searchsorted(b.cu, np.maximum(l2r, 0), side="right") - 1
    kdoc = np.searchsorted(b.cu, keys, side="right") - 1
    u = torch.from_numpy(np.maximum(l2r, 0) - b.cu[doc]).cuda()[:, None]
    j = torch.from_numpy(keys - b.cu[kdoc]).cuda()[None]
    same = torch.from_numpy(doc).cuda()[:, None] == torch.from_numpy(kdoc).cuda()[None]
    real = torch.from_numpy(l2r >= 0).cuda()[:, None]
    return real & same & (u >= j) & ((u - j < b.window) | (j < b.sinks))


def to_padded(x, cu, cup, Tpad):
    """Raw global rows placed in padded global order, zeros in padding."""
    out = torch.zeros((Tpad,) + tuple(x.shape[1:]), dtype=x.dtype, device=x.device)
    at = np.arange(cu[-1]) + np.repeat(cup[:-1] - cu[:-1], np.diff(cu))
    out[torch.from_numpy(at).to(x.device)] = x
    return out


def rotate64(x, pos, inv_freq, axis, interleaved, inverse):
    """x [T, H, D] (numpy float64) rotated by pos [axes, T]."""
    n = len(inv_freq)
    theta = np.stack([pos[a].astype(np.float64) * f for a, f in zip(axis, inv_freq)], 1)[:, None, :]
    c, s = np.cos(theta), np.sin(theta) * (-1.0 if inverse else 1.0)
    y = x.copy()
    if interleaved:
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        y[..., 0:2 * n:2], y[..., 1:2 * n:2] = a * c - b * s, a * s + b * c
    else:
        a, b = x[..., :n], x[..., n:2 * n]
        y[..., :n], y[..., n:2 * n] = a * c - b * s, a * s + b * c
    return y
