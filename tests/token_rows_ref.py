"""64-bit forms of the calls that work on token rows, with the bounds that the kernels are held to.

u = 2^-24 is half a step of binary32. Bounds count roundings: a row's sum of squares is added by every thread
over its unit (8 terms), then over 10 levels, then divided, offset and its root taken, so the statistic is off by fewer than
16 u; every product after it by one u. Results of bf16 are rounded once more, by 2^-8 of themselves (half a step
relative to the value, at most).
"""
import numpy as np
import torch

U = 2.0 ** -24


def philox(key, ctr):
    """Ten rounds of Philox-4x32 on uint64 arrays of 32-bit words."""
    c, k = [np.asarray(x, dtype=np.uint64) for x in ctr], [int(key[0]), int(key[1])]
    low, s = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> s) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> s) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) % 2 ** 32, (k[1] + 0xBB67AE85) % 2 ** 32]
    return c


def keep(seed, step, site, tokens, columns, p):
    """Truth values [tokens, columns]: which elements a dropout keeps."""
    seed, step = seed % 2 ** 64, step % 2 ** 64
    t = np.asarray(tokens, dtype=np.uint64)[:, None]
    g = np.arange((columns + 7) // 8, dtype=np.uint64)[None, :]
    shape = (t.shape[0], g.shape[1])
    words = philox((seed % 2 ** 32, seed >> 32),
                   (np.broadcast_to(g, shape), np.broadcast_to(t, shape), np.full(shape, step % 2 ** 32, dtype=np.uint64),
                    np.full(shape, site, dtype=np.uint64)))
    w = np.stack(words, -1)
    bits = np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], -1).reshape(shape[0], -1)[:, :columns]
    return bits < kept(p)


def kept(p):
    return int(np.floor((1.0 - p) * 65536 + 0.5))


def factor(seed, step, site, tokens, columns, p):
    k = kept(p)
    m = keep(seed, step, site, tokens, columns, p)
    return torch.from_numpy(m.astype(np.float64) * (65536.0 / k if k else 0.0)).cuda()


def bound(got_dtype, exact, mag):
    """What a result may be off: `mag` in binary32, and its rounding."""
    return mag + (2.0 ** -8 * exact.abs() if got_dtype == torch.bfloat16 else 2 * U * exact.abs())


def close(got, exact, mag, what=""):
    """`got` against 64 bits: equal where exact is not finite, within the bound elsewhere."""
    g = got.double()
    fin = torch.isfinite(exact)
    assert torch.equal(torch.isnan(g), torch.isnan(exact)), f"{what}: NaN in other places"
    assert torch.equal(g[~fin & ~torch.isnan(exact)], exact[~fin & ~torch.isnan(exact)]), what
    off = ((g - exact).abs() - bound(got.dtype, exact, mag))[fin]
    assert off.numel() == 0 or off.max().item() <= 0, f"{what}: off by {off.max().item()} more than its bound"


def rows_of(l2r, order, T):
    """Raw token of every row (-1: padding), as a CUDA tensor."""
    return torch.from_numpy(np.asarray(l2r if order else np.arange(T), dtype=np.int64)).cuda()


def norm(x, eps):
    return 1.0 / torch.sqrt(x.square().mean(1, keepdim=True) + eps)


def residual_norm(x, h, gate, post, pre, scale, drop, eps):
    """(y, bound of y, n, bound of n) of real rows, float64 [rows, C]; gate and drop [rows, C] or None."""
    y, ymag = x, torch.zeros_like(x)
    if h is not None:
        b = h
        if post is not None:
            b = b * norm(h, eps) * post
        if gate is not None:
            b = b * gate
        b = b * scale if drop is None else torch.where(drop > 0, b * (drop * scale), 0.0)
        y = x + b
        ymag = 32 * U * b.abs() + 2 * U * x.abs()
    if pre is None:
        return y, ymag, None, None
    r = norm(y, eps)
    n = y * r * pre
    # an error of y reaches n by itself and through the row's statistic
    rms = torch.sqrt(y.square().mean(1, keepdim=True))
    nmag = ymag * r * pre.abs() + n.abs() * (24 * U + torch.sqrt(ymag.square().mean(1, keepdim=True)) / rms.clamp(min=1e-30))
    return y, ymag, n, nmag


def residual_norm_backward(h, y, dy, dn, gate, post, pre, scale, drop, eps):
    """Dictionary of (gradient, bound) per token: dx, dh, dgate, and per-token terms of dpost, dpre."""
    out = {}
    d = torch.zeros_like(dn if dy is None else dy) if dy is None else dy
    mag = d.abs()
    if pre is not None:
        r = norm(y, eps)
        yn, e = y * r, dn * pre
        d = d + r * (e - yn * (e * yn).mean(1, keepdim=True))
        mag = mag + r * (e.abs() + yn.abs() * (e * yn).abs().mean(1, keepdim=True))
        out["dpre"] = (dn * yn, 32 * U * (dn * yn).abs())
    out["dx"] = (d, 64 * U * mag)
    if h is None:
        return out
    f = scale if drop is None else drop * scale
    d, mag = d * f, mag * abs(f) if drop is None else mag * f.abs()
    hn = h if post is None else h * norm(h, eps)
    w = 1.0 if post is None else post
    if gate is not None:
        out["dgate"] = (d * hn * w, 96 * U * (mag * hn * w).abs())
        d, mag = d * gate, mag * gate.abs()
    if post is not None:
        out["dpost"] = (d * hn, 96 * U * (mag * hn).abs())
        r = norm(h, eps)
        e, em = d * w, mag * abs(w)
        d = r * (e - hn * (e * hn).mean(1, keepdim=True))
        mag = r * (em + hn.abs() * (em * hn.abs()).mean(1, keepdim=True))
    out["dh"] = (d, 160 * U * mag)
    return out


def layout(kind, P, lens):
    """(raw token of every local row, boundaries); kind 0: chunks swapped, 1: packed, 3: padded."""
    lens = np.asarray(lens, dtype=np.int64)
    cu = np.concatenate([[0], np.cumsum(lens)])
    if kind == 1:
        return np.arange(cu[-1]), cu
    pad = -(-lens // (2 * P)) * (2 * P)
    rows = []
    for r in range(P):
        for i, L in enumerate(lens):
            m = pad[i] // (2 * P)
            u = np.concatenate([np.arange(r * m, (r + 1) * m), np.arange((2 * P - 1 - r) * m, (2 * P - r) * m)])
            rows.append(np.where(u < L, cu[i] + u, -1))
    return np.concatenate(rows + [np.zeros(0, dtype=np.int64)]).astype(np.int64), cu


class Batch:
    """A plan with its maps, for one row order."""

    def __init__(self, cpt, kind, P, lens, order):
        l2r, cu = layout(kind, P, lens)
        self.cpt, self.P, self.lens, self.order = cpt, P, list(lens), order
        self.T, self.n = int(cu[-1]), len(lens)
        self.plan = cpt.cpt_plan_create(kind, P, cu.tolist(), self.T)
        self.tokens = rows_of(l2r, order, self.T)          # raw token of every row
        self.R = len(self.tokens)
        self.real = torch.nonzero(self.tokens >= 0).squeeze(1)
        self.at = self.tokens[self.real]                   # raw token of every real row
        self.doc = torch.from_numpy(np.repeat(np.arange(self.n), self.lens)).cuda()
        self.lead = (P, self.R // P) if order else (self.R,)

    def randn(self, g, *row, dtype=torch.float32, sigma=1.0):
        return (torch.randn(self.lead + row, device="cuda", generator=g) * sigma).to(dtype)

    def flat(self, t):
        return t.reshape(self.R, -1 if self.R else t.shape[-1])

    def pick(self, t):
        """Real rows in float64."""
        return self.flat(t)[self.real].double()

    def padding_is_zero(self, t):
        x = self.flat(t)
        return bool((x[self.tokens < 0] == 0).all())


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g
