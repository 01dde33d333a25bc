"""Refusals of the attention layer's calls that need device memory or a plan,
through the C entries: nothing is launched, every output stays as it was."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32 = 1, 0


def _array(*tensors):
    return (ctypes.c_void_p * len(tensors))(*[None if t is None else t.data_ptr() for t in tensors])


class Rotary:
    """A call of cpt_rotary_apply that succeeds, one argument of which a test replaces."""

    def __init__(self, cpt, T=32, heads=2, D=8):
        self.cpt, self.T = cpt, T
        self.plan = cpt.cpt_plan_create(0, 2, [0, T], T)
        self.rot = cpt.cpt_rotary_create(D, [1.0] * (D // 2), [0] * (D // 2), 1)
        self.x = torch.randn(T, heads, D, device="cuda")
        self.y = torch.full_like(self.x, 7.0)
        self.pos = torch.zeros(1, T, dtype=torch.int32, device="cuda")
        self.args = dict(rotary=self.rot.handle, plan=self.plan.handle, n=1, src=_array(self.x), dst=_array(self.y),
                         heads=(ctypes.c_int32 * 4)(heads, 1, 1, 1), dtype=F32, positions=self.pos.data_ptr(),
                         src_order=0, dst_order=1, inverse=0, stream=torch.cuda.current_stream().cuda_stream)

    def status(self, **kw):
        assert set(kw) <= set(self.args)
        st = self.cpt._lib.cpt_rotary_apply(*{**self.args, **kw}.values())
        torch.cuda.synchronize()
        return st


def test_rotary_apply_refuses(cpt, cuda_device):
    r = Rotary(cpt)
    x, y, pos = r.x, r.y, r.pos
    one = (ctypes.c_int32 * 4)
    bad = [
        (dict(rotary=None), cpt.CPT_ERR_INVALID_ARG),
        (dict(plan=None), cpt.CPT_ERR_INVALID_ARG),
        (dict(n=0), cpt.CPT_ERR_INVALID_ARG),
        (dict(n=4), cpt.CPT_ERR_INVALID_ARG),
        (dict(src=None), cpt.CPT_ERR_INVALID_ARG),
        (dict(dst=None), cpt.CPT_ERR_INVALID_ARG),
        (dict(heads=None), cpt.CPT_ERR_INVALID_ARG),
        (dict(src=_array(None)), cpt.CPT_ERR_INVALID_ARG),
        (dict(dst=_array(None)), cpt.CPT_ERR_INVALID_ARG),
        (dict(positions=None), cpt.CPT_ERR_INVALID_ARG),
        (dict(heads=one(0, 1, 1, 1)), cpt.CPT_ERR_INVALID_ARG),
        (dict(heads=one(-3, 1, 1, 1)), cpt.CPT_ERR_INVALID_ARG),
        (dict(heads=one(1 << 26, 1, 1, 1)), cpt.CPT_ERR_INVALID_ARG),
        (dict(dtype=2), cpt.CPT_ERR_INVALID_ARG),
        (dict(dtype=-1), cpt.CPT_ERR_INVALID_ARG),
        (dict(src_order=2), cpt.CPT_ERR_INVALID_ARG),
        (dict(dst_order=-1), cpt.CPT_ERR_INVALID_ARG),
        (dict(src=_array(x.cpu())), cpt.CPT_ERR_DEVICE),
        (dict(dst=_array(x.cpu())), cpt.CPT_ERR_DEVICE),
        (dict(positions=pos.cpu().data_ptr()), cpt.CPT_ERR_DEVICE),
        (dict(src=_array(x.view(-1)[1:])), cpt.CPT_ERR_ALIGNMENT),
        (dict(dst=_array(y.view(-1)[2:])), cpt.CPT_ERR_ALIGNMENT),
        (dict(positions=pos.data_ptr() + 2), cpt.CPT_ERR_ALIGNMENT),
        (dict(dst=_array(x)), cpt.CPT_ERR_ALIAS),                                          # in place
        (dict(dst=_array(x), src_order=1, dst_order=1), cpt.CPT_ERR_ALIAS),
        (dict(src=_array(y.view(-1)[256:]), dst=_array(y)), cpt.CPT_ERR_ALIAS),            # part of it
        (dict(n=2, src=_array(x, x), dst=_array(y, y)), cpt.CPT_ERR_ALIAS),                # twice the same
        (dict(dst=_array(pos)), cpt.CPT_ERR_ALIAS),
    ]
    for kw, want in bad:
        assert r.status(**kw) == want, kw
        assert (y == 7.0).all()
    assert r.status(src=_array(x)) == 0 and not (y == 7.0).any()


@pytest.mark.parametrize("D,heads,dtype", [(6, 1, F32), (2, 1, F32), (4, 1, BF16), (10, 3, BF16)])
def test_rotary_rows_of_no_whole_16_bytes(cpt, cuda_device, D, heads, dtype):
    r = Rotary(cpt)
    rot = cpt.cpt_rotary_create(D, [1.0] * (D // 2), [0] * (D // 2), 1)
    assert r.status(rotary=rot.handle, heads=(ctypes.c_int32 * 1)(heads), dtype=dtype) == cpt.CPT_ERR_ALIGNMENT
    assert (r.y == 7.0).all()


def test_attention_refuses(cpt, cuda_device):
    T, Hq, Hk, D = 32, 4, 2, 64
    plan = cpt.cpt_plan_create(0, 2, [0, T], T)
    bf = dict(device="cuda", dtype=torch.bfloat16)
    q, k, v = torch.randn(T, Hq, D, **bf), torch.randn(T, Hk, D, **bf), torch.randn(T, Hk, D, **bf)
    out, lse = torch.full((T, Hq, D), 7.0, **bf), torch.full((Hq, T), 7.0, device="cuda")
    dout, dq = torch.randn(T, Hq, D, **bf), torch.full((T, Hq, D), 7.0, **bf)
    dk, dv = ([torch.full((T, Hk, D), 7.0, **bf) for _ in range(2)] for _ in range(2))
    stream = torch.cuda.current_stream().cuda_stream
    need = cpt.cpt_attention_backward_workspace_bytes(plan, Hq, Hk, D)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    ptr = lambda t: t.data_ptr()  # noqa: E731
    shape = dict(q_heads=Hq, kv_heads=Hk, head_dim=D, dtype=BF16, scale=0.1, window=8, sinks=1)
    fwd = dict(plan=plan.handle, q=ptr(q), k=ptr(k), v=ptr(v), out=ptr(out), lse=ptr(lse), **shape, stream=stream)
    back = dict(plan=plan.handle, q=ptr(q), k=ptr(k), v=ptr(v), out=ptr(out), lse=ptr(lse), dout=ptr(dout), dq=ptr(dq),
                dkw=_array(*dk), dvw=_array(*dv), **shape, ws=ptr(ws), ws_bytes=need, stream=stream)
    A, U, L = cpt.CPT_ERR_INVALID_ARG, cpt.CPT_ERR_UNSUPPORTED, cpt.CPT_ERR_ALIGNMENT
    both = [
        (dict(plan=None), A), (dict(q=None), A), (dict(k=None), A), (dict(v=None), A), (dict(out=None), A),
        (dict(lse=None), A), (dict(q_heads=0), A), (dict(kv_heads=0), A), (dict(kv_heads=3), A), (dict(q_heads=-4), A),
        (dict(q_heads=1026), U), (dict(head_dim=0), U), (dict(head_dim=12), U), (dict(head_dim=136), U),
        (dict(dtype=F32), U), (dict(dtype=7), A), (dict(scale=0.0), A), (dict(scale=float("inf")), A),
        (dict(scale=float("nan")), A), (dict(window=-1), A), (dict(sinks=-1), A),
        (dict(q=ptr(q) + 8), L), (dict(k=ptr(k) + 2), L), (dict(out=ptr(out) + 8), L), (dict(lse=ptr(lse) + 4), L),
        (dict(v=torch.zeros(T, Hk, D, dtype=torch.bfloat16).data_ptr()), cpt.CPT_ERR_DEVICE),
    ]
    X = cpt.CPT_ERR_ALIAS
    for kw, want in both + [(dict(out=ptr(q)), X), (dict(out=ptr(k)), X), (dict(lse=ptr(out)), X), (dict(lse=ptr(v)), X)]:
        assert cpt._lib.cpt_attention(*{**fwd, **kw}.values()) == want, kw
    W = cpt.CPT_ERR_WORKSPACE
    more = [
        (dict(dout=None), A), (dict(dq=None), A), (dict(dkw=None), A), (dict(dvw=None), A), (dict(dkw=_array(dk[0], None)), A),
        (dict(dq=ptr(dout)), X), (dict(dq=ptr(lse)), X), (dict(dkw=_array(dk[0], dk[0])), X), (dict(dvw=_array(*dk)), X),
        (dict(dkw=_array(dk[0], q)), X), (dict(ws=None), W), (dict(ws_bytes=need - 1), W), (dict(ws=ptr(ws) + 16), W),
        (dict(dq=ptr(ws)), X),
    ]
    for kw, want in both + more:
        assert cpt._lib.cpt_attention_backward(*{**back, **kw}.values()) == want, kw
    torch.cuda.synchronize()
    assert all((x == 7.0).all() for x in [out, lse, dq] + dk + dv)
    assert cpt._lib.cpt_attention(*fwd.values()) == 0
    assert cpt._lib.cpt_attention_backward(*back.values()) == 0
    torch.cuda.synchronize()
    assert not any((x == 7.0).all() for x in [out, lse, dq] + dk + dv)
