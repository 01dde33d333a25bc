"""Refusals of the attention calls that need no GPU, and the reference forms'
own checks."""
import numpy as np
import pytest
import torch

import attention_ref as ref


def _plan(cpt, T=16, P=2, pad=None):
    return cpt.Plan(0, None, 0, P, 1, T, pad or T)


def test_binding_refuses_before_the_library(cpt):
    plan = _plan(cpt)
    bf = torch.bfloat16
    q, k = torch.zeros(16, 4, 8, dtype=bf), torch.zeros(16, 2, 8, dtype=bf)
    lse = torch.zeros(4, 16)
    ok = dict(q=q, k=k, v=k.clone(), out=q.clone(), lse=lse, scale=1.0, window=4, sinks=0)
    bad = [
        dict(q=q[:15]), dict(k=k[:15]), dict(out=q[:15].clone()), dict(lse=lse[:, :15].contiguous()),
        dict(lse=lse.double()), dict(v=torch.zeros(16, 4, 8, dtype=bf)), dict(out=torch.zeros(16, 2, 8, dtype=bf)),
        dict(k=torch.zeros(16, 2, 16, dtype=bf)), dict(v=torch.zeros(16, 2, 8)), dict(q=torch.zeros(8, dtype=bf)),
        dict(q=torch.zeros(16, 8, 8, dtype=bf)[:, ::2]),
    ]
    for kw in bad:
        with pytest.raises(ValueError):
            cpt.cpt_attention(plan, **{**ok, **kw}, stream=0)
    with pytest.raises(cpt.CptError) as e:
        cpt.cpt_attention(plan, **ok, stream=0)
    assert e.value.status == cpt.CPT_ERR_INVALID_ARG  # a plan without a handle
    ws = torch.zeros(1024, dtype=torch.uint8)
    w = [torch.zeros(16, 2, 8, dtype=bf) for _ in range(2)]
    back = dict(q=q, k=k, v=k.clone(), out=q.clone(), lse=lse, dout=q.clone(), dq=q.clone(), dk_writers=w,
                dv_writers=[x.clone() for x in w], scale=1.0, window=4, sinks=0, workspace=ws)
    bad = [
        dict(dq=q[:15].clone()), dict(dout=torch.zeros(16, 4, 8)), dict(dk_writers=w[:1]),
        dict(dk_writers=[torch.zeros(15, 2, 8, dtype=bf)] * 2), dict(dv_writers=[torch.zeros(16, 2, 8)] * 2),
        dict(dv_writers=[torch.zeros(16, 4, 8, dtype=bf)] * 2), dict(workspace=None),
    ]
    for kw in bad:
        with pytest.raises(ValueError):
            cpt.cpt_attention_backward(plan, **{**back, **kw}, stream=0)
    with pytest.raises(cpt.CptError) as e:
        cpt.cpt_attention_backward(plan, **back, stream=0)
    assert e.value.status == cpt.CPT_ERR_INVALID_ARG


def test_workspace_of_no_plan_is_zero(cpt):
    assert cpt.cpt_attention_backward_workspace_bytes(_plan(cpt), 4, 2, 64) == 0


@pytest.mark.parametrize("layout,P,lens", [(0, 2, [16, 24, 24]), (1, 2, [13, 0, 51]), (3, 4, [3, 17, 0, 1])])
def test_reference_maps_agree_with_the_oracle(oracle_lib, layout, P, lens):
    l2r, l2g, cu, cup = ref.local_rows(layout, P, lens)
    want, _ = oracle_lib.index_map(0 if layout == 3 else layout, P, cup.astype(np.int32), int(cup[-1]))
    assert np.array_equal(l2g, want)
    doc = np.searchsorted(cup, l2g, side="right") - 1
    u = l2g - cup[doc]
    assert np.array_equal(l2r, np.where(u < np.diff(cu)[doc], cu[doc] + u, -1))


def test_reference_gradient_is_autograd():
    """The 64-bit backward form against torch's autograd."""
    P, lens, W, S, G = 2, [24, 8, 40], 9, 2, 2
    l2r, l2g, cu, cup = ref.local_rows(0, P, lens)
    T = int(cu[-1])
    g = torch.Generator().manual_seed(0)
    q, do = (torch.randn(T, 4, 8, generator=g, dtype=torch.float64) for _ in range(2))
    k, v = (torch.randn(T, 2, 8, generator=g, dtype=torch.float64) for _ in range(2))
    see = ref.visible(l2r, cu, T, W, S, "cpu")
    x = [t.clone().requires_grad_() for t in (q, k, v)]
    s = torch.einsum("ihd,jhd->hij", x[0], x[1].repeat_interleave(G, 1)) * 0.3
    p = torch.softmax(s.masked_fill(~see, -float("inf")), -1)
    out = torch.einsum("hij,jhd->ihd", p, x[2].repeat_interleave(G, 1))
    (out * do).sum().backward()
    o, lse, _ = ref.attention64(q, k, v, see, 0.3)
    assert torch.allclose(o, out.detach(), atol=1e-12)
    dq, _, writers = ref.backward64(q, k, v, o, do, see, 0.3, P)
    assert torch.allclose(dq, x[0].grad, atol=1e-12)
    assert torch.allclose(writers[0][0][0] + writers[1][0][0], x[1].grad, atol=1e-12)
    assert torch.allclose(writers[0][1][0] + writers[1][1][0], x[2].grad, atol=1e-12)
