"""Refusals of the rotary calls that need no GPU."""
import pytest
import torch


def test_create_refuses(cpt):
    ok = dict(head_dim=8, inv_freq=[1.0, 0.5], axis_of_pair=[0, 1], n_axes=2)
    cpt.cpt_rotary_destroy(cpt.cpt_rotary_create(**ok))

    def status(**kw):
        with pytest.raises(cpt.CptError) as e:
            cpt.cpt_rotary_create(**{**ok, **kw})
        return e.value.status

    assert status(head_dim=7) == cpt.CPT_ERR_UNSUPPORTED
    assert status(head_dim=0) == cpt.CPT_ERR_UNSUPPORTED
    assert status(head_dim=258) == cpt.CPT_ERR_UNSUPPORTED
    assert status(head_dim=2) == cpt.CPT_ERR_INVALID_ARG              # two pairs in two elements
    assert status(inv_freq=[], axis_of_pair=[]) == cpt.CPT_ERR_INVALID_ARG
    assert status(n_axes=0) == cpt.CPT_ERR_INVALID_ARG
    assert status(n_axes=9) == cpt.CPT_ERR_INVALID_ARG
    assert status(n_axes=1) == cpt.CPT_ERR_INVALID_ARG                # axis 1 of one
    assert status(axis_of_pair=[0, -1]) == cpt.CPT_ERR_INVALID_ARG
    assert status(inv_freq=[1.0, float("nan")]) == cpt.CPT_ERR_INVALID_ARG
    assert status(inv_freq=[1.0, float("inf")]) == cpt.CPT_ERR_INVALID_ARG
    assert status(inv_freq=[1.0, 2.0 ** 21]) == cpt.CPT_ERR_INVALID_ARG
    assert status(pairing=2) == cpt.CPT_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        cpt.cpt_rotary_create(8, [1.0], [0, 1], 2)


def _plan(cpt, T=16, P=2, pad=None):
    """A Plan object without a device: the binding's checks run before the library."""
    return cpt.Plan(0, None, 0, P, 1, T, pad or T)


def test_binding_refuses_before_the_library(cpt):
    rot = cpt.cpt_rotary_create(8, [1.0] * 4, [0] * 4, 1)
    plan = _plan(cpt)
    x = torch.zeros(16, 2, 8)
    pos = torch.zeros(1, 16, dtype=torch.int32)
    bad = [
        dict(srcs=[], dsts=[]),
        dict(srcs=[x], dsts=[]),
        dict(srcs=[x], dsts=[x.to(torch.bfloat16)]),
        dict(srcs=[x], dsts=[torch.zeros(16, 4, 8)]),
        dict(srcs=[torch.zeros(16, 2, 16)], dsts=[x]),
        dict(srcs=[torch.zeros(15, 2, 8)], dsts=[x]),
        dict(srcs=[x], dsts=[torch.zeros(15, 2, 8)]),
        dict(srcs=[x], dsts=[x], positions=pos[:, :15].contiguous()),
        dict(srcs=[x], dsts=[x], positions=pos.long()),
        dict(srcs=[x], dsts=[x], src_order=2),
    ]
    for kw in bad:
        with pytest.raises(ValueError):
            cpt.cpt_rotary_apply(rot, plan, **{"positions": pos, **kw}, stream=0)
    with pytest.raises(cpt.CptError) as e:  # a plan without a handle
        cpt.cpt_rotary_apply(rot, plan, [x], [x.clone()], pos, stream=0)
    assert e.value.status == cpt.CPT_ERR_INVALID_ARG
