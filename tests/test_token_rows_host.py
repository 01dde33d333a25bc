"""The generator's reference against published vectors, and refusals of the calls on token rows that need no GPU."""
import ctypes

import numpy as np
import pytest
import torch

from token_rows_ref import kept, philox


@pytest.mark.parametrize("key,ctr,want", [
    # the vectors that the generator's authors publish for ten rounds
    ((0, 0), (0, 0, 0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
    ((0xffffffff,) * 2, (0xffffffff,) * 4, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
    ((0xa4093822, 0x299f31d0), (0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344),
     (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1)),
])
def test_generator_reference(key, ctr, want):
    got = philox(key, [np.array([c]) for c in ctr])
    assert tuple(int(g[0]) for g in got) == want


def test_kept_share():
    assert kept(0.0) == 65536 and kept(1.0) == 0 and kept(0.5) == 32768 and kept(0.1) == 58982


def _plan(cpt, T=16, P=2, n=1):
    """A Plan object without a device: the binding's checks run before the library."""
    return cpt.Plan(0, None, 0, P, n, T, T)


def test_binding_refuses_rows(cpt):
    plan, x = _plan(cpt), torch.zeros(2, 8, 16)
    G = cpt.CPT_ORDER_GLOBAL
    bad = [
        lambda: cpt.cpt_dropout(plan, x, x.bfloat16(), 0.1, stream=0),
        lambda: cpt.cpt_dropout(plan, x, torch.zeros(2, 8, 8), 0.1, stream=0),
        lambda: cpt.cpt_dropout(plan, x, torch.zeros(2, 7, 16), 0.1, stream=0),
        lambda: cpt.cpt_dropout(plan, x, x, 0.1, order=G, stream=0),                 # 2 rows of 16 wanted
        lambda: cpt.cpt_dropout(plan, x, x, 0.1, order=2, stream=0),
        lambda: cpt.cpt_dropout(plan, x, x, 0.1, rng=torch.zeros(2, dtype=torch.int32), stream=0),
        lambda: cpt.cpt_dropout(plan, x, x, 0.1, rng=torch.zeros(1, dtype=torch.int64), stream=0),
        lambda: cpt.cpt_dropout(plan, x.transpose(0, 1).reshape(2, 8, 16).transpose(1, 2), x, 0.1, stream=0),
        lambda: cpt.cpt_residual_norm(plan, x, x.bfloat16(), x, None, stream=0),
        lambda: cpt.cpt_residual_norm(plan, x, x, x, x, pre_weight=torch.ones(15), stream=0),
        lambda: cpt.cpt_residual_norm(plan, x, x, x, x, pre_weight=torch.ones(16).double(), stream=0),
        lambda: cpt.cpt_residual_norm(plan, x, x, x, None, gate=torch.zeros(2, 7, 16), stream=0),
        lambda: cpt.cpt_residual_norm(plan, x, x, x, None, gate=x.bfloat16(), stream=0),
        lambda: cpt.cpt_residual_norm(plan, x, x, x, None, gate=torch.zeros(0, 16), gate_per_document=True, stream=0),
        lambda: cpt.cpt_residual_norm_backward(plan, x, None, x, None, x, x, gate=x, dgate=torch.zeros(1), stream=0),
        lambda: cpt.cpt_residual_norm_backward(plan, x, None, x, None, x, x, gate=torch.zeros(1, 16),
                                               gate_per_document=True, dgate=torch.zeros(1, 16).bfloat16(), stream=0),
        lambda: cpt.cpt_residual_norm_backward(plan, x, None, x, None, x, x, post_weight=torch.ones(16),
                                               dpost_weight=torch.ones(8), stream=0),
        lambda: cpt.cpt_residual_norm_backward(plan, None, None, x, None, x, x, stream=0),   # no workspace
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            raise AssertionError(i)


def test_binding_refuses_losses(cpt):
    plan, x, t = _plan(cpt), torch.zeros(2, 8, 16), torch.zeros(16, dtype=torch.int32)
    f, two = torch.zeros(16), torch.zeros(16, 2)
    one, four = torch.zeros(1), torch.zeros(1, 4)
    bad = [
        lambda: cpt.cpt_token_logprob(plan, x[:1], t, f, two, stream=0),
        lambda: cpt.cpt_token_logprob(plan, x, t.long(), f, two, stream=0),
        lambda: cpt.cpt_token_logprob(plan, x, t[:15], f, two, stream=0),
        lambda: cpt.cpt_token_logprob(plan, x, t, f[:15], two, stream=0),
        lambda: cpt.cpt_token_logprob(plan, x, t, f, f, stream=0),
        lambda: cpt.cpt_token_logprob(plan, x, t, f.bfloat16(), two, stream=0),
        lambda: cpt.cpt_token_logprob(plan, x, t, f, two, order=5, stream=0),
        lambda: cpt.cpt_token_logprob(plan, x, t, f, two, vocab=17, stream=0),
        lambda: cpt.cpt_token_logprob(plan, x, t, f, two, vocab=0, stream=0),
        lambda: cpt.cpt_token_logprob(plan, x, t, f, two, vocab=2 ** 64 + 5, stream=0),
        lambda: cpt.cpt_token_logprob_backward(plan, x, t, two, f, x, vocab=5 - 2 ** 64, stream=0),
        lambda: cpt.cpt_token_logprob_backward(plan, x, t, two, f, x.bfloat16(), stream=0),
        lambda: cpt.cpt_token_logprob_backward(plan, x, t, two, f, x[:1], stream=0),
        lambda: cpt.cpt_policy_loss(plan, f[:15], f, one, four, f, stream=0),
        lambda: cpt.cpt_policy_loss(plan, f, f.double(), one, four, f, stream=0),
        lambda: cpt.cpt_policy_loss(plan, f, f, torch.zeros(0), four, f, stream=0),
        lambda: cpt.cpt_policy_loss(plan, f, f, one, four[:, :3].contiguous(), f, stream=0),
        lambda: cpt.cpt_policy_loss(plan, f, f, one, four, f, mask=f, stream=0),
        lambda: cpt.cpt_policy_loss(plan, f, f, one, four, f, mask=torch.zeros(15, dtype=torch.bool), stream=0),
        lambda: cpt.cpt_policy_loss(plan, f, f, one, four, f, weights=torch.zeros(0), stream=0),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            raise AssertionError(i)


def test_calls_without_a_plan(cpt):
    x, t, f, two = torch.zeros(2, 8, 16), torch.zeros(16, dtype=torch.int32), torch.zeros(16), torch.zeros(16, 2)
    plan = _plan(cpt)
    calls = [
        lambda: cpt.cpt_dropout(plan, x, x, 0.0, stream=0),
        lambda: cpt.cpt_residual_norm(plan, x, x, x, None, stream=0),
        lambda: cpt.cpt_residual_norm_backward(plan, None, None, x, None, x, x, workspace=f, stream=0),
        lambda: cpt.cpt_token_logprob(plan, x, t, f, two, stream=0),
        lambda: cpt.cpt_token_logprob_backward(plan, x, t, two, f, x, stream=0),
        lambda: cpt.cpt_policy_loss(plan, f, f, f, torch.zeros(1, 4), f, stream=0),
    ]
    for call in calls:
        with pytest.raises(cpt.CptError) as e:
            call()
        assert e.value.status == cpt.CPT_ERR_INVALID_ARG
    assert cpt.cpt_residual_norm_backward_workspace_bytes(plan, 16, torch.float32) == 0


def test_options_have_the_headers_layout(cpt):
    # three pointers, an enumerator, two floats (one of padding), a double, a pointer, 32 bits (and padding)
    f = cpt._Residual
    assert [getattr(f, n).offset for n, _ in f._fields_] == [0, 8, 16, 24, 28, 32, 40, 48, 56]
    assert ctypes.sizeof(f) == 64
