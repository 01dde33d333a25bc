"""The binding compares the shapes of gates, weights, logits and per-row buffers with the documented ones: what only holds
enough elements would be read as other rows. (A call that these checks let through ends at the library's first one: there is no plan.)"""
import pytest
import torch


def _plan(cpt, T=16, P=2, n=3):
    return cpt.Plan(0, None, 0, P, n, T, T)


def refused(call):
    with pytest.raises(ValueError):
        call()


def accepted(cpt, call):
    with pytest.raises(cpt.CptError) as e:
        call()
    assert e.value.status == cpt.CPT_ERR_INVALID_ARG


ROW, DOC = (2, 8, 16), (3, 16)


@pytest.mark.parametrize("shape,per_document,good", [
    (ROW, False, True), ((16, 16), False, True), ((256,), False, True), ((2, 8, 4, 4), False, True),
    ((2, 8, 32), False, False), ((2, 16, 16), False, False), ((32, 16), False, False), ((4, 8, 16), False, False), ((512,), False, False),
    ((16, 32), False, False), (DOC, False, False), ((8, 32), False, False),
    (DOC, True, True), ((48,), True, True), ((3, 4, 4), True, True), ((3, 1, 16), True, True),
    ((16, 16), True, False), (ROW, True, False), ((4, 16), True, False), ((3, 32), True, False), ((16, 3), True, False),
    ((2, 16), True, False), ((96,), True, False), ((), True, False),
])
def test_gates(cpt, shape, per_document, good):
    plan, x, g = _plan(cpt), torch.zeros(ROW), torch.zeros(shape)
    right = torch.zeros(DOC if per_document else ROW)
    calls = [
        lambda: cpt.cpt_residual_norm(plan, x, x, x, None, gate=g, gate_per_document=per_document, stream=0),
        lambda: cpt.cpt_residual_norm_backward(plan, x, None, x, None, x, x, gate=g, gate_per_document=per_document, dgate=right,
                                               workspace=x, stream=0),
        lambda: cpt.cpt_residual_norm_backward(plan, x, None, x, None, x, x, gate=right, gate_per_document=per_document, dgate=g,
                                               workspace=x, stream=0),
    ]
    for call in calls:
        accepted(cpt, call) if good else refused(call)


@pytest.mark.parametrize("shape,good", [((16,), True), ((4, 4), True), ((17,), False), ((2, 16), False), ((15,), False)])
def test_weights(cpt, shape, good):
    plan, x, w, right = _plan(cpt), torch.zeros(ROW), torch.ones(shape), torch.ones(16)
    calls = [
        lambda: cpt.cpt_residual_norm(plan, x, x, x, None, post_weight=w, stream=0),
        lambda: cpt.cpt_residual_norm(plan, x, x, x, x, pre_weight=w, stream=0),
        lambda: cpt.cpt_residual_norm_backward(plan, x, x, x, x, x, x, post_weight=right, pre_weight=right, dpost_weight=w,
                                               dpre_weight=right, workspace=x, stream=0),
        lambda: cpt.cpt_residual_norm_backward(plan, x, x, x, x, x, x, post_weight=right, pre_weight=right, dpost_weight=right,
                                               dpre_weight=w, workspace=x, stream=0),
    ]
    for call in calls:
        accepted(cpt, call) if good else refused(call)


@pytest.mark.parametrize("shape,good", [
    (ROW, True), ((16, 16), True), ((20, 16), True), ((4, 4, 16), True), ((1, 16, 16), True),
    ((2, 8, 2, 16), False), ((2, 8, 2, 8), False), ((2, 9, 16), False), ((3, 8, 16), False), ((15, 16), False), ((256,), False), ((), False),
])
def test_logits(cpt, shape, good):
    plan, x = _plan(cpt), torch.zeros(shape)
    t, f, two = torch.zeros(16, dtype=torch.int32), torch.zeros(16), torch.zeros(16, 2)
    calls = [lambda: cpt.cpt_token_logprob(plan, x, t, f, two, stream=0),
             lambda: cpt.cpt_token_logprob_backward(plan, x, t, two, f, x, stream=0),
             lambda: cpt.cpt_token_logprob_backward(plan, torch.zeros(ROW), t, two, f, x, stream=0)]
    for call in calls:
        accepted(cpt, call) if good else refused(call)


def test_values_of_a_row(cpt):
    plan, x, t, f = _plan(cpt), torch.zeros(ROW), torch.zeros(16, dtype=torch.int32), torch.zeros(16)
    three, terms = torch.zeros(3), torch.zeros(3, 4)
    for shape, good in (((16, 2), True), ((32,), True), ((20, 2), True), ((2, 16), False), ((16, 4), False)):
        s = torch.zeros(shape)
        for call in (lambda: cpt.cpt_token_logprob(plan, x, t, f, s, stream=0),
                     lambda: cpt.cpt_token_logprob_backward(plan, x, t, s, f, x, stream=0)):
            accepted(cpt, call) if good else refused(call)
    for shape, good in (((3, 4), True), ((12,), True), ((5, 4), True), ((4, 3), False), ((2, 6), False), ((3, 8), False)):
        call = lambda: cpt.cpt_policy_loss(plan, f, f, three, torch.zeros(shape), f, stream=0)  # noqa: B023, E731
        accepted(cpt, call) if good else refused(call)
    accepted(cpt, lambda: cpt.cpt_policy_loss(plan, f, f, three, terms, f, stream=0))
