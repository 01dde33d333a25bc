"""The bounded waits of the residual norms' rings, made to run out on purpose.

A test switch makes every copy's barrier expect 16 bytes more than the copies deliver. The copies still complete and nothing
faults, but no wait can finish: each gives up after about a second. The calls have to count that, store nothing
of a row that they could not wait for, and return; with the switch off, the same calls give the same bits as before.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

T, P = 8192, 2   # several rows for every team
MARK = 7.0


def tensors(dtype, C, gate, seed=5):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*shape, dtype=dtype):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)

    t = {"h": rand(T, C), "x": rand(T, C), "dy": rand(T, C), "dn": rand(T, C)}
    t["post_weight"], t["pre_weight"] = rand(C, dtype=torch.float32), rand(C, dtype=torch.float32)
    t["gate"] = {"none": None, "token": rand(T, C), "document": rand(2, C)}[gate]
    return t


def marked(n, C, dtype):
    return torch.full((n, C), MARK, dtype=dtype, device="cuda")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("post, pre, gate", [(True, True, "none"), (False, True, "none"), (True, False, "token"),
                                             (False, False, "document"), (True, True, "document")])
def test_rings_that_run_out(cpt, cuda_device, dtype, post, pre, gate):
    C = 1040   # long rows, the last thread's share not whole
    plan = cpt.cpt_plan_create(0, P, [0, 24, T], T)
    t = tensors(dtype, C, gate)
    block = {"gate": t["gate"], "gate_per_document": gate == "document"}
    if post:
        block["post_weight"] = t["post_weight"]
    if pre:
        block["pre_weight"] = t["pre_weight"]

    def forward():
        y, n = marked(T, C, dtype), marked(T, C, dtype) if pre else None
        cpt.cpt_residual_norm(plan, t["x"], t["h"], y, n, **block)
        torch.cuda.synchronize()
        return [v for v in (y, n) if v is not None]

    y = forward()[0]

    def backward():
        dx, dh = marked(T, C, dtype), marked(T, C, dtype)
        sums, rows = {}, [dx, dh]
        if post:
            sums["dpost_weight"] = torch.zeros(C, device="cuda")
        if pre:
            sums["dpre_weight"] = torch.zeros(C, device="cuda")
        if gate == "token":
            sums["dgate"] = marked(T, C, dtype)
            rows.append(sums["dgate"])
        elif gate == "document":
            sums["dgate"] = torch.zeros(2, C, device="cuda")
        cpt.cpt_residual_norm_backward(plan, t["h"], y if pre else None, t["dy"], t["dn"] if pre else None, dx, dh, **sums, **block)
        torch.cuda.synchronize()
        return rows, list(sums.values())

    cpt.cpt_kernel_wait_timeouts(reset=True)
    want, (want_rows, want_sums) = forward(), backward()
    assert cpt.cpt_kernel_wait_timeouts() == 0
    for call in (forward, lambda: backward()[0]):
        cpt.cpt_test_stall_bulk_waits(True)
        try:
            got = call()
        finally:
            cpt.cpt_test_stall_bulk_waits(False)
        assert cpt.cpt_kernel_wait_timeouts(reset=True) >= 1
        for v in got:
            assert torch.equal(v, torch.full_like(v, MARK))
    got, (got_rows, got_sums) = forward(), backward()
    assert cpt.cpt_kernel_wait_timeouts() == 0
    for a, b in zip(want + want_rows + want_sums, got + got_rows + got_sums):
        assert torch.equal(a, b) and not torch.equal(a, torch.full_like(a, MARK))
