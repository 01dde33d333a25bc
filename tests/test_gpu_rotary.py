"""Rotary positions with several axes on the GPU, against 64-bit rotations.

Tolerance: the angle is held to 2^-31 of a turn (3e-9 rad) and the sine and
cosine to a few 2^-24; a product and a sum in binary32 add 2^-23 of |x| + |y|.
4 * 2^-22 * (|x| + |y|) covers these; a bf16 output adds half a step, 2^-8 of
its value."""
import numpy as np
import pytest
import torch

import attention_ref as ref
from gpu_helpers import Guarded

pytestmark = pytest.mark.gpu

LENS = {0: [48, 0, 16, 96, 160], 1: [47, 0, 1, 130, 66, 76], 3: [47, 0, 1, 130, 66, 77, 5]}
ORDERS = [(0, 1), (1, 0), (1, 1), (0, 0)]


def _run(cpt, layout, P, lens, heads, D, n, axes, dtype, interleaved, inverse, orders, pos=None, seed=0):
    rng = np.random.default_rng(seed)
    l2r, _, cu, _ = ref.local_rows(layout, P, lens)
    T, Tpad = int(cu[-1]), len(l2r)
    plan = cpt.cpt_plan_create(layout, P, cu.tolist(), T)
    freq = [10000.0 ** (-i / n) for i in range(n)]
    axis = [int(a) for a in rng.integers(0, axes, n)]
    rot = cpt.cpt_rotary_create(D, freq, axis, axes, int(interleaved))
    if pos is None:
        pos = rng.integers(-(1 << 31), 1 << 31, size=(axes, T), dtype=np.int64).astype(np.int32)
    rows = (T, Tpad)
    src, dst = [], []
    for h in heads:
        x = torch.from_numpy(rng.standard_normal((rows[orders[0]], h, D)).astype(np.float32)).to(dtype)
        src.append(x.cuda())
        dst.append(Guarded((rows[orders[1]], h, D), dtype))
    cpt.cpt_rotary_apply(rot, plan, src, [d.t for d in dst], torch.from_numpy(pos).cuda(), *orders, inverse)
    torch.cuda.synchronize()
    for x, d in zip(src, dst):
        assert d.bands_intact()
        x = x.double().cpu().numpy()
        if orders[0] == 1:
            y = np.zeros((T,) + x.shape[1:])
            y[l2r[l2r >= 0]] = x[l2r >= 0]
            x = y
        want = ref.rotate64(x, pos, freq, axis, interleaved, inverse)
        tol = 4 * 2.0 ** -22 * (np.abs(x) + np.abs(np.roll(x, n, -1)) + np.abs(np.roll(x, -n, -1))
                                + np.abs(np.roll(x, 1, -1)) + np.abs(np.roll(x, -1, -1)))
        if dtype == torch.bfloat16:
            tol = tol + np.abs(want) * 2.0 ** -8
        if orders[1] == 1:
            full = np.zeros((Tpad,) + x.shape[1:])
            t2 = np.zeros_like(full)
            full[l2r >= 0], t2[l2r >= 0] = want[l2r[l2r >= 0]], tol[l2r[l2r >= 0]]
            want, tol = full, t2
        got = d.t.double().cpu().numpy()
        assert np.all(np.abs(got - want) <= tol), float(np.max(np.abs(got - want) - tol))
        # what is not rotated is copied, bit for bit
        assert np.array_equal(got[..., 2 * n:], want[..., 2 * n:])


@pytest.mark.parametrize("orders", ORDERS)
@pytest.mark.parametrize("layout", [0, 1, 3])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_orders_and_layouts(cpt, cuda_device, layout, orders, dtype):
    _run(cpt, layout, 4, LENS[layout] if layout else [48, 0, 16, 96, 160], [4, 2], 64, 32, 3, dtype, False, False,
         orders)
    _run(cpt, layout, 2, LENS[layout], [2], 32, 12, 2, dtype, True, True, orders)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,n,heads", [(2, 1, [8]), (8, 4, [2, 2]), (10, 3, [8]), (72, 18, [6, 2]), (72, 36, [2, 4, 6]),
                                       (80, 40, [3, 1]), (96, 24, [5]), (128, 64, [20, 20, 20]), (256, 128, [3]),
                                       (256, 1, [2])])
def test_head_shapes(cpt, cuda_device, D, n, heads, interleaved):
    for dtype in (torch.float32, torch.bfloat16):
        _run(cpt, 3, 2, [37, 5, 129], heads, D, n, min(n, 3), dtype, interleaved, False, (0, 1), seed=D + n)


@pytest.mark.parametrize("lens,P", [([1], 1), ([2, 0, 0], 2), ([0, 3], 3)])
def test_shortest_batches(cpt, cuda_device, lens, P):
    _run(cpt, 3, P, lens, [2], 8, 4, 1, torch.float32, False, False, (0, 1))
    _run(cpt, 3, P, lens, [2], 8, 4, 1, torch.float32, False, True, (1, 0))


def test_many_tokens(cpt, cuda_device):
    _run(cpt, 0, 4, [8 * 2500], [3, 1], 64, 32, 3, torch.bfloat16, False, False, (0, 1))


def test_frequencies_beyond_a_turn_and_negative(cpt, cuda_device):
    plan = cpt.cpt_plan_create(1, 1, [0, 5], 5)
    freq = [1048576.0, -3.0, 6.283185307179586, -1e-300]
    rot = cpt.cpt_rotary_create(8, freq, [0] * 4, 1)
    pos = np.array([[0, 1, -7, 12345, 2 ** 20]], dtype=np.int32)
    x = np.random.default_rng(1).standard_normal((5, 1, 8)).astype(np.float32)
    y = torch.empty((5, 1, 8), device="cuda")
    cpt.cpt_rotary_apply(rot, plan, [torch.from_numpy(x).cuda()], [y], torch.from_numpy(pos).cuda(), 0, 0)
    # the 64-bit product itself is off by 2^-53 of an angle of up to 2^40
    want = ref.rotate64(x.astype(np.float64), pos, freq, [0] * 4, False, False)
    assert np.max(np.abs(y.cpu().numpy() - want)) <= 8 * (2.0 ** -20 + 2.0 ** -12)
    first = ref.rotate64(x[:3].astype(np.float64), pos[:, :3], freq, [0] * 4, False, False)
    assert np.max(np.abs(y.cpu().numpy()[:3] - first)) <= 8 * 2.0 ** -20


def test_inverse_is_the_gradient(cpt, cuda_device):
    """<R x, y> = <x, R' y>, and R' R x = x, across the orders."""
    l2r, _, cu, _ = ref.local_rows(3, 4, [33, 100, 7])
    T, Tpad = int(cu[-1]), len(l2r)
    plan = cpt.cpt_plan_create(3, 4, cu.tolist(), T)
    rot = cpt.cpt_rotary_create(16, [1.0, 0.3, 0.1, 0.01, 0.001], [0, 1, 2, 1, 0], 3)
    g = torch.Generator(device="cuda").manual_seed(3)
    pos = torch.randint(0, 1 << 20, (3, T), dtype=torch.int32, device="cuda", generator=g)
    x = torch.randn(T, 2, 16, device="cuda", generator=g)
    y = torch.randn(Tpad, 2, 16, device="cuda", generator=g)
    rx, ry, back = torch.empty_like(y), torch.empty_like(x), torch.empty_like(x)
    cpt.cpt_rotary_apply(rot, plan, [x], [rx], pos, cpt.CPT_ORDER_GLOBAL, cpt.CPT_ORDER_LOCAL)
    cpt.cpt_rotary_apply(rot, plan, [y], [ry], pos, cpt.CPT_ORDER_LOCAL, cpt.CPT_ORDER_GLOBAL, True)
    cpt.cpt_rotary_apply(rot, plan, [rx], [back], pos, cpt.CPT_ORDER_LOCAL, cpt.CPT_ORDER_GLOBAL, True)
    a, b = (rx.double() * y.double()).sum(), (x.double() * ry.double()).sum()
    scale = (rx.double() * y.double()).abs().sum()
    assert abs(a - b) <= 2.0 ** -20 * scale
    assert (back - x).abs().max() <= 16 * 2.0 ** -22 * 5


def test_no_rotation_is_partition_and_restore(cpt, cuda_device):
    """At position zero the call moves bits exactly as the reorder does."""
    l2r, _, cu, _ = ref.local_rows(3, 4, [33, 100, 7])
    T, Tpad = int(cu[-1]), len(l2r)
    plan = cpt.cpt_plan_create(3, 4, cu.tolist(), T)
    rot = cpt.cpt_rotary_create(16, [1.0] * 8, [0] * 8, 1)
    x = torch.randn(T, 2, 16, device="cuda", dtype=torch.bfloat16)
    pos = torch.zeros((1, T), dtype=torch.int32, device="cuda")
    a, b = (torch.empty(Tpad, 2, 16, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    cpt.cpt_rotary_apply(rot, plan, [x], [a], pos)
    cpt.cpt_partition(plan, [x], [b])
    assert torch.equal(a, b)
    y = torch.empty_like(x)
    cpt.cpt_rotary_apply(rot, plan, [a], [y], pos, cpt.CPT_ORDER_LOCAL, cpt.CPT_ORDER_GLOBAL)
    assert torch.equal(x, y)


def test_garbage_in_padding_is_not_read(cpt, cuda_device):
    l2r, _, cu, _ = ref.local_rows(3, 4, [33, 1])
    T, Tpad = int(cu[-1]), len(l2r)
    plan = cpt.cpt_plan_create(3, 4, cu.tolist(), T)
    rot = cpt.cpt_rotary_create(8, [1.0] * 4, [0] * 4, 1)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")[None].contiguous()
    x = torch.full((Tpad, 1, 8), float("nan"), device="cuda")
    x[torch.from_numpy(l2r >= 0).cuda()] = 1.0
    y, z = torch.empty_like(x), torch.empty(T, 1, 8, device="cuda")
    cpt.cpt_rotary_apply(rot, plan, [x], [y], pos, cpt.CPT_ORDER_LOCAL, cpt.CPT_ORDER_LOCAL)
    cpt.cpt_rotary_apply(rot, plan, [x], [z], pos, cpt.CPT_ORDER_LOCAL, cpt.CPT_ORDER_GLOBAL)
    assert torch.isfinite(y).all() and torch.isfinite(z).all()
    assert (y[torch.from_numpy(l2r < 0).cuda()] == 0).all()


def test_streams_and_graphs(cpt, cuda_device):
    T = 640
    plan = cpt.cpt_plan_create(0, 2, [0, T], T)
    rot = cpt.cpt_rotary_create(64, [0.9 ** i for i in range(32)], [i % 3 for i in range(32)], 3)
    pos = torch.randint(0, 1000, (3, T), dtype=torch.int32, device="cuda")
    x = torch.randn(T, 4, 64, device="cuda")
    want, got = torch.empty_like(x), torch.zeros_like(x)
    cpt.cpt_rotary_apply(rot, plan, [x], [want], pos)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    cpt.cpt_rotary_apply(rot, plan, [x], [got], pos, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cpt.cpt_rotary_apply(rot, plan, [x], [got], pos)
    for k in range(2):
        x.mul_(2.0)
        graph.replay()
        cpt.cpt_rotary_apply(rot, plan, [x], [want], pos)
        assert torch.equal(got, want)
