"""Rotary positions at the ends of their ranges."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def _turned(cpt, x, pos, freq, inverse=False):
    T, _, D = x.shape
    plan = cpt.cpt_plan_create(1, 1, [0, T], T)
    rot = cpt.cpt_rotary_create(D, freq, [0] * len(freq), 1)
    y = torch.empty(x.shape, device="cuda")
    cpt.cpt_rotary_apply(rot, plan, [torch.from_numpy(x).cuda()], [y], torch.from_numpy(pos).cuda(),
                         cpt.CPT_ORDER_GLOBAL, cpt.CPT_ORDER_GLOBAL, inverse)
    return y.double().cpu().numpy()


FREQ = [1e-4, 0.3, 0.9, 1e-6, 0.01, 1e-3, 0.1, 0.037]


def _inputs(n):
    rng = np.random.default_rng(7)
    top = np.int64(1) << 31
    pos = np.concatenate([rng.integers(top - (1 << 20), top, n // 2), -rng.integers(top - (1 << 20), top, n // 2)])
    return rng.standard_normal((n, 1, 2 * len(FREQ))).astype(np.float32), pos.astype(np.int32)[None]


# The angle: 2^31 positions times half a step of 2^-64 of a turn, the phase cut to 32 bits (2^-32 of a turn,
# 1.5e-9 rad), an angle of up to pi/4 converted and multiplied with one rounding each (2 * 2^-25 of pi/4, and the
# constant's 2^-24 of it): below 1e-7 rad. Sine and cosine are off by some 2^-23 more, and the two products and
# their sum by 3 * 2^-24 of |x| + |y|. The reference's own angle is held in 64 bits or more of mantissa.
TOL = 1e-7 + 2.0 ** -23 + 3 * 2.0 ** -24


@pytest.mark.parametrize("inverse", [False, True])
def test_far_positions_with_negative_frequencies(cpt, cuda_device, inverse):
    """Frequencies below zero turn as exactly as those above: the angle in 80 bits, reduced before it is a double."""
    x, pos = _inputs(4096)
    freq = [-f for f in FREQ]
    got = _turned(cpt, x, pos, freq, inverse)
    two_pi = 2 * np.longdouble("3.14159265358979323846264338327950288")
    n = len(freq)
    want = x.astype(np.float64)
    for i, f in enumerate(freq):
        turns = (pos[0].astype(np.longdouble) * np.longdouble(f)) / two_pi
        theta = ((turns - np.floor(turns)) * two_pi).astype(np.float64) * (-1.0 if inverse else 1.0)
        a, b = x[:, 0, i].astype(np.float64), x[:, 0, n + i].astype(np.float64)
        want[:, 0, i] = a * np.cos(theta) - b * np.sin(theta)
        want[:, 0, n + i] = a * np.sin(theta) + b * np.cos(theta)
    mag = np.abs(x[..., :n]) + np.abs(x[..., n:])
    assert np.all(np.abs(got - want) <= TOL * np.concatenate([mag, mag], -1))


def test_opposite_frequencies_are_inverse_rotations(cpt, cuda_device):
    x, pos = _inputs(4096)
    a = _turned(cpt, x, pos, FREQ, True)
    b = _turned(cpt, x, pos, [-f for f in FREQ])
    n = len(FREQ)
    mag = np.abs(x[..., :n]) + np.abs(x[..., n:])
    # both are off by TOL at most
    assert np.all(np.abs(a - b) <= 2 * TOL * np.concatenate([mag, mag], -1))
