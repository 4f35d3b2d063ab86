"""GPU tests of the ramp scaling of rotary positions where its two ends meet or cross.

The speeds here are written pair by pair from the words of include/ra.h: t = (j - j0) / (j1 - j0) held to 0..1, with
j1 - j0 at least 0.001."""

import math

import pytest

torch = pytest.importorskip("torch")
ra = pytest.importorskip("context_ring_attention_gb300")
from tests.window_ref import assert_within  # noqa: E402

RAMPS = [
    # rotary_dim, base, factor, original, low, high; j0 and j1; the share of each pair's speed that is divided
    (32, 100.0, 8.0, 1 << 21, 1.0, 32.0, (32, 31), lambda j: 0.0),                 # every pair turns more than `high` times
    (32, 100.0, 8.0, 1 << 30, 1.0, 32.0, (53, 31), lambda j: 0.0),
    (128, 10000.0, 8.0, 4, 1.0, 32.0, (0, -3), lambda j: 0.0 if j == 0 else 1.0),  # no pair turns `low` times
    (64, 10000.0, 4.0, 1, 1.0, 2.0, (0, -6), lambda j: 0.0 if j == 0 else 1.0),
    (64, 10000.0, 4.0, 7, 1.0, 32.0, (0, 1), lambda j: min(j, 1)),                 # pairs 0 and 1
    (16, 1000.0, 2.0, 100, 1.2, 1.3, (2, 3), lambda j: 0.0 if j <= 2 else 1.0),
    (2, 10000.0, 4.0, 1 << 20, 1.0, 4.0, (1, 1), lambda j: 0.0),                   # one pair, both ends behind it
    (64, 10000.0, 8.0, 4096, 1.0, 32.0, (10, 23), lambda j: min(1.0, max(0.0, (j - 10) / 13))),
]


def ends(rot, base, original, low, high):
    at = lambda turns: rot * math.log(original / (2 * math.pi * turns)) / (2 * math.log(base))
    return max(math.floor(at(high)), 0), min(math.ceil(at(low)), rot - 1)


@pytest.mark.parametrize("rot,base,factor,original,low,high,j01,share", RAMPS)
def test_the_ends(rot, base, factor, original, low, high, j01, share):
    """The shares above are those of the definition."""
    j0, j1 = ends(rot, base, original, low, high)
    assert (j0, j1) == j01
    for j in range(rot // 2):
        assert abs(min(1.0, max(0.0, (j - j0) / max(j1 - j0, 0.001))) - share(j)) < 1e-12


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot,base,factor,original,low,high,j01,share", RAMPS)
def test_ramp(rot, base, factor, original, low, high, j01, share, interleaved):
    """Rows whose pairs are (1, 0): the outputs are the angles' cosines and sines.  Each is off by 2^-21 as
    paged_ref.py counts it (the angle cut to 2^-33 of a turn, float32 functions, one rounding), and by 2^-51 of the
    angle for the speeds' float64 arithmetic here and there."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    rope = ra.ra_rope_plan(rot, base=base, scaling="ramp", factor=factor, original=original, low=low, high=high,
                           interleaved=interleaved, dtype="f32")
    pos = torch.tensor([[0, 1, 2, 3, 7, 100, 4095, -5, 1000003]], dtype=torch.int32)
    half, n = rot // 2, pos.shape[1]
    one, two = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, half), slice(half, rot))
    x = torch.zeros((1, 1, n, rot))
    x[..., one] = 1.0
    got = ra.ra_rope(rope, x.cuda(), position=pos.cuda()).cpu()
    w = [base ** (-2.0 * j / rot) for j in range(half)]
    speed = torch.tensor([(1 - share(j)) * w[j] + share(j) * w[j] / factor for j in range(half)], dtype=torch.float64)
    a = pos[0].double()[:, None] * speed
    bound = 2.0 ** -21 + 2.0 ** -51 * a.abs()
    assert_within(got[0, 0][:, one], a.cos(), bound, "cosines")
    assert_within(got[0, 0][:, two], a.sin(), bound, "sines")
