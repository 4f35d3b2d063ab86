"""GPU tests of chunks whose tokens see two or three keys, where every rounding shows.

bf16 chunks weigh the values by rounded weights r_i = p_i (1 + d_i), |d_i| <= u = 2^-8 (half a step), and divide by the
sum of the exact ones with each key tile's largest one, t, as rounded: O' = sum r_i v_i / (l + sum_t (r_t - p_t)).  To first
order O' - O = sum d_i p_i v_i / l - O sum_t d_t p_t / l.  The first term is at most u sum p_i |v_i| / l, which
paged_ref.attend's bound has; the second is at most u |O| sum_t p_t / l <= u |O|, which it lacks: it holds for a sum of
the exact weights, as the kernels of few rows divide by.  Terms of second order are u^2 = 2^-16 of the magnitudes, below the
2^-14 of them that the bound has for the scores."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytest.importorskip("context_ring_attention_gb300")
from tests import paged_ref  # noqa: E402
from tests.paged_ref import U  # noqa: E402
from tests.test_gpu_paged import Batch, ra  # noqa: E402
from tests.window_ref import assert_within  # noqa: E402


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hk,d,scale", [(10, 2, 64, None), (8, 2, 128, None), (128, 1, 64, 0.5), (20, 1, 128, 0.5)])
@pytest.mark.parametrize("window,sinks", [(2, 1), (3, 0), (1, 2), (2, 0)])
@pytest.mark.parametrize("seed", range(3))
def test_few_keys(hq, hk, d, scale, window, sinks, seed):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    rng = np.random.default_rng(seed)
    counts = [int(rng.integers(1, 40)) for _ in range(40)]
    lengths = [n + int(rng.integers(0, 400)) for n in counts]
    t = Batch(rng, counts, lengths, hq, hk, d, "bf16", 16, window=window, sinks=sinks, scale=scale)
    o, lse = (x.cpu() for x in t.attend())
    ra.ra_paged_sync_status(t.kv)
    u = U["bf16"]
    for b, n in enumerate(lengths):
        j = torch.arange(n)
        j = j[paged_ref.sees(t.slots(b), j, window, sinks).any(0)]
        ow, lw, ob, lb = paged_ref.attend(t.ref.rows(b, j, 0), t.ref.rows(b, j, 1), t.q[t.rows(b)], t.slots(b), j, window, sinks, u, scale)
        assert_within(lse[t.rows(b)], lw, lb, f"LSE of sequence {b}")
        assert_within(o[t.rows(b)], ow, ob + u * ow.abs(), f"O of sequence {b}")
