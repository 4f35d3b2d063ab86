"""GPU tests of calls with something out of range: it is reported, and everything else is done as without it."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
ra = pytest.importorskip("context_ring_attention_gb300")
from tests.test_gpu_paged import Batch, _i32, _same_bits  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ra.load_library()


def _reported(kv):
    with pytest.raises(ra.RaError) as err:
        ra.ra_paged_sync_status(kv)
    assert err.value.name == "RA_ERR_INVALID_ARG"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rotated", [False, True])
@pytest.mark.parametrize("many", [0, 300])
@pytest.mark.parametrize("offset,good", [
    ([0, 100, 8, 16], [2]),          # one that ends behind the tokens, one that falls, one that is fine
    ([8, 2, 8, 16], [1, 2]),         # (tokens before the first offset)
    ([0, 5, 5, 3], [0, 1]),          # one that falls behind the others
    ([20, -7, 4, 16], [2]),
    ([0, 8, 2 ** 31 - 1, 8], [0]),
    ([100, 0, 16, 12], [1]),         # (tokens behind the last offset)
])
def test_appends_beside_offsets_that_fall(offset, good, many, rotated, dtype):
    """The sequences that are fine are appended whole, whatever the others' offsets are.  `many`: empty sequences behind."""
    lengths = [50, 33, 40]
    t = Batch(np.random.default_rng(3), [5, 5, 6], lengths, 4, 2, 64, dtype, 16)
    table = np.concatenate([t.ref.table, np.full((many, t.ref.width), -1)])
    off, n = _i32(offset + [offset[-1]] * many), _i32(lengths + [0] * many)
    k, v = t.random(16, 2).cuda(), t.random(16, 2).cuda()
    rope = ra.ra_rope_plan(64, dtype=dtype) if rotated else None
    q = t.q.cuda()
    q_out = torch.full_like(q, 7.0) if rotated else None
    ra.ra_paged_append(t.kv, t.cache, k, v, _i32(table), off, n, rope=rope, q=q if rotated else None, q_out=q_out)
    _reported(t.kv)
    want_q = torch.full_like(q, 7.0)
    for b in [b for b in good if offset[b + 1] > offset[b]]:
        rows = slice(offset[b], offset[b + 1])
        slots = torch.arange(lengths[b] - (rows.stop - rows.start), lengths[b])
        kk, at = k[rows], slots.int().cuda()[None]
        if rotated:
            kk = ra.ra_rope(rope, kk.transpose(0, 1)[None], position=at)[0].transpose(0, 1)
            want_q[rows] = ra.ra_rope(rope, q[rows].transpose(0, 1)[None], position=at)[0].transpose(0, 1)
        t.ref.put(b, slots, kk.cpu(), v[rows].cpu())
    assert _same_bits(t.cache, t.ref.data)
    if rotated:
        assert _same_bits(q_out, want_q)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("place", [False, True])
@pytest.mark.parametrize("tokens,counts", [(40, [0]), (2, [0, 0]), (300, [0, 0, 0])])
def test_weights_of_no_tokens(dtype, place, tokens, counts):
    """Sequences without new tokens keep their weights, in place and in another tensor, and slots beyond the
    weights are reported in both."""
    b, n = len(counts), 90
    t = Batch(np.random.default_rng(4), counts, [n] * b, 4, 2, 64, dtype, 16, tail=tokens)
    q, lse = t.q.cuda(), torch.zeros((tokens, 4), device="cuda")
    for width, fine in ((n, True), (n - 1, False)):
        before = torch.rand((b, 2, width)).cuda()
        weight = before.clone() if place else torch.zeros_like(before)
        ra.ra_paged_weigh(t.kv, t.cache, q, lse, t.table, t.offset, t.length, weight, weight_in=weight if place else before)
        if fine:
            ra.ra_paged_sync_status(t.kv)
        else:
            _reported(t.kv)
        assert _same_bits(weight, before)
