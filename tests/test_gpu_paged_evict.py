"""GPU tests of evictions from long sequences: weights that the CTAs of a cluster do not keep in shared memory, one
CTA and clusters of two and four a head, in place and elsewhere."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
ra = pytest.importorskip("context_ring_attention_gb300")
from tests import paged_ref  # noqa: E402
from tests.test_gpu_paged import _i32, _same_bits, _weights  # noqa: E402

SMEM = 49152  # weights that a CTA keeps at most


def stays(weight, n, keep, first, recent):
    """paged_ref.evict by one sort: the last key of lexsort counts first."""
    if n <= keep:
        return np.arange(n)
    j = np.arange(first, n - recent)
    w = np.asarray(weight, np.float64)[j]
    nan = np.isnan(w)
    order = np.lexsort((j, -np.where(nan, 0.0, w), nan))[:keep - first - recent]
    return np.concatenate([np.arange(first), np.sort(j[order]), np.arange(n - recent, n)])


@pytest.mark.parametrize("kind", ["plain", "ties", "odd"])
def test_the_order(kind):
    rng = np.random.default_rng(1)
    for n, keep, first, recent in ((40, 12, 0, 0), (40, 12, 3, 4), (40, 40, 0, 0), (40, 12, 12, 0), (40, 1, 0, 0), (40, 39, 1, 2)):
        for w in _weights(rng, 4, 1, n, kind)[:, 0].numpy():
            assert np.array_equal(stays(w, n, keep, first, recent), paged_ref.evict(w, n, keep, first, recent))


# heads, sequence lengths, weight_width more than the longest, keep, first, recent.  Of a GPU of 152 SMs a cluster has
# 4 CTAs up to 38 heads of all sequences, 2 up to 76, then 1; each keeps a fourth, half or all of a sequence's weights.
LONG = [
    (1, [200000], 3, 60000, 7, 50),          # four CTAs, in place one of them takes all
    (1, [4 * SMEM + 1], 0, 4 * SMEM, 0, 0),  # the first length that they do not hold, one slot leaves
    (1, [4 * SMEM - 40], 0, 300, 4, 100),    # the last lengths that they do
    (3, [200000, 5, 0, 70000], 0, 1000, 4, 500),
    (2, [200000], 70000, 4096, 4096, 0),     # the first ones alone
    (2, [200001], 0, 4096, 0, 4096),         # the last ones alone
    (40, [2 * SMEM + 700], 5, 50000, 4, 512),  # two CTAs
    (80, [SMEM + 1], 0, 20000, 4, 512),      # one CTA
    (80, [SMEM + 5000], 900, SMEM + 4999, 0, 1),
    (80, [SMEM - 4], 0, 2000, 1, 1),
]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["plain", "ties", "odd"])
@pytest.mark.parametrize("heads,lengths,more,keep,first,recent", LONG, ids=str)
def test_weights_beyond_shared_memory(heads, lengths, more, keep, first, recent, kind):
    """Lists, weights (into another tensor and in place) and some of the rows, which move into other pages; the old page
    table names a few pages again and again."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    rng = np.random.default_rng(keep + heads)
    b, pr, d = len(lengths), 256, 64
    width = -(-max(lengths) // pr)
    fits = [-(-min(n, keep) // pr) for n in lengths]
    pages = 8 + sum(fits)
    kv = ra.ra_paged_plan(pages, pr, heads, heads, d)
    cache = torch.zeros(ra.ra_paged_cache_shape(kv), dtype=torch.bfloat16, device="cuda")
    cache[:8] = torch.randn(cache[:8].shape, device="cuda").bfloat16()
    table = torch.from_numpy(rng.integers(0, 8, (b, width))).int().cuda()
    new = torch.full((b, max(1, -(-keep // pr))), -1, dtype=torch.int32)
    at = 8
    for i, n in enumerate(fits):
        new[i, :n] = torch.arange(at, at + n)
        at += n
    new = new.cuda()
    weight = _weights(rng, b, heads, max(lengths) + more, kind)
    want = [[stays(weight[i, h].numpy(), n, keep, first, recent) for h in range(heads)] for i, n in enumerate(lengths)]
    for form in ("out", "place"):
        w = weight.cuda()
        out = torch.full_like(w, 7.0) if form == "out" else w
        kept, new_length = ra.ra_paged_evict(kv, cache, table, _i32(lengths), w, keep, first=first, recent=recent, new_table=new,
                                             weight_out=out)
        ra.ra_paged_sync_status(kv)
        assert list(new_length.cpu()) == [min(n, keep) for n in lengths]
        kept, got = kept.cpu(), out.cpu()
        for i, n in enumerate(lengths):
            m = min(n, keep)
            lists = np.stack(want[i]) if m else np.zeros((heads, 0), np.int64)
            assert np.array_equal(kept[i, :, :m].numpy(), lists) and (kept[i, :, m:] == -1).all()
            lists = torch.from_numpy(lists)
            assert _same_bits(got[i, :, :m], weight[i].gather(1, lists))
            rest = weight[i, :, m:] if form == "place" else torch.full_like(weight[i, :, m:], 7.0)
            assert _same_bits(got[i, :, m:], rest)
            # the rows of a few slots
            some = torch.from_numpy(np.unique(np.append(rng.integers(0, m, 200), [0, m - 1]))) if m else torch.zeros(0).long()
            old, to = lists[:, some].cuda(), some.cuda()
            page = table[i].long()[old // pr]
            head = torch.arange(heads, device="cuda")[:, None]
            assert _same_bits(cache[new[i].long()[to // pr][None].expand_as(old), :, head, (to % pr)[None].expand_as(old)],
                              cache[page, :, head, old % pr])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f32", 128)])
@pytest.mark.parametrize("heads,lengths,keep", [(1, [33001], 8192), (2, [20000, 12000], 11000), (5, [9000], 8999), (3, [7000, 100, 6000], 3000),
                                                (8, [5000] * 4, 4096), (16, [3000] * 8, 1000)])
def test_rows_in_place(heads, lengths, keep, dtype, d):
    """Clusters of one to eight CTAs walk the lists of one head or of many: every row of the cache, bit for bit."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    rng = np.random.default_rng(keep)
    b, pr = len(lengths), 64
    used = [-(-n // pr) for n in lengths]
    kv = ra.ra_paged_plan(sum(used) + 1, pr, heads, heads, d, dtype=dtype)
    cache = torch.randn(ra.ra_paged_cache_shape(kv), device="cuda").to(paged_ref.DT[dtype])
    order, table, at = rng.permutation(sum(used) + 1), np.full((b, max(used)), -1), 0
    for i, n in enumerate(used):
        table[i, :n] = order[at:at + n]
        at += n
    weight = _weights(rng, b, heads, max(lengths), "ties")
    before, w = cache.clone(), weight.cuda()
    kept, _ = ra.ra_paged_evict(kv, cache, _i32(table), _i32(lengths), w, keep, first=4, recent=100)
    ra.ra_paged_sync_status(kv)
    want = before.clone()
    table = torch.from_numpy(table)
    for i, n in enumerate(lengths):
        m, pages = min(n, keep), table[i].cuda()
        for h in range(heads):
            stay = torch.from_numpy(stays(weight[i, h].numpy(), n, keep, 4, 100)).cuda()
            assert torch.equal(kept[i, h, :m].long(), stay)
            to = torch.arange(m, device="cuda")
            want[pages[to // pr], :, h, to % pr] = before[pages[stay // pr], :, h, stay % pr]
    assert _same_bits(cache, want)
