"""GPU tests of the paged cache: appending, attention of chunks, weights, eviction, and a sequence
taken through all of them, against the plain form in paged_ref.py."""

import math
import os
import subprocess
import sys

import numpy as np
import pytest

from tests.conftest import ROOT

torch = pytest.importorskip("torch")
ra = pytest.importorskip("context_ring_attention_gb300")
from tests import paged_ref  # noqa: E402
from tests.paged_ref import DT, U  # noqa: E402
from tests.window_ref import assert_within  # noqa: E402

gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library(request):
    if torch.cuda.is_available():
        ra.load_library()


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _same_bits(a, b):
    view = torch.int16 if a.dtype == torch.bfloat16 else torch.int32
    return torch.equal(a.cpu().contiguous().view(view), b.cpu().contiguous().view(view))


class Batch:
    """A packed batch over a cache: `lead` and `tail` tokens of no sequence around it."""

    def __init__(self, rng, counts, lengths, hq, hk, d, dtype, page_rows, lead=0, tail=0, window=0, sinks=0, scale=None, **kw):
        self.rng, self.counts, self.lengths = rng, list(counts), list(lengths)
        self.hq, self.hk, self.d, self.dtype, self.window, self.sinks, self.scale = hq, hk, d, dtype, window, sinks, scale
        self.ref = paged_ref.Cache(rng, lengths, page_rows, hk, d, dtype, **kw)
        self.kv = ra.ra_paged_plan(self.ref.pages, page_rows, hq, hk, d, dtype=dtype, window=window, sinks=sinks,
                                   scale=scale)
        self.cache, self.table = self.ref.data.cuda(), _i32(self.ref.table)
        self.first = np.concatenate([[lead], lead + np.cumsum(counts)])
        self.tokens = int(self.first[-1]) + tail
        self.offset, self.length = _i32(self.first), _i32(lengths)
        self.q = self.random(self.tokens, hq)

    def random(self, n, h):
        return torch.from_numpy(self.rng.normal(size=(n, h, self.d))).to(DT[self.dtype])

    def rows(self, b):
        return slice(int(self.first[b]), int(self.first[b + 1]))

    def slots(self, b):
        return torch.arange(self.lengths[b] - self.counts[b], self.lengths[b])

    def attend(self, **kw):
        return ra.ra_paged_attend(self.kv, self.cache, self.q.cuda(), self.table, self.offset, self.length, **kw)

    def check_attend(self, o, lse):
        ra.ra_paged_sync_status(self.kv)
        o, lse = o.cpu(), lse.cpu()
        for b, n in enumerate(self.lengths):
            if not self.counts[b]:
                continue
            j = torch.arange(n)
            seen = paged_ref.sees(self.slots(b), j, self.window, self.sinks).any(0)
            j = j[seen]
            ow, lw, ob, lb = paged_ref.attend(self.ref.rows(b, j, 0), self.ref.rows(b, j, 1), self.q[self.rows(b)], self.slots(b), j,
                                              self.window, self.sinks, U[self.dtype], self.scale)
            assert_within(lse[self.rows(b)], lw, lb, f"LSE of sequence {b}")
            assert_within(o[self.rows(b)], ow, ob, f"O of sequence {b}")

    def check_weigh(self, weight, before, lse):
        """weight, before: [batch, Hkv, slots], the first on the CPU after the call."""
        ra.ra_paged_sync_status(self.kv)
        for b, n in enumerate(self.lengths):
            j = torch.arange(n)
            old = n - self.counts[b]
            want, bound = torch.zeros((self.hk, n), dtype=torch.float64), torch.zeros((self.hk, n), dtype=torch.float64)
            if self.counts[b]:
                seen = paged_ref.sees(self.slots(b), j, self.window, self.sinks).any(0)
                js = j[seen]
                want[:, js], bound[:, js] = paged_ref.weigh(self.ref.rows(b, js, 0), self.q[self.rows(b)],
                                                            lse[self.rows(b)].cpu(), self.slots(b), js, self.window, self.sinks,
                                                            self.scale)
            want[:, :old] += before[b, :, :old].double()
            assert_within(weight[b, :, :n], want, bound + U["f32"] * want.abs() + 1e-37, f"weights of sequence {b}")


# ------------------------------------------------------------------------ append --
@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,rot,interleaved", [(64, 64, False), (128, 128, True), (128, 64, False), (64, 6, True), (128, 126, False)])
@pytest.mark.parametrize("counts,lengths,page_rows", [([1], [1], 16), ([3, 0, 40], [50, 7, 40], 32),
                                                      ([1] * 20, list(range(1, 21)), 16), ([700], [1000], 112)])
def test_append(dtype, d, rot, interleaved, counts, lengths, page_rows):
    """Every row of the cache bit for bit: rotated keys as ra_rope makes them, values as they are,
    everything else untouched; rotated queries; tokens of no sequence left alone."""
    rng = np.random.default_rng(d + len(counts))
    hq, hk = 6, 2
    t = Batch(rng, counts, lengths, hq, hk, d, dtype, page_rows, lead=2, tail=3)
    rope = ra.ra_rope_plan(d, rot, interleaved=interleaved, dtype=dtype)
    qkv = t.random(t.tokens, hq + 2 * hk).cuda()  # side by side, as one projection leaves them
    q, k, v = qkv.split([hq, hk, hk], 1)
    for position in (None, torch.from_numpy(rng.integers(0, 100000, t.tokens)).int().cuda()):
        at = torch.zeros(t.tokens, dtype=torch.int32)
        for b in range(len(counts)):
            at[t.rows(b)] = t.slots(b).int()
        if position is not None:
            at = position.cpu()
        turned = [ra.ra_rope(rope, x.transpose(0, 1)[None], position=at.cuda()[None])[0].transpose(0, 1).cpu() for x in (q, k)]
        q_out = torch.full((t.tokens, hq, d), 7.0, dtype=DT[dtype], device="cuda")
        got = ra.ra_paged_append(t.kv, t.cache, k, v, t.table, t.offset, t.length, rope=rope, position=position, q=q, q_out=q_out)
        ra.ra_paged_sync_status(t.kv)
        assert got is q_out
        want = torch.full((t.tokens, hq, d), 7.0, dtype=DT[dtype])
        for b in range(len(counts)):
            want[t.rows(b)] = turned[0][t.rows(b)]
            t.ref.put(b, t.slots(b), turned[1][t.rows(b)], v[t.rows(b)].cpu())
        assert _same_bits(got, want)
        assert _same_bits(t.cache, t.ref.data)
    # without a rotation: as they are
    assert ra.ra_paged_append(t.kv, t.cache, k, v, t.table, t.offset, t.length) is None
    for b in range(len(counts)):
        t.ref.put(b, t.slots(b), k[t.rows(b)].cpu(), v[t.rows(b)].cpu())
    assert _same_bits(t.cache, t.ref.data)
    # queries in place, an output of the call's own, keys alone
    q2 = q.contiguous()
    own = ra.ra_paged_append(t.kv, t.cache, k, v, t.table, t.offset, t.length, rope=rope, q=q)
    assert ra.ra_paged_append(t.kv, t.cache, k, v, t.table, t.offset, t.length, rope=rope, q=q2, q_out=q2) is q2
    for b in range(len(counts)):
        assert _same_bits(own[t.rows(b)], q2[t.rows(b)])
    before = t.cache.clone()
    ra.ra_paged_append(t.kv, t.cache, k, v, t.table, t.offset, t.length, rope=rope)
    ra.ra_paged_sync_status(t.kv)
    assert _same_bits(before, t.cache)


# --------------------------------------------------------------------- attention --
HEADS = [(1, 1), (4, 1), (6, 2), (16, 2), (3, 3)]
BATCHES = [([1], [1]), ([1, 1, 1], [15, 16, 17]), ([2, 0, 5, 1], [300, 31, 5, 129]), ([40, 1, 3], [40, 1000, 500]),
           ([1], [5000]), ([17, 130], [130, 400])]


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hk", HEADS)
@pytest.mark.parametrize("counts,lengths", BATCHES, ids=str)
def test_attention(dtype, d, hq, hk, counts, lengths):
    """From one token to chunks, one share to many, groups and tokens that fill no tile, sequences
    without new tokens.  Everything that no sequence wrote is NaN."""
    t = Batch(np.random.default_rng(hq + sum(counts)), counts, lengths, hq, hk, d, dtype, 48, lead=1, tail=2)
    o = torch.full((t.tokens, hq, d), 7.0, dtype=DT[dtype], device="cuda")
    lse = torch.full((t.tokens, hq), 7.0, device="cuda")
    t.check_attend(*t.attend(o=o, lse=lse))
    assert (o[:1] == 7).all() and (o[-2:] == 7).all() and (lse[:1] == 7).all() and (lse[-2:] == 7).all()


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 3), (16, 16), (100, 4), (129, 200), (5000, 0), (1 << 40, 1 << 40)])
@pytest.mark.parametrize("counts", [[1, 1, 1, 1], [5, 3, 70, 16], [300, 1, 2, 0]], ids=str)
def test_windowed_attention(dtype, window, sinks, counts):
    rng = np.random.default_rng(window % 1000 + counts[0])
    t = Batch(rng, counts, [700, 3, 129, 16], 6, 2, 128, dtype, 32, window=window, sinks=sinks)
    t.check_attend(*t.attend())


@gpu
@pytest.mark.parametrize("page_rows", [16, 32, 48, 64, 112, 128, 256, 4096])
@pytest.mark.parametrize("counts,lengths", [([1, 1], [1500, 700]), ([200, 33], [1500, 700])])
def test_page_sizes(page_rows, counts, lengths):
    """Pages that end inside a tile."""
    t = Batch(np.random.default_rng(page_rows), counts, lengths, 8, 2, 128, "bf16", page_rows)
    t.check_attend(*t.attend())


@gpu
@pytest.mark.parametrize("counts,lengths,hq,hk", [([1500], [1500], 4, 1), ([1000, 600, 1], [4000, 700, 3000], 8, 2),
                                                  ([257], [2000], 5, 1), ([300] * 6, [300, 600, 2000, 301, 900, 5000], 2, 2),
                                                  ([9], [500], 72, 1), ([7, 3], [300, 200], 128, 1), ([5], [200], 160, 1)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (300, 40)])
def test_chunks(counts, lengths, hq, hk, d, window, sinks):
    """Prompts without and with a prefix, chunks that fill several tiles."""
    t = Batch(np.random.default_rng(hq + d), counts, lengths, hq, hk, d, "bf16", 64, window=window, sinks=sinks)
    t.check_attend(*t.attend())


@gpu
@pytest.mark.parametrize("counts", [[1, 2], [150, 1]])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_cache_beyond_4_gb(dtype, counts):
    """The same sequences on pages at the end of a pool of 6 GB: every call's results bit for bit."""
    rng = np.random.default_rng(2)
    t = Batch(rng, counts, [700, 300], 4, 2, 128, dtype, 64)
    far = int(6e9 / (2 * 2 * 64 * 128 * DT[dtype].itemsize))
    kv = ra.ra_paged_plan(far, 64, 4, 2, 128, dtype=dtype)
    cache = torch.empty(ra.ra_paged_cache_shape(kv), dtype=DT[dtype], device="cuda")
    cache[far - t.ref.pages:] = t.cache
    table = t.table + (far - t.ref.pages)
    rope = ra.ra_rope_plan(128, dtype=dtype)
    k, v, q = t.random(t.tokens, 2).cuda(), t.random(t.tokens, 2).cuda(), t.q.cuda()
    out = []
    for plan, c, tab in ((t.kv, t.cache, t.table), (kv, cache, table)):
        turned = ra.ra_paged_append(plan, c, k, v, tab, t.offset, t.length, rope=rope, q=q)
        o, lse = ra.ra_paged_attend(plan, c, turned, tab, t.offset, t.length)
        w = torch.zeros((2, 2, 700), device="cuda")
        ra.ra_paged_weigh(plan, c, turned, lse, tab, t.offset, t.length, w)
        weighed = w.clone()
        kept, n = ra.ra_paged_evict(plan, c, tab, t.length, w, 250, first=1, recent=20)
        ra.ra_paged_sync_status(plan)
        out.append((turned, o, lse, weighed, kept, n, c[-t.ref.pages:]))
    for a, e in zip(*out):
        assert _same_bits(a, e) if a.is_floating_point() else torch.equal(a, e)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_difficult_scores(dtype):
    """One key far above the others, all scores equal, scores of +-200, tiny ones."""
    rng = np.random.default_rng(8)
    t = Batch(rng, [4, 40], [200, 300], 4, 2, 128, dtype, 32)
    for b, (n, size) in enumerate(((200, 25.0), (300, 1e-3))):
        k = t.ref.random(rng, n) * size
        k[n // 2] *= 3
        t.ref.put(b, np.arange(n), k, t.ref.random(rng, n))
    t.ref.put(1, np.arange(100), torch.zeros((100, 2, 128), dtype=DT[dtype]), t.ref.random(rng, 100))
    t.cache = t.ref.data.cuda()
    t.check_attend(*t.attend())


@gpu
@pytest.mark.parametrize("counts", [[2, 1], [90, 60]])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_unseen_slots_may_hold_anything(dtype, counts):
    """NaN and infinities outside the window and beyond the length, and pages that no token sees
    missing from the table."""
    rng = np.random.default_rng(5)
    window, sinks, lengths = 33, 4, [400, 230]
    t = Batch(rng, counts, lengths, 4, 2, 128, dtype, 16, window=window, sinks=sinks)
    o, lse = t.attend()
    t.check_attend(o, lse)
    table = t.ref.table.copy()
    for b, n in enumerate(lengths):
        gone = np.arange(sinks, n - counts[b] - window + 1)
        junk = torch.where(torch.rand((len(gone), 2, 128)) < 0.5, math.nan, math.inf).to(DT[dtype])
        t.ref.put(b, gone, junk, -junk)
        for e in range(t.ref.width):
            if e > 0 and (e + 1) * 16 <= n - counts[b] - window + 1:
                table[b, e] = -1 - e
    t.cache, t.table = t.ref.data.cuda(), _i32(table)
    o2, lse2 = t.attend()
    ra.ra_paged_sync_status(t.kv)
    assert _same_bits(o, o2) and _same_bits(lse, lse2)
    w = torch.zeros((2, 2, 400), device="cuda")
    ra.ra_paged_weigh(t.kv, t.cache, t.q.cuda(), lse, t.table, t.offset, t.length, w)
    ra.ra_paged_sync_status(t.kv)
    assert torch.isfinite(w).all()
    # a NaN that every token sees comes through
    t.ref.put(0, [0], torch.full((1, 2, 128), math.nan, dtype=DT[dtype]), torch.zeros((1, 2, 128), dtype=DT[dtype]))
    t.cache, t.table = t.ref.data.cuda(), _i32(t.ref.table)
    o3, lse3 = t.attend()
    assert torch.isnan(o3[t.rows(0)]).all() and torch.isnan(lse3[t.rows(0)]).all() and _same_bits(o3[t.rows(1)], o[t.rows(1)])


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("counts", [[2, 1, 3], [200, 1, 30]])
def test_out_of_range_tables_are_reported_and_skipped(dtype, counts):
    rng = np.random.default_rng(13)
    lengths = [300, 60, 33]
    t = Batch(rng, counts, lengths, 4, 2, 64, dtype, 32)
    q, before = t.q.cuda(), t.cache.clone()
    k = v = t.random(t.tokens, 2).cuda()
    weight = torch.full((3, 2, 320), 3.0, device="cuda")

    def reported():
        with pytest.raises(ra.RaError) as err:
            ra.ra_paged_sync_status(t.kv)
        assert err.value.name == "RA_ERR_INVALID_ARG"
        ra.ra_paged_sync_status(t.kv)  # cleared

    n, w = t.tokens, t.ref.width * 32
    for offset, length in (([0, 5, 3, 3], lengths), ([-1, 0, 0, 0], lengths), ([0, 0, 0, n + 1], lengths), ([5, 2, 2, 2], lengths),
                           (t.first, [counts[0] - 1, 60, 33]), (t.first, [w + 1, 60, 33]), (t.first, [-1, 60, 33]),
                           (t.first, [2 ** 31 - 1, 60, 33]), ([0, -2 ** 31, 2 ** 31 - 1, n], lengths)):
        off, ln = _i32(offset), _i32(length)
        good = [b for b in range(3) if 0 <= offset[b] <= offset[b + 1] <= n and offset[b + 1] - offset[b] <= length[b] <= w]
        o, lse = torch.full_like(q, 7.0), torch.full((n, 4), 7.0, device="cuda")
        ra.ra_paged_attend(t.kv, t.cache, q, t.table, off, ln, o=o, lse=lse)
        reported()
        left = np.ones(n, bool)
        for b in good:
            rows = slice(int(offset[b]), int(offset[b + 1]))
            left[rows] = False
            if rows.start == t.first[b] and rows.stop == t.first[b + 1] and rows.stop > rows.start:
                ow, lw, ob, lb = paged_ref.attend(t.ref.rows(b, np.arange(length[b]), 0), t.ref.rows(b, np.arange(length[b]), 1),
                                                  t.q[rows], t.slots(b), torch.arange(length[b]), 0, 0, U[dtype])
                assert_within(o[rows].cpu(), ow, ob, "O")
        assert (o[torch.from_numpy(left)] == 7).all() and (lse[torch.from_numpy(left)] == 7).all()
        out = weight.clone()
        ra.ra_paged_weigh(t.kv, t.cache, q, lse, t.table, off, ln, out)
        reported()
        for b in set(range(3)) - set(good):
            assert (out[b] == 3).all()
        ra.ra_paged_append(t.kv, t.cache, k, v, t.table, off, ln)
        reported()
        t.cache = before.clone()
    # pages that are none: their slots are left out, not written, not weighed
    table = t.ref.table.copy()
    table[0, 1], table[0, 8], table[2, 0] = 1 << 30, -1, t.ref.pages
    o, lse = ra.ra_paged_attend(t.kv, t.cache, q, _i32(table), t.offset, t.length)
    reported()
    for b in range(2):
        j = torch.tensor([x for x in range(lengths[b]) if b or x // 32 not in (1, 8)])
        ow, lw, ob, lb = paged_ref.attend(t.ref.rows(b, j, 0), t.ref.rows(b, j, 1), t.q[t.rows(b)], t.slots(b), j, 0, 0, U[dtype])
        assert_within(o[t.rows(b)].cpu(), ow, ob, "O")
        assert_within(lse[t.rows(b)].cpu(), lw, lb, "LSE")
    one = t.rows(2).start  # tokens whose only slots lie on the page that is none
    some = int(max(0, 32 - (lengths[2] - counts[2])))
    assert (o[one:one + some] == 0).all() and torch.isneginf(lse[one:one + some]).all()
    ra.ra_paged_weigh(t.kv, t.cache, q, torch.zeros_like(lse), _i32(table), t.offset, t.length, weight)
    reported()
    assert (weight[0, :, 32:64] == 3).all() and (weight[0, :, 256:288] == 3).all() and (weight[2, :, :32] == 3).all()
    assert (weight[0, :, :32] != 3).all() and (weight[0, :, 300:] == 3).all()
    ra.ra_paged_append(t.kv, t.cache, k, v, _i32(table), t.offset, t.length)
    reported()
    for b in range(3):
        ok = torch.tensor([int(s) for s in t.slots(b) if 0 <= table[b, int(s) // 32] < t.ref.pages], dtype=torch.long)
        at = ok - (lengths[b] - counts[b]) + t.rows(b).start
        t.ref.put(b, ok, k[at].cpu(), v[at].cpu())
    assert _same_bits(t.cache, t.ref.data)


@gpu
@pytest.mark.parametrize("counts,lengths", [([1] * 150, None), ([1] * 64, [2000] * 64), ([1, 300] * 20, None), ([0] * 300 + [1], None)])
def test_many_sequences(counts, lengths):
    rng = np.random.default_rng(len(counts))
    lengths = lengths or [int(c + rng.integers(0, 400)) for c in counts]
    t = Batch(rng, counts, lengths, 8, 2, 64, "bf16", 32)
    o, lse = t.attend()
    t.check_attend(o, lse)
    before = torch.rand((len(counts), 2, max(lengths)))
    weight = before.cuda()
    ra.ra_paged_weigh(t.kv, t.cache, t.q.cuda(), lse, t.table, t.offset, t.length, weight, weight_in=weight)
    t.check_weigh(weight.cpu(), before, lse)


@gpu
def test_most_sequences():
    """As many as a call takes, with equal lengths: every row is the mean of two values."""
    n, kv = 4096, ra.ra_paged_plan(4096, 16, 2, 1, 64)
    cache = torch.zeros((4096, 2, 1, 16, 64), dtype=torch.bfloat16, device="cuda")
    table = torch.randperm(n).int()[:, None].contiguous().cuda()
    offset, length = torch.arange(n + 1).int().cuda(), torch.full((n,), 2, dtype=torch.int32, device="cuda")
    v = torch.arange(n, device="cuda").remainder(64)[:, None, None].expand(n, 1, 64).bfloat16()
    for step in (1, 2):
        ra.ra_paged_append(kv, cache, torch.zeros_like(v), v * step, table, offset, length - 2 + step)
    o, lse = ra.ra_paged_attend(kv, cache, torch.ones((n, 2, 64), dtype=torch.bfloat16, device="cuda"), table, offset, length)
    ra.ra_paged_sync_status(kv)
    assert torch.equal(o[:, 0], (v[:, 0] * 1.5)) and torch.allclose(lse, torch.full_like(lse, math.log(2)), atol=1e-6)


@gpu
def test_own_outputs_strides_and_shared_pages():
    """Queries and outputs in other orders, scratch with room behind it, two sequences on one page."""
    rng = np.random.default_rng(9)
    t = Batch(rng, [3, 40], [2000, 1500], 8, 2, 128, "bf16", 32)
    t.ref.table[1, :3] = t.ref.table[0, :3]
    t.table = _i32(t.ref.table)
    need = ra.ra_paged_attend_scratch_size(t.kv, 2, 43, t.ref.width)
    assert need > 0
    scratch = torch.full((need // 4 + 64,), math.nan, device="cuda")
    want = t.attend(scratch=scratch)
    assert torch.isnan(scratch[need // 4:]).all()
    t.check_attend(*want)
    q = torch.zeros((8, 43, 136), dtype=torch.bfloat16, device="cuda")[:, :, 8:].transpose(0, 1)
    q.copy_(t.q)
    out = torch.full((8, 50, 136), 7.0, dtype=torch.bfloat16, device="cuda")
    o = out[:, 2:45, 8:].transpose(0, 1)
    got = ra.ra_paged_attend(t.kv, t.cache, q, t.table, t.offset, t.length, o=o, scratch=scratch)
    ra.ra_paged_sync_status(t.kv)
    assert got[0] is o and _same_bits(o, want[0]) and _same_bits(got[1], want[1])
    o.fill_(7.0)
    assert (out == 7).all()
    with pytest.raises(ValueError):
        t.attend(scratch=scratch[:need // 4 - 1])
    with pytest.raises(ra.RaError):
        t.attend(scratch=scratch[1:])
    with pytest.raises(ra.RaError):
        t.attend(o=torch.empty((43, 8, 132), dtype=torch.bfloat16, device="cuda")[:, :, 2:130])


@gpu
@pytest.mark.parametrize("counts", [[1, 1, 1], [130, 1, 60]])
def test_graphs_follow_the_tables(counts):
    """A captured step replayed after its lengths, offsets and pages changed; two graphs side by
    side with a scratch each."""
    rng = np.random.default_rng(21)
    lengths = [900, 300, 400]
    batches = [Batch(rng, counts, lengths, 8, 2, 128, "bf16", 32) for _ in range(2)]
    rope = ra.ra_rope_plan(128)
    graphs = []
    for t in batches:
        t.k, t.v, t.qd = t.random(t.tokens, 2).cuda(), t.random(t.tokens, 2).cuda(), t.q.cuda()
        t.o, t.lse, t.turned = torch.empty_like(t.qd), torch.empty((t.tokens, 8), device="cuda"), torch.empty_like(t.qd)
        t.scratch = torch.empty(max(1, ra.ra_paged_attend_scratch_size(t.kv, 3, t.tokens, t.ref.width) // 4), device="cuda")
        t.weight = torch.zeros((3, 2, 1000), device="cuda")
        t.more = torch.empty(max(1, ra.ra_paged_weigh_scratch_size(t.kv, 3, t.tokens, t.ref.width) // 4), device="cuda")

        def step(t=t):
            ra.ra_paged_append(t.kv, t.cache, t.k, t.v, t.table, t.offset, t.length, rope=rope, q=t.qd, q_out=t.turned)
            ra.ra_paged_attend(t.kv, t.cache, t.turned, t.table, t.offset, t.length, o=t.o, lse=t.lse, scratch=t.scratch)
            ra.ra_paged_weigh(t.kv, t.cache, t.turned, t.lse, t.table, t.offset, t.length, t.weight, scratch=t.more)

        step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        graphs.append((t, g, step))
    n = batches[0].tokens
    fewer = [0, 1, 1, 2] if counts[0] == 1 else [0, 7, 9, n - 3]
    for length, offset in ((lengths, None), ([800, 131, 61], None), ([500, 2, 300], fewer)):
        streams = [torch.cuda.Stream() for _ in graphs]
        for t, _, _ in graphs:
            t.length.copy_(_i32(length))
            if offset is not None:
                t.offset.copy_(_i32(offset))
            t.ref.table[:, [0, 1]] = t.ref.table[:, [1, 0]]
            t.table.copy_(_i32(t.ref.table))
        torch.cuda.synchronize()
        for (t, g, _), s in zip(graphs, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                for _ in range(3):
                    g.replay()
        torch.cuda.synchronize()
        for t, _, step in graphs:
            o, lse, w = t.o.clone(), t.lse.clone(), t.weight.clone()
            t.o.fill_(5.0), t.lse.fill_(5.0), t.weight.fill_(0.0)
            step()
            ra.ra_paged_sync_status(t.kv)
            end = int(t.offset[-1])
            assert _same_bits(o[:end], t.o[:end]) and _same_bits(lse[:end], t.lse[:end])
            for b in range(3):
                assert _same_bits(w[b, :, :length[b]], t.weight[b, :, :length[b]])


@gpu
@pytest.mark.parametrize("counts", [[1, 1], [260, 50]])
def test_another_stream(counts):
    """Calls on a stream of their own, with buffers of its own, beside calls on the current one."""
    rng = np.random.default_rng(31)
    t = Batch(rng, counts, [3000, 700], 8, 2, 128, "bf16", 64)
    want = t.attend()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q = t.q.cuda()
    torch.cuda.synchronize()
    got = [ra.ra_paged_attend(t.kv, t.cache, q, t.table, t.offset, t.length, stream=s) for s in (side, None, side, None)]
    torch.cuda.synchronize()
    for o, lse in got:
        assert _same_bits(o, want[0]) and _same_bits(lse, want[1])
    ra.ra_paged_sync_status(t.kv, side)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("keep", [40, 1200])
def test_a_captured_step_under_a_budget(dtype, keep):
    """A decoding step with its eviction in place, captured and replayed on another stream, against
    the same calls one by one: every output, the cache and the weights, bit for bit."""
    b, hq, hk, d, pr, steps = 2, 4, 2, 64, 16, 12
    rng = np.random.default_rng(keep)
    lengths = [keep - 5, keep]
    rows = lambda h: torch.from_numpy(rng.normal(size=(steps, b, h, d))).to(DT[dtype]).cuda()
    q, k, v = rows(hq), rows(hk), rows(hk)
    width = -(-(keep + 1) // pr)
    rope = ra.ra_rope_plan(d, dtype=dtype)
    runs = []
    start = torch.from_numpy(rng.normal(size=(b * width, 2, hk, pr, d))).to(DT[dtype]).cuda()
    heavy = torch.from_numpy(rng.exponential(size=(b, hk, keep + 1))).float().cuda()
    for captured in (False, True):
        kv = ra.ra_paged_plan(b * width, pr, hq, hk, d, dtype=dtype)
        cache, weight = start.clone(), heavy.clone()
        table, offset = _i32(np.arange(b * width).reshape(b, width)[:, ::-1].copy()), _i32([0, 1, 2])
        length, position = _i32(lengths), _i32([5000, 70000])
        x = [torch.zeros_like(t[0]) for t in (q, k, v)]
        kept, left = torch.zeros((b, hk, keep), dtype=torch.int32, device="cuda"), _i32([0, 0])
        out = {}

        def step():
            length.add_(1)
            turned = ra.ra_paged_append(kv, cache, x[1], x[2], table, offset, length, rope=rope, position=position, q=x[0])
            out["o"], out["lse"] = ra.ra_paged_attend(kv, cache, turned, table, offset, length)
            ra.ra_paged_weigh(kv, cache, turned, out["lse"], table, offset, length, weight, weight_in=weight)
            ra.ra_paged_evict(kv, cache, table, length, weight, keep, first=2, recent=7, kept=kept, new_length=left)
            length.copy_(left)
            position.add_(1)

        if captured:
            torch.cuda.synchronize()
            graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
            with torch.cuda.graph(graph):
                step()
        seen = []
        for i in range(steps):
            for t, new in zip(x, (q, k, v)):
                t.copy_(new[i])
            if captured:
                side.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(side):
                    graph.replay()
                torch.cuda.current_stream().wait_stream(side)
            else:
                step()
            seen.append([out["o"].clone(), out["lse"].clone(), kept.clone(), length.clone()])
        ra.ra_paged_sync_status(kv)
        seen.append([cache, weight])
        runs.append(seen)
    assert list(runs[0][-2][3].cpu()) == [keep, keep]
    for one, two in zip(*runs):
        for x, y in zip(one, two):
            assert _same_bits(x, y) if x.dtype != torch.int32 else torch.equal(x, y)


# ----------------------------------------------------------------------- weights --
@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hk", HEADS)
@pytest.mark.parametrize("counts,lengths", BATCHES + [([200, 1, 77], [900, 2000, 77])], ids=str)
def test_weights(dtype, d, hq, hk, counts, lengths):
    rng = np.random.default_rng(hq + sum(counts))
    t = Batch(rng, counts, lengths, hq, hk, d, dtype, 48, lead=1, tail=2)
    _, lse = t.attend()
    width = max(lengths) + 5
    before = torch.from_numpy(rng.exponential(size=(len(counts), hk, width))).float()
    weight = torch.full((len(counts), hk, width), 7.0, device="cuda")
    assert ra.ra_paged_weigh(t.kv, t.cache, t.q.cuda(), lse, t.table, t.offset, t.length, weight, weight_in=before.cuda()) is weight
    t.check_weigh(weight.cpu(), before, lse)
    for b, n in enumerate(lengths):
        assert (weight[b, :, n:] == 7).all()
    same = before.cuda()  # in place
    ra.ra_paged_weigh(t.kv, t.cache, t.q.cuda(), lse, t.table, t.offset, t.length, same, weight_in=same)
    fresh = torch.zeros_like(weight)
    ra.ra_paged_weigh(t.kv, t.cache, t.q.cuda(), lse, t.table, t.offset, t.length, fresh)
    t.check_weigh(fresh.cpu(), torch.zeros_like(before), lse)
    for b, n in enumerate(lengths):
        assert _same_bits(same[b, :, :n], weight[b, :, :n])
        # all of a row's weight is given out once
        total = fresh[b, :, :n].double().sum(-1).cpu()
        want = counts[b] * hq / hk
        assert (total - want).abs().max() <= want * (2.0 ** -14 * 40) + 1e-9


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [2.0 ** -100, 2.0 ** -7, 0.3, 3.0])
@pytest.mark.parametrize("counts,lengths,hq,hk", [([1, 2], [700, 90], 6, 2), ([150, 90], [700, 90], 6, 2), ([150, 1], [700, 90], 4, 1)])
def test_scales(dtype, scale, counts, lengths, hq, hk):
    """Scales from the smallest one, at which all weights are alike, groups that leave rows of a query tile empty."""
    t = Batch(np.random.default_rng(3), counts, lengths, hq, hk, 128, dtype, 32, scale=scale)
    o, lse = t.attend()
    t.check_attend(o, lse)
    before = torch.rand((2, hk, 700))
    weight = before.cuda()
    ra.ra_paged_weigh(t.kv, t.cache, t.q.cuda(), lse, t.table, t.offset, t.length, weight, weight_in=weight)
    t.check_weigh(weight.cpu(), before, lse)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 3), (100, 4), (129, 200), (1 << 40, 0)])
@pytest.mark.parametrize("counts", [[1, 1, 1, 1], [5, 3, 70, 16], [300, 1, 2, 0]], ids=str)
def test_windowed_weights(dtype, window, sinks, counts):
    rng = np.random.default_rng(window % 1000 + counts[0])
    t = Batch(rng, counts, [700, 3, 129, 16], 6, 2, 128, dtype, 32, window=window, sinks=sinks)
    _, lse = t.attend()
    before = torch.rand((4, 2, 700))
    weight = torch.zeros((4, 2, 700), device="cuda")
    ra.ra_paged_weigh(t.kv, t.cache, t.q.cuda(), lse, t.table, t.offset, t.length, weight, weight_in=before.cuda())
    t.check_weigh(weight.cpu(), before, lse)


@gpu
def test_weights_of_fewer_slots_are_reported():
    t = Batch(np.random.default_rng(1), [3], [100], 4, 2, 64, "bf16", 32)
    _, lse = t.attend()
    wide = torch.full((1, 2, 100), 7.0, device="cuda")
    ra.ra_paged_weigh(t.kv, t.cache, t.q.cuda(), lse, t.table, t.offset, t.length, wide)
    ra.ra_paged_sync_status(t.kv)
    some = torch.full((1, 2, 60), 7.0, device="cuda")
    ra.ra_paged_weigh(t.kv, t.cache, t.q.cuda(), lse, t.table, t.offset, t.length, some)
    with pytest.raises(ra.RaError):
        ra.ra_paged_sync_status(t.kv)
    assert _same_bits(some, wide[:, :, :60])


# ---------------------------------------------------------------------- eviction --
def _weights(rng, b, hk, width, kind):
    if kind == "ties":
        return torch.from_numpy(rng.integers(0, 4, (b, hk, width)) * 0.25).float()
    w = torch.from_numpy(rng.exponential(size=(b, hk, width)) * np.exp(4 * rng.normal(size=(b, hk, width)))).float()
    if kind == "odd":
        special = torch.tensor([math.nan, math.inf, -math.inf, -0.0, 0.0, -1.0, 1e-45, 3e38])
        pick = torch.from_numpy(rng.integers(0, 16, w.shape))
        w = torch.where(pick < 8, special[pick.clamp(max=7)], w)
    return w


@gpu
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 64), ("f32", 128)])
@pytest.mark.parametrize("kind", ["plain", "ties", "odd"])
@pytest.mark.parametrize("lengths,keep,first,recent", [
    ([1], 1, 0, 0), ([5, 0, 3], 2, 1, 1), ([300, 100, 101, 250], 100, 4, 30), ([2500, 1300], 1200, 0, 0), ([700], 699, 3, 3),
    ([640, 64], 64, 64, 0), ([640, 65], 64, 0, 64), ([90, 50], 200, 4, 8), ([1111], 1, 0, 0)])
@pytest.mark.parametrize("place", ["same", "copy", "other"])
def test_eviction(dtype, d, kind, lengths, keep, first, recent, place):
    """What stays, slot by slot; its rows and weights moved bit for bit; everything else untouched.
    In place, by an equal table, and into other pages."""
    rng = np.random.default_rng(keep + len(lengths))
    hk, pr, b = 3, 32, len(lengths)
    spare = sum(-(-min(n, keep) // pr) for n in lengths) + 1
    ref = paged_ref.Cache(rng, lengths, pr, hk, d, dtype, spare=spare)
    kv = ra.ra_paged_plan(ref.pages, pr, hk, hk, d, dtype=dtype)
    cache, table = ref.data.cuda(), _i32(ref.table)
    weight = _weights(rng, b, hk, max(lengths) + 3, kind)
    new = ref.table.copy()
    if place == "other":
        new, at = np.full((b, -(-keep // pr)), -7), 0
        for i, n in enumerate(lengths):
            used = -(-min(n, keep) // pr)
            new[i, :used] = ref.free[at:at + used]
            at += used
    out = torch.full(weight.shape, 7.0, device="cuda") if place == "other" else weight.cuda()
    kept, new_length = ra.ra_paged_evict(kv, cache, table, _i32(lengths), weight.cuda() if place == "other" else out, keep,
                                         first=first, recent=recent, new_table=None if place == "same" else _i32(new),
                                         weight_out=out)
    ra.ra_paged_sync_status(kv)
    assert kept.shape == (b, hk, keep) and list(new_length.cpu()) == [min(n, keep) for n in lengths]
    want, w_out = ref.data.clone(), torch.full(weight.shape, 7.0) if place == "other" else weight.clone()
    for i, n in enumerate(lengths):
        for h in range(hk):
            stay = paged_ref.evict(weight[i, h].numpy(), n, keep, first, recent)
            m = len(stay)
            assert np.array_equal(kept[i, h, :m].cpu().numpy(), stay) and (kept[i, h, m:] == -1).all()
            w_out[i, h, :m] = weight[i, h, stay]
            page, row = ref.place(i, stay)
            to = np.arange(m)
            to_page = torch.from_numpy(new[i][to // pr].astype(np.int64)) if m else page
            want[to_page, :, h, torch.from_numpy(to % pr)] = ref.data[page, :, h, row]
    assert _same_bits(cache, want)
    assert _same_bits(out, w_out)


@gpu
@pytest.mark.parametrize("n,keep", [(60000, 20000), (60000, 59999), (49153, 100)])
def test_long_eviction(n, keep):
    """More slots than the weights that one CTA keeps by it; in place."""
    rng = np.random.default_rng(n)
    kv = ra.ra_paged_plan(240, 256, 1, 1, 64)
    cache = torch.randn((240, 2, 1, 256, 64), device="cuda").bfloat16()
    table = torch.randperm(240)[None].int().cuda()
    weight = torch.from_numpy(rng.integers(0, 5000, (1, 1, n))).float()
    before, w = cache.clone(), weight.cuda()
    kept, new_length = ra.ra_paged_evict(kv, cache, table, _i32([n]), w, keep, first=7, recent=50)
    ra.ra_paged_sync_status(kv)
    stay = torch.from_numpy(paged_ref.evict(weight[0, 0].numpy(), n, keep, 7, 50))
    assert torch.equal(kept[0, 0].cpu().long(), stay) and int(new_length) == keep
    assert torch.equal(w[0, 0, :keep].cpu(), weight[0, 0, stay])
    flat = lambda x, s: x[table[0].cpu().long()[s // 256].cuda(), :, 0, (s % 256).cuda()]
    assert _same_bits(flat(cache, torch.arange(keep)), flat(before, stay))


@gpu
def test_refused_evictions_are_reported():
    """Lengths beyond the table or the weights, places that are too few, pages that are none."""
    rng = np.random.default_rng(3)
    ref = paged_ref.Cache(rng, [100, 90], 16, 2, 64, "bf16")
    kv = ra.ra_paged_plan(ref.pages, 16, 2, 2, 64)
    cache, table, weight = ref.data.cuda(), _i32(ref.table), torch.rand((2, 2, 100)).cuda()

    def run(lengths, keep, **kw):
        w = kw.pop("weight", weight)
        out = ra.ra_paged_evict(kv, cache, kw.pop("table", table), _i32(lengths), w, keep, weight_out=torch.zeros_like(w), **kw)
        with pytest.raises(ra.RaError) as err:
            ra.ra_paged_sync_status(kv)
        assert err.value.name == "RA_ERR_INVALID_ARG"
        ra.ra_paged_sync_status(kv)
        return out

    for lengths, kw in (([-1, 60], {}), ([ref.width * 16 + 1, 60], {}), ([90, 60], dict(weight=weight[:, :, :70].contiguous())),
                        ([90, 40], dict(new_table=table[:, :3].contiguous()))):
        kept, n = run(lengths, 60, **kw)
        assert list(n.cpu()) == [0, min(lengths[1], 60)] and (kept[0] == -1).all() and (kept[1, :, :lengths[1]] >= 0).all()
        for i in (0, 1):
            assert _same_bits(cache[torch.from_numpy(ref.table[i, :6])], ref.data[torch.from_numpy(ref.table[i, :6])]) or i == 1
    cache.copy_(ref.data)
    bad = ref.table.copy()
    bad[0, 5] = -1  # rows 80..95 cannot be read
    kept, _ = run([100, 90], 100, table=_i32(bad), new_table=table)
    assert _same_bits(cache, ref.data)
    for kw in (dict(keep=0), dict(keep=4, first=3, recent=2), dict(keep=4, first=-1)):
        with pytest.raises(ra.RaError):
            ra.ra_paged_evict(kv, cache, table, _i32([100, 90]), weight, **kw)


# -------------------------------------------------------------------- all together --
@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_sequence_from_the_ring_through_the_cache(dtype):
    """A prompt's attention by the ring and, chunk by chunk, over the cache; then eviction and
    tokens after it, whose attention is that over the slots that stayed."""
    rng = np.random.default_rng(17)
    d, hq, hk, s, pr, chunk = 128, 4, 2, 384, 32, 130
    rope = ra.ra_rope_plan(d, base=1000.0, dtype=dtype)
    x = [torch.from_numpy(rng.normal(size=(s, h, d))).to(DT[dtype]).cuda() for h in (hq, hk, hk)]
    # the ring, on two zigzag shards
    plan = ra.ra_plan(1, s, hq, hk, d, 2, layout="zigzag", causal=True, dtype=dtype)
    order = torch.from_numpy(np.asarray(ra.ra_layout_index("zigzag", s, 2)).astype(np.int64)).cuda()
    q, k, v = (t[order].transpose(0, 1)[None] for t in x)
    q, k = ra.ra_rope(rope, q, k, layout="zigzag", n_shards=2)
    ring_o, ring_lse = ra.ra_fwd(plan, q, k, v.contiguous())
    ra.ra_sync_status(plan)
    # the cache, chunk by chunk, beside another sequence of single tokens
    kv = ra.ra_paged_plan(40, pr, hq, hk, d, dtype=dtype)
    cache = torch.full(ra.ra_paged_cache_shape(kv), math.nan, dtype=DT[dtype], device="cuda")
    table = torch.from_numpy(rng.permutation(40)[:30].reshape(2, 15)).int().cuda()
    weight = torch.zeros((2, hk, 480), device="cuda")
    other = [torch.from_numpy(rng.normal(size=(3, h, d))).to(DT[dtype]).cuda() for h in (hq, hk, hk)]
    o, lse, done, step = [], [], 0, 0
    while done < s:
        n = min(chunk, s - done)
        qc, kc, vc = (torch.cat([a[done:done + n], b[step:step + 1]]) for a, b in zip(x, other))
        offset, length = _i32([0, n, n + 1]), _i32([done + n, step + 1])
        qr = ra.ra_paged_append(kv, cache, kc, vc, table, offset, length, rope=rope, q=qc)
        oc, lc = ra.ra_paged_attend(kv, cache, qr, table, offset, length)
        ra.ra_paged_weigh(kv, cache, qr, lc, table, offset, length, weight, weight_in=weight)
        o.append(oc[:n]), lse.append(lc[:n])
        done, step = done + n, step + 1
    ra.ra_paged_sync_status(kv)
    o, lse = torch.cat(o)[order], torch.cat(lse)[order]
    tol = 2.0 ** -6 if dtype == "bf16" else 2.0 ** -17  # two results, each within half of it of the exact one
    assert (o.float() - ring_o[0].transpose(0, 1).float()).abs().max() <= tol * ring_o.float().abs().max()
    # (the ring's bf16 kernel adds every tile's largest weight to the sum as rounded to bf16: these weights are
    # off by at most half a step, 2^-8 of themselves, and so is a sum of which they are a part; its logarithm
    # moves by as much, beside 1e-4 for both results' float32 errors)
    assert (lse - ring_lse[0].transpose(0, 1)).abs().max() <= 1e-4 + (2.0 ** -8 if dtype == "bf16" else 0.0)
    # all weight was given out: every row of the group once
    assert torch.allclose(weight[0, :, :s].sum(-1), torch.full((hk,), float(s * hq // hk), device="cuda"), rtol=1e-4)
    # the cache cut to 200 slots, then four more tokens at their own positions
    before, keep = cache.clone(), 200
    kept, new_length = ra.ra_paged_evict(kv, cache, table, _i32([s, 3]), weight, keep, first=4, recent=64)
    more = [torch.from_numpy(rng.normal(size=(4, h, d))).to(DT[dtype]).cuda() for h in (hq, hk, hk)]
    pos = torch.arange(s, s + 4, dtype=torch.int32, device="cuda")
    offset, length = _i32([0, 4, 4]), new_length + _i32([4, 0])
    qr = ra.ra_paged_append(kv, cache, more[1], more[2], table, offset, length, rope=rope, q=more[0], position=pos)
    oc, lc = ra.ra_paged_attend(kv, cache, qr, table, offset, length)
    ra.ra_paged_sync_status(kv)
    kr = ra.ra_rope(rope, more[1].transpose(0, 1)[None], position=pos[None])[0]
    page = table[0].cpu().long()
    for h in range(hk):
        stay = kept[0, h].cpu().long()
        rows = [torch.cat([before[page[stay // pr].cuda(), w, h, (stay % pr).cuda()], t]).cpu().double()[None]
                for w, t in ((0, kr[h]), (1, more[2][:, h]))]
        g = hq // hk
        ow, lw, ob, lb = paged_ref.attend(*rows, qr[:, h * g:(h + 1) * g].cpu(), torch.arange(keep, keep + 4), torch.arange(keep + 4),
                                          0, 0, U[dtype])
        assert_within(oc[:, h * g:(h + 1) * g].cpu(), ow, ob, "O")
        assert_within(lc[:, h * g:(h + 1) * g].cpu(), lw, lb, "LSE")


# --------------------------------------------------------------------- debug build --
def test_addresses_are_checked():
    """The kernels of the paged cache check what they read and write, at sites of their own."""
    import re
    csrc = os.path.join(ROOT, "context_ring_attention_gb300", "csrc")
    sites, kernels = {}, []
    for name in sorted(os.listdir(csrc)):
        if name.endswith(".cu"):
            with open(os.path.join(csrc, name)) as f:
                text = f.read()
            sites[name] = [int(x) for x in re.findall(r"RA_BOUNDS\(.*?,\s*(\d+)\);", text, re.S)]
            kernels += [name] * ("__global__" in text)
    for name in kernels:
        if name.startswith("paged_"):
            assert sites[name], name
            others = {x for other, v in sites.items() if other != name for x in v}
            assert not others & set(sites[name]) and max(sites[name]) < 256


def paged_outputs():
    """Every call on ragged batches, for each type and head size."""
    out, rng = {}, np.random.default_rng(41)
    for n, (dtype, d, counts, lengths, hq, hk, window, sinks) in enumerate([
            ("bf16", 128, [1], [1900], 4, 1, 0, 0), ("bf16", 64, [3, 0, 33], [70, 5, 33], 6, 2, 20, 3),
            ("f32", 128, [9, 1, 1], [300, 16, 1], 3, 3, 0, 0), ("bf16", 128, [300, 1, 5], [2300, 1801, 40], 16, 2, 1500, 20),
            ("bf16", 64, [700, 129], [700, 2000], 4, 2, 0, 0), ("f32", 64, [1, 40], [1700, 40], 4, 2, 0, 0),
            ("f32", 128, [300], [613], 4, 1, 0, 0), ("bf16", 128, [20], [9000], 8, 1, 0, 0)]):
        t = Batch(rng, counts, lengths, hq, hk, d, dtype, 48, window=window, sinks=sinks)
        rope = ra.ra_rope_plan(d, d // 2, dtype=dtype)
        k, v = t.random(t.tokens, hk).cuda(), t.random(t.tokens, hk).cuda()
        q = ra.ra_paged_append(t.kv, t.cache, k, v, t.table, t.offset, t.length, rope=rope, q=t.q.cuda())
        o, lse = ra.ra_paged_attend(t.kv, t.cache, q, t.table, t.offset, t.length)
        w = torch.zeros((len(counts), hk, max(lengths)), device="cuda")
        ra.ra_paged_weigh(t.kv, t.cache, q, lse, t.table, t.offset, t.length, w)
        weighed = w.clone()
        kept, m = ra.ra_paged_evict(t.kv, t.cache, t.table, t.length, w, max(lengths) // 2, first=1, recent=2)
        ra.ra_paged_sync_status(t.kv)
        for name, x in dict(q=q, o=o, l=lse, w=weighed, k=kept, m=m, c=t.cache.nan_to_num(9.0)).items():
            out[f"{n}/{name}"] = x.float().cpu().numpy()
    return out


@gpu
def test_debug_library_passes_its_bounds_checks(tmp_path):
    path = str(tmp_path / "out.npz")
    code = "import numpy as np, sys; from tests import test_gpu_paged as t; np.savez(sys.argv[1], **t.paged_outputs())"
    res = subprocess.run([sys.executable, "-c", code, path], cwd=ROOT, env=dict(os.environ, RA_LIBRARY_VARIANT="debug"),
                         capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr[-2000:]
    here = paged_outputs()
    with np.load(path) as debug:
        assert set(debug.files) == set(here)
        for name, a in here.items():
            assert np.array_equal(a, debug[name]), name
