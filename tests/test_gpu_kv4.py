"""GPU tests of the 4-bit cache: bytes written, values read back, attention over it, and a
sequence continued from a windowed prompt, against the plain form in kv4_ref.py."""

import math
from fractions import Fraction

import numpy as np
import pytest

torch = pytest.importorskip("torch")
ra = pytest.importorskip("context_ring_attention_gb300")
from tests import kv4_ref, window_ref  # noqa: E402
from tests.window_ref import assert_within  # noqa: E402

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ra.load_library()


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _dev(x, dtype):
    return torch.from_numpy(np.asarray(x, np.float64)).to(DT[dtype]).cuda()


def _rows(rng, b, h, t, d, dtype):
    """Rows with channels of different sizes and offsets, as the dtype holds them (float64)."""
    x = rng.normal(size=(b, h, t, d)) * np.exp(0.5 * rng.normal(size=d)) + rng.normal(size=d)
    return torch.from_numpy(x).to(DT[dtype]).double().numpy()


def _filled(rng, lengths, page_rows, hk, d, dtype, heads_q=None, spare=2, fill=0xFF, **kw):
    """A device cache with lengths[b] tokens of every sequence on scattered pages, its
    reference, and the page table (its unused entries name a page outside the pool)."""
    width = max(1, max(-(-n // page_rows) for n in lengths) + 1)
    need = sum(-(-n // page_rows) for n in lengths)
    pages = need + spare
    order = rng.permutation(pages)
    table = np.full((len(lengths), width), pages + 5)
    at = 0
    for b, n in enumerate(lengths):
        used = -(-n // page_rows)
        table[b, :used] = order[at:at + used]
        at += used
    kv = ra.ra_kv4_plan(pages, page_rows, heads_q or hk, hk, d, dtype=dtype, **kw)
    ref = kv4_ref.Cache(pages, page_rows, hk, d, fill)
    t = max(1, max(lengths))
    k, v = _rows(rng, len(lengths), hk, t, d, dtype), _rows(rng, len(lengths), hk, t, d, dtype)
    ref.write(k, v, table, np.zeros(len(lengths), int), lengths)
    cache = torch.full((ra.ra_kv4_cache_size(kv),), fill, dtype=torch.uint8, device="cuda")
    ra.ra_kv4_write(kv, cache, _dev(k, dtype), _dev(v, dtype), _i32(table), _i32([0] * len(lengths)), _i32(lengths))
    ra.ra_kv4_sync_status(kv)
    return kv, cache, ref, table


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hk,page_rows", [(1, 16), (3, 112), (8, 64)])
def test_written_bytes(dtype, d, hk, page_rows):
    """Every byte: codes and parameters of the written rows, and all others untouched."""
    rng = np.random.default_rng(d + hk)
    pages, b, t = 9, 3, 41
    kv = ra.ra_kv4_plan(pages, page_rows, hk, hk, d, dtype=dtype)
    ref = kv4_ref.Cache(pages, page_rows, hk, d)
    table = rng.permutation(pages)[:9].reshape(3, 3)
    if page_rows == 16:
        table = np.concatenate([table, table], 1)[:, :3]
    cache = torch.full((ra.ra_kv4_cache_size(kv),), 0xAB, dtype=torch.uint8, device="cuda")
    for first, count in (([0, 5, 6], [0, 41, 7]), ([3, 0, 0], [1, 1, 40]), ([7, 6, 7], [41, 41, 41])):
        first = [min(f, 3 * page_rows - 41) for f in first]
        k, v = _rows(rng, b, hk, t, d, dtype), _rows(rng, b, hk, t, d, dtype)
        ref.write(k, v, table, first, count)
        whole = min(count) == t
        ra.ra_kv4_write(kv, cache, _dev(k, dtype), _dev(v, dtype), _i32(table), _i32(first), None if whole else _i32(count))
    ra.ra_kv4_sync_status(kv)
    assert np.array_equal(cache.cpu().numpy().reshape(ref.bytes.shape), ref.bytes)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_difficult_groups(dtype, d):
    """Constant groups, borders of two codes hit exactly, one far value, tiny and huge
    ranges, infinities and NaN, signed zeros."""
    rng = np.random.default_rng(7)
    rows = [np.full(d, 3.25), np.full(d, -1.0 / 3), np.zeros(d), np.where(np.arange(d) % 2, 0.0, -0.0),
            np.arange(d) % 32 / 2.0, (np.arange(d) % 32 - 16) / 2.0 + 0.25,      # ties at every half step
            np.arange(d) % 31 * 0.5 - 7, np.where(np.arange(d) == 5, 1e4, rng.normal(size=d)),
            rng.normal(size=d) * 1e-30, rng.normal(size=d) * 1e-38, rng.normal(size=d) * 1e30,
            np.where(np.arange(d) % 32 == 3, 3e38, -3e38), np.where(np.arange(d) == 40, np.inf, 1.0),
            np.where(np.arange(d) == 2, -np.inf, 1.0), np.where(np.arange(d) == 33, np.nan, rng.normal(size=d)),
            rng.normal(size=d) + 1000, rng.normal(size=d) * 1e-3 + 1]
    x = np.stack(rows)[None, None]
    x = torch.from_numpy(x).to(DT[dtype]).double().numpy()
    t = x.shape[2]
    kv = ra.ra_kv4_plan(2, 32, 1, 1, d, dtype=dtype)
    ref = kv4_ref.Cache(2, 32, 1, d)
    ref.write(x, x, [[1]], [0], [t])
    cache = torch.full((ra.ra_kv4_cache_size(kv),), 0xAB, dtype=torch.uint8, device="cuda")
    ra.ra_kv4_write(kv, cache, _dev(x, dtype), _dev(x, dtype), _i32([[1]]), _i32([0]))
    assert np.array_equal(cache.cpu().numpy().reshape(ref.bytes.shape), ref.bytes)
    for got, want in zip(ra.ra_kv4_read(kv, cache, _i32([[1]]), _i32([0]), t), (ref.k, ref.v)):
        want = torch.from_numpy(want[1, :, :t])[None]
        got = got.double().cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        fin = ~torch.isnan(want)
        assert ((got - want).abs()[fin] <= kv4_ref.U[dtype] * 1.001 * want.abs()[fin] + 1e-45).all()
    ra.ra_kv4_sync_status(kv)


def test_float32_codes_next_to_borders():
    """float32 values one place on either side of every border of two codes."""
    step = np.float32(0.37)
    x = np.zeros((1, 1, 31, 64), np.float32)
    for t in range(30):
        border = np.float32(bf := float(kv4_ref.bf16(np.float64(15 * step) / 15)) * (t // 2 + 0.5))
        x[0, 0, t, :32] = np.linspace(0, 15 * step, 32, dtype=np.float32)
        x[0, 0, t, 5] = np.nextafter(border, np.float32(100 if t % 2 else -100))
        x[0, 0, t, 6] = border
        x[0, 0, t, 32:] = x[0, 0, t, :32] - np.float32(1000.0)
    kv = ra.ra_kv4_plan(2, 32, 1, 1, 64, dtype="f32")
    ref = kv4_ref.Cache(2, 32, 1, 64)
    ref.write(x.astype(np.float64), x.astype(np.float64), [[0]], [0], [31])
    cache = torch.full((ra.ra_kv4_cache_size(kv),), 0xAB, dtype=torch.uint8, device="cuda")
    ra.ra_kv4_write(kv, cache, torch.from_numpy(x).cuda(), torch.from_numpy(x).cuda(), _i32([[0]]), _i32([0]))
    ra.ra_kv4_sync_status(kv)
    assert np.array_equal(cache.cpu().numpy().reshape(ref.bytes.shape), ref.bytes)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_minima_far_below_the_values(dtype, d):
    """Values on the border of two codes above a minimum so small that x - low rounds to x: the
    quotient lies below the border for a positive minimum, and above it for a negative one."""
    rows = []
    for scale in (1.0, 0.75, 129 / 128 * 2.0 ** 40, 2.0 ** -60):
        for e in (-16, -18, -20, -23, -24, -25, -30, -45, -126):
            for sign in (1, -1):
                g = np.full(32, sign * 1.5 * 2.0 ** e * (scale if e > -126 else 1))
                g[1:16] = (np.arange(15) + 0.5) * scale  # borders (those that the dtype holds)
                g[16:31] = np.arange(1, 16) * scale
                rows.append(np.tile(g, d // 32))
    x = torch.from_numpy(np.stack(rows)[None, None]).to(DT[dtype]).double().numpy()
    t = x.shape[2]
    kv = ra.ra_kv4_plan(1, 80, 1, 1, d, dtype=dtype)
    cache = torch.full((ra.ra_kv4_cache_size(kv),), 0xAB, dtype=torch.uint8, device="cuda")
    ra.ra_kv4_write(kv, cache, _dev(x, dtype), _dev(x, dtype), _i32([[0]]), _i32([0]))
    got = ra.ra_kv4_read(kv, cache, _i32([[0]]), _i32([0]), t)
    ra.ra_kv4_sync_status(kv)
    _, scale, low = kv4_ref.quantise(x)  # (the parameters; a difference in 64 bits may round as well)
    exact = np.empty(x.shape, np.int64)
    for at in np.ndindex(x.shape):
        s, l = (Fraction(float(p[at[:-1] + (at[-1] // 32,)])) for p in (scale, low))
        exact[at] = min(max(math.floor((Fraction(float(x[at])) - l) / s + Fraction(1, 2)), 0), 15)
    for values in got:  # a value is nearest to its own code, whatever the dtype's rounding
        codes = (values.double().cpu().numpy() - np.repeat(low, 32, -1)) / np.repeat(scale, 32, -1)
        assert np.array_equal(np.rint(codes), exact)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_read_back(dtype, d):
    rng = np.random.default_rng(d)
    kv, cache, ref, table = _filled(rng, [70, 1, 33], 48, 2, d, dtype)
    first, count, rows = [11, 0, 30], [59, 1, 0], 60
    k, v = (torch.full((3, 2, rows, d), 7.0, dtype=DT[dtype], device="cuda") for _ in range(2))
    assert ra.ra_kv4_read(kv, cache, _i32(table), _i32(first), rows, _i32(count), k=k, v=v)[0] is k
    ra.ra_kv4_sync_status(kv)
    for b in range(3):
        assert (k[b, :, count[b]:] == 7).all() and (v[b, :, count[b]:] == 7).all()  # left as they were
        if count[b]:
            want = ref.rows(table[b], np.arange(first[b], first[b] + count[b]))
            for got, w in zip((k, v), want):
                w = torch.from_numpy(w)
                # one rounding of the dtype, after a float32 one
                bound = (kv4_ref.U[dtype] + 2.0 ** -23) * w.abs()
                assert_within(got[b, :, :count[b]].cpu(), w, bound, "value")
    # outputs of the call's own: zeros there
    k2, v2 = ra.ra_kv4_read(kv, cache, _i32(table), _i32(first), rows, _i32(count))
    for b in range(3):
        assert torch.equal(k2[b, :, :count[b]], k[b, :, :count[b]])
        assert (k2[b, :, count[b]:] == 0).all() and (v2[b, :, count[b]:] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_values_are_float32_sums(dtype):
    """low + scale * code is a float32 number first: where it lies a hair from the middle of two
    bf16 numbers (a minimum of -2^-40, 3 * 129/128), the second rounding starts from the middle."""
    x = np.zeros((1, 1, 1, 64))
    x[..., :32] = np.linspace(0, 15.125, 32)
    x[..., 0], x[..., 31] = -2.0 ** -40, 15.125
    x[..., 32:] = -x[..., :32]
    x = torch.from_numpy(x).to(DT[dtype]).double().numpy()
    codes, scale, low = kv4_ref.quantise(x)
    assert scale[0, 0, 0, 0] == 129 / 128 and 3 in codes[0, 0, 0, :32]
    want = (np.repeat(low, 32, -1) + np.repeat(scale, 32, -1) * codes).astype(np.float32)  # (exact in 64 bits)
    kv = ra.ra_kv4_plan(1, 16, 1, 1, 64, dtype=dtype)
    cache = torch.zeros(ra.ra_kv4_cache_size(kv), dtype=torch.uint8, device="cuda")
    ra.ra_kv4_write(kv, cache, _dev(x, dtype), _dev(x, dtype), _i32([[0]]), _i32([0]))
    for got in ra.ra_kv4_read(kv, cache, _i32([[0]]), _i32([0]), 1):
        assert torch.equal(got.cpu(), torch.from_numpy(want).to(DT[dtype]))
    ra.ra_kv4_sync_status(kv)


def _check_attend(kv, cache, ref, table, lengths, hq, t, d, dtype, window, sinks, rng, **kw):
    q = _rows(rng, len(lengths), hq, t, d, dtype) * 0.7
    q = torch.from_numpy(q).to(DT[dtype])
    o, lse = ra.ra_kv4_attend(kv, cache, q.cuda(), _i32(table), _i32(lengths), **kw)
    ra.ra_kv4_sync_status(kv)
    for b, n in enumerate(lengths):
        k, v = ref.rows(table[b], np.arange(n))
        ow, lw, ob, lb = kv4_ref.attend(k, v, q[b].double().numpy(), n, window, sinks, kv4_ref.U[dtype])
        assert_within(lse[b].cpu(), lw, lb, f"LSE of sequence {b}")
        assert_within(o[b].cpu(), ow, ob, f"O of sequence {b}")
    return q, o, lse


LENGTHS = [[0], [1], [15, 16, 17], [300, 0, 31, 128, 1], [1000, 2]]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lengths", LENGTHS, ids=str)
@pytest.mark.parametrize("t,hq,hk", [(1, 4, 1), (1, 24, 8), (3, 6, 2), (5, 16, 2), (16, 3, 3)])
def test_attention(dtype, d, lengths, t, hq, hk):
    """From no token to several splits, fewer tokens than queries, group sizes and tokens
    that fill no 8-row tile.  Unwritten places hold bytes that read as NaN."""
    rng = np.random.default_rng(len(lengths) + t)
    kv, cache, ref, table = _filled(rng, lengths, 48, hk, d, dtype, heads_q=hq)
    _check_attend(kv, cache, ref, table, lengths, hq, t, d, dtype, 0, 0, rng)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 3), (16, 16), (100, 4), (129, 200), (5000, 0), (1 << 40, 1 << 40)])
@pytest.mark.parametrize("t", [1, 4])
def test_windowed_attention(dtype, window, sinks, t):
    rng = np.random.default_rng(window % 1000 + t)
    lengths = [700, 3, 129, 16]
    kv, cache, ref, table = _filled(rng, lengths, 32, 2, 128, dtype, heads_q=6, window=window, sinks=sinks)
    _check_attend(kv, cache, ref, table, lengths, 6, t, 128, dtype, window, sinks, rng)


def test_unseen_rows_may_hold_anything():
    """NaN groups, and codes of any kind, outside the window and beyond the length."""
    rng = np.random.default_rng(5)
    lengths, window, sinks = [200, 90], 33, 4
    kv, cache, ref, table = _filled(rng, lengths, 16, 2, 128, "bf16", heads_q=4, window=window, sinks=sinks)
    q, o, lse = _check_attend(kv, cache, ref, table, lengths, 4, 2, 128, "bf16", window, sinks, rng)
    bad = torch.full((2, 2, 200, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    ra.ra_kv4_write(kv, cache, bad, bad, _i32(table), _i32([sinks, sinks]),
                    _i32([n - 1 - window - sinks for n in lengths]))  # up to the first query's window
    o2, lse2 = ra.ra_kv4_attend(kv, cache, q.cuda(), _i32(table), _i32(lengths))
    ra.ra_kv4_sync_status(kv)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    # a NaN that is seen comes through
    ra.ra_kv4_write(kv, cache, bad[:, :, :1].contiguous(), bad[:, :, :1].contiguous(), _i32(table), _i32([150, 80]))
    o3, _ = ra.ra_kv4_attend(kv, cache, q.cuda(), _i32(table), _i32(lengths))
    assert torch.isnan(o3[0]).any() or torch.isnan(o3[1]).any()
    assert torch.isnan(o3[1]).all()


def test_shared_pages_and_own_outputs():
    """Two sequences with a common first page; caller's o, lse and scratch."""
    rng = np.random.default_rng(9)
    lengths = [900, 640]
    kv, cache, ref, table = _filled(rng, lengths, 32, 2, 64, "f32", heads_q=8)
    table[1, :3] = table[0, :3]
    table = np.concatenate([table, np.full((2, 60 - table.shape[1]), -1)], 1)  # room for 1920 tokens
    need = ra.ra_kv4_attend_scratch_size(kv, 2, 1, table.shape[1])
    assert need > 0
    scratch = torch.full((need // 4 + 3,), float("nan"), device="cuda")
    o = torch.empty((2, 8, 1, 64), device="cuda")
    lse = torch.empty((2, 8, 1), device="cuda")
    _check_attend(kv, cache, ref, table, lengths, 8, 1, 64, "f32", 0, 0, rng, o=o, lse=lse, scratch=scratch)
    with pytest.raises(ValueError):
        ra.ra_kv4_attend(kv, cache, torch.zeros((2, 8, 1, 64), device="cuda"), _i32(table), _i32(lengths),
                         scratch=scratch[:need // 4 - 1])


def test_out_of_range_tables_are_reported_and_skipped():
    """Pages outside the pool, positions outside the table, counts and lengths out of range:
    nothing out of bounds is touched, the rest of the call is right, the status says so."""
    rng = np.random.default_rng(13)
    lengths = [100, 60]
    kv, cache, ref, table = _filled(rng, lengths, 32, 1, 64, "f32")
    before = cache.clone()
    bad = table.copy()
    bad[0, 1] = 1 << 30
    bad[1, 0] = -1
    x = torch.ones((2, 1, 8, 64), device="cuda")
    q = torch.ones((2, 1, 1, 64), device="cuda")

    def reported():
        with pytest.raises(ra.RaError) as err:
            ra.ra_kv4_sync_status(kv)
        assert err.value.name == "RA_ERR_INVALID_ARG"
        ra.ra_kv4_sync_status(kv)  # cleared

    width = table.shape[1] * 32
    for tab, first, count in ((bad, [32, 0], None), (table, [-5, -1], None), (table, [width, width - 4 + 10 ** 6], None),
                              (table, [0, 0], [9, -1]), (table, [2 ** 31 - 1, 2 ** 31 - 3], None)):
        args = (_i32(tab), _i32(first))
        c = None if count is None else _i32(count)
        ra.ra_kv4_write(kv, cache, x, x, *args, c)
        reported()
        k = torch.full((2, 1, 8, 64), 5.0, device="cuda")
        ra.ra_kv4_read(kv, cache, *args, 8, c, k=k, v=k.clone())
        reported()
        assert (k == 5).all()
        assert torch.equal(cache, before)
    # attention leaves a bad page's keys out: the other pages' remain
    o, lse = ra.ra_kv4_attend(kv, cache, q, _i32(bad), _i32(lengths))
    reported()
    for b, keep in ((0, np.r_[0:32, 64:100]), (1, np.r_[32:60])):
        k, v = ref.rows(table[b], keep)
        ow, lw, ob, lb = kv4_ref.attend(k, v, np.ones((1, 1, 64)), len(keep), 0, 0, kv4_ref.U["f32"])
        assert_within(o[b].cpu(), ow, ob, "O")
        assert_within(lse[b].cpu(), lw, lb, "LSE")
    o, lse = ra.ra_kv4_attend(kv, cache, q, _i32(table), _i32([-1, width + 1]))
    reported()
    assert (o == 0).all() and torch.isneginf(lse).all()


def test_offsets_beyond_32_bits():
    """A pool of 2.7 GB: pages at its end are reached, and only they."""
    pages, page_rows, hk, d = 32768, 64, 8, 128
    kv = ra.ra_kv4_plan(pages, page_rows, hk, hk, d)
    assert ra.ra_kv4_cache_size(kv) > 1 << 31
    cache = torch.zeros(ra.ra_kv4_cache_size(kv), dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(3)
    x = _rows(rng, 1, hk, 70, d, "bf16")
    table = np.array([[pages - 1, pages - 2]])
    ra.ra_kv4_write(kv, cache, _dev(x, "bf16"), _dev(x, "bf16"), _i32(table), _i32([0]))
    k, v = ra.ra_kv4_read(kv, cache, _i32(table), _i32([0]), 70)
    want = torch.from_numpy(kv4_ref.values(x))
    bound = (kv4_ref.U["bf16"] + 2.0 ** -23) * want.abs()
    assert_within(k.cpu(), want, bound, "k")
    assert_within(v.cpu(), want, bound, "v")
    q = _rows(rng, 1, hk, 1, d, "bf16")
    o, _ = ra.ra_kv4_attend(kv, cache, _dev(q, "bf16"), _i32(table), _i32([70]))
    ow, _, ob, _ = kv4_ref.attend(want[0].numpy(), want[0].numpy(), q[0], 70, 0, 0, kv4_ref.U["bf16"])
    assert_within(o[0].cpu(), ow, ob, "O")
    ra.ra_kv4_sync_status(kv)
    assert not cache[:(pages - 2) * hk * page_rows * 160].any()


def test_captured_decoding_step_follows_its_tables():
    """write + attend captured once, replayed as lengths, pages and tokens move on; another
    captured call shares nothing with it; repeated results are the same bits."""
    rng = np.random.default_rng(17)
    b, hk, hq, d, page_rows, steps = 2, 2, 8, 128, 16, 20
    start = [30, 5]
    pages = 12
    table = rng.permutation(pages)[:8].reshape(2, 4)
    kv = ra.ra_kv4_plan(pages, page_rows, hq, hk, d, window=24, sinks=2)
    cache = torch.full((ra.ra_kv4_cache_size(kv),), 0xFF, dtype=torch.uint8, device="cuda")
    hist_k, hist_v = (_rows(rng, b, hk, 60, d, "bf16") for _ in range(2))
    tab = _i32(table)
    ra.ra_kv4_write(kv, cache, _dev(hist_k, "bf16"), _dev(hist_v, "bf16"), tab, _i32([0, 0]), _i32(start))
    k, v, q = (torch.zeros((b, h, 1, d), dtype=torch.bfloat16, device="cuda") for h in (hk, hk, hq))
    first, length = _i32(start), _i32(start) + 1

    def step():
        ra.ra_kv4_write(kv, cache, k, v, tab, first)
        return ra.ra_kv4_attend(kv, cache, q, tab, length)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = step()
    vals_k, vals_v = kv4_ref.values(hist_k), kv4_ref.values(hist_v)
    for s in range(steps):
        at = [n + s for n in start]
        for x, hist in ((k, hist_k), (v, hist_v)):
            x.copy_(_dev(np.stack([hist[i, :, at[i]] for i in range(b)])[:, :, None], "bf16"))
        qs = _rows(rng, b, hq, 1, d, "bf16")
        q.copy_(_dev(qs, "bf16"))
        first.copy_(_i32(at))
        length.copy_(_i32(at) + 1)
        graph.replay()
        ra.ra_kv4_sync_status(kv)
        for i in range(b):
            n = at[i] + 1
            ow, lw, ob, lb = kv4_ref.attend(vals_k[i, :, :n], vals_v[i, :, :n], qs[i], n, 24, 2, kv4_ref.U["bf16"])
            assert_within(o[i].cpu(), ow, ob, f"O at step {s}")
            assert_within(lse[i].cpu(), lw, lb, f"LSE at step {s}")
    keep = o.clone()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, keep)


def test_calls_on_two_streams_at_once():
    rng = np.random.default_rng(19)
    lengths = [900, 333]
    kv, cache, ref, table = _filled(rng, lengths, 32, 2, 128, "bf16", heads_q=8)
    q = [torch.from_numpy(_rows(rng, 2, 8, 2, 128, "bf16")).bfloat16().cuda() for _ in range(2)]
    tab, n = _i32(table), _i32(lengths)
    want = [ra.ra_kv4_attend(kv, cache, x, tab, n) for x in q]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [ra.ra_kv4_attend(kv, cache, x, tab, n, stream=s) for x, s in zip(q, streams)]
        torch.cuda.synchronize()
        for (o, lse), (ow, lw) in zip(got, want):
            assert torch.equal(o, ow) and torch.equal(lse, lw)
    ra.ra_kv4_sync_status(kv)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_then_tokens(dtype):
    """As a serving loop uses them: the prompt's keys and values go into the cache and are
    read back, a windowed plan attends over the values that were read, and the next tokens
    continue from the cache -- every row against one float64 attention over all of it."""
    rng = np.random.default_rng(23)
    b, hq, hk, d, n_prompt, n_new, window, sinks, page_rows = 2, 4, 2, 128, 150, 10, 40, 3, 32
    total = n_prompt + n_new
    k, v = (_rows(rng, b, hk, total, d, dtype) for _ in range(2))
    q = _rows(rng, b, hq, total, d, dtype)
    width = -(-total // page_rows)
    table = rng.permutation(b * width + 1)[:b * width].reshape(b, width)
    kv = ra.ra_kv4_plan(b * width + 1, page_rows, hq, hk, d, dtype=dtype, window=window, sinks=sinks)
    cache = torch.full((ra.ra_kv4_cache_size(kv),), 0xFF, dtype=torch.uint8, device="cuda")
    tab, zero = _i32(table), _i32([0] * b)
    ra.ra_kv4_write(kv, cache, _dev(k[:, :, :n_prompt], dtype), _dev(v[:, :, :n_prompt], dtype), tab, zero)
    kr, vr = ra.ra_kv4_read(kv, cache, tab, zero, n_prompt)
    plan = ra.ra_plan_window(b, n_prompt, hq, hk, d, 3, window, sinks, layout="zigzag", dtype=dtype)
    to = lambda x: ra.ra_layout_perm(x, "zigzag", 3)
    o, lse = ra.ra_fwd(plan, to(_dev(q[:, :, :n_prompt], dtype)), to(kr), to(vr))
    o, lse = (ra.ra_layout_perm(x, "zigzag", 3, inverse=True) for x in (o, lse))
    ra.ra_sync_status(plan)
    outs, lses = [o], [lse]
    for x in range(n_prompt, total, 2):  # two tokens at a time
        rows = slice(x, x + 2)
        ra.ra_kv4_write(kv, cache, _dev(k[:, :, rows], dtype), _dev(v[:, :, rows], dtype), tab, _i32([x] * b))
        o, lse = ra.ra_kv4_attend(kv, cache, _dev(q[:, :, rows], dtype), tab, _i32([x + 2] * b))
        outs.append(o)
        lses.append(lse)
    ra.ra_kv4_sync_status(kv)
    o, lse = torch.cat(outs, 2).cpu(), torch.cat(lses, 2).cpu()
    u = kv4_ref.U[dtype]
    for i in range(b):
        ow, lw, ob, lb = kv4_ref.attend(kv4_ref.values(k[i]), kv4_ref.values(v[i]), q[i], total, window, sinks, u)
        # the prompt's values were rounded once more, to the dtype: u of every product in a
        # score and of every value
        mag = torch.as_tensor(np.abs(q[i])) @ torch.as_tensor(np.abs(kv4_ref.values(k[i]))).repeat_interleave(
            hq // hk, 0).transpose(-1, -2) * d ** -0.5
        more = u * mag.amax(-1)
        assert_within(lse[i], lw, lb + more, "LSE")
        assert_within(o[i], ow, ob * (1 + 2 * more[..., None] / u) + u * 3 * ob / u, "O")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("length,page_rows", [(1, 16), (9, 16), (700, 64)])
def test_rows_that_see_only_nan(dtype, length, page_rows):
    """A query whose visible keys are all NaN gets NaN, not the zeros of an empty row; with
    700 keys they are shared by several CTAs.  The other sequence is as it was."""
    rng = np.random.default_rng(length)
    kv, cache, _, table = _filled(rng, [length, length], page_rows, 1, 64, dtype, heads_q=2)
    q = _dev(rng.normal(size=(2, 2, 1, 64)), dtype)
    tab, n = _i32(table), _i32([length, length])
    o0, lse0 = ra.ra_kv4_attend(kv, cache, q, tab, n)
    bad = torch.full((2, 1, length, 64), float("nan"), dtype=DT[dtype], device="cuda")
    good = _dev(rng.normal(size=(2, 1, length, 64)), dtype)
    ra.ra_kv4_write(kv, cache, bad, good, tab, _i32([0, 0]), _i32([length, 0]))
    o, lse = ra.ra_kv4_attend(kv, cache, q, tab, n)
    ra.ra_kv4_sync_status(kv)
    assert torch.isnan(o[0]).all() and torch.isnan(lse[0]).all()
    assert torch.equal(o[1], o0[1]) and torch.equal(lse[1], lse0[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,hk,d,window,sinks", [(150, 1, 64, 0, 0), (70, 8, 128, 0, 0), (150, 1, 128, 40, 3)])
def test_many_ragged_sequences(dtype, n, hk, d, window, sinks):
    """More sequences than threads of a CTA, empty ones among them, and more sequences than
    CTAs of a head: shares that hold the end of one sequence, several whole ones and the
    beginning of another."""
    rng = np.random.default_rng(n + d)
    lengths = [int(x) for x in rng.integers(0, 90, n)]
    lengths[0], lengths[7], lengths[n // 2], lengths[-1] = 0, 600, 333, 0
    kv, cache, ref, table = _filled(rng, lengths, 32, hk, d, dtype, heads_q=2 * hk, window=window, sinks=sinks)
    table = np.concatenate([table, np.full((n, 132 - table.shape[1]), -1)], 1)  # room for 4224 tokens
    assert ra.ra_kv4_attend_scratch_size(kv, n, 1, table.shape[1]) > 0 or window
    _check_attend(kv, cache, ref, table, lengths, 2 * hk, 1, d, dtype, window, sinks, rng)


def test_shares_follow_the_lengths_in_a_graph():
    """A captured call shares the blocks out anew at every replay."""
    rng = np.random.default_rng(21)
    top = [700, 320, 900, 64]
    kv, cache, ref, table = _filled(rng, top, 32, 2, 64, "bf16", heads_q=4)
    table = np.concatenate([table, np.full((4, 60 - table.shape[1]), -1)], 1)  # room for 1920 tokens
    q = _dev(rng.normal(size=(4, 4, 1, 64)), "bf16")
    tab, n = _i32(table), _i32(top)
    need = ra.ra_kv4_attend_scratch_size(kv, 4, 1, table.shape[1])
    assert need > 0
    o, lse, scratch = torch.empty_like(q), torch.empty((4, 4, 1), device="cuda"), torch.empty(need // 4, device="cuda")
    call = lambda: ra.ra_kv4_attend(kv, cache, q, tab, n, o=o, lse=lse, scratch=scratch)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lengths in (top, [1, 320, 0, 64], [0, 0, 900, 0], [0, 0, 0, 0], [700, 1, 1, 1]):
        n.copy_(_i32(lengths))
        o.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        got = o.clone(), lse.clone()
        call()
        torch.cuda.synchronize()
        assert torch.equal(got[0], o) and torch.equal(got[1], lse)
        for b, length in enumerate(lengths):
            alone = ra.ra_kv4_attend(kv, cache, q[b:b + 1].contiguous(), tab[b:b + 1].contiguous(), _i32([length]))
            if length == 0:
                assert torch.isneginf(lse[b]).all() and (o[b] == 0).all()
                continue
            # The same sums cut otherwise.  Each side rounds every weight (2^-8 of it) and the
            # output once; the statistic's exponentials are off by 2^-21, its 900 additions by
            # 2^-24 each at most.
            top = float(np.abs(ref.rows(table[b], np.arange(length))[1]).max())
            assert torch.allclose(o[b].float(), alone[0][0].float(), rtol=2.0 ** -7, atol=2.0 ** -7 * top)
            assert torch.allclose(lse[b], alone[1][0], rtol=2.0 ** -22, atol=2 * (2.0 ** -21 + 900 * 2.0 ** -24))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1500, 20), (1700, 0)])
@pytest.mark.parametrize("t,hq,hk", [(1, 4, 1), (5, 16, 2), (9, 3, 3)])
def test_shared_in_a_row(dtype, window, sinks, t, hq, hk):
    """Few long sequences of different lengths, several query tiles, sinks behind which the
    window begins within a share."""
    rng = np.random.default_rng(window + t)
    lengths = [2300, 0, 1801, 40, 3]
    kv, cache, ref, table = _filled(rng, lengths, 48, hk, 128, dtype, heads_q=hq, window=window, sinks=sinks)
    assert ra.ra_kv4_attend_scratch_size(kv, 5, t, table.shape[1]) > 0
    _check_attend(kv, cache, ref, table, lengths, hq, t, 128, dtype, window, sinks, rng)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lengths,hq", [([4], 2), ([300, 9], 12), ([5000], 2)], ids=str)
@pytest.mark.parametrize("size", [1e19, 1e20, 1e25])
def test_values_far_from_zero(dtype, lengths, hq, size):
    """Value groups of one large constant (scale 0), as many of equal weight as sum past
    float32 when a weight carries 2^60, beside groups of ordinary size and of a large scale."""
    rng = np.random.default_rng(len(lengths))
    d, hk = 64, 2
    kv, cache, ref, table = _filled(rng, lengths, 32, hk, d, dtype, heads_q=hq)
    t = max(lengths)
    k = np.repeat(_rows(rng, len(lengths), hk, 1, d, dtype), t, 2)  # keys alike: equal weights
    v = _rows(rng, len(lengths), hk, t, d, dtype)
    # (a bf16 number: the float32 1e25 is 2^74 above its group's low, which makes a scale of
    # 2^70.6, and the scales that the attention takes end at 2^58)
    v[..., :32] = kv4_ref.bf16(size)
    v[:, 1, :, 32:] *= 2.0 ** 50
    v = torch.from_numpy(v).to(DT[dtype]).double().numpy()
    ref.write(k, v, table, [0] * len(lengths), lengths)
    ra.ra_kv4_write(kv, cache, _dev(k, dtype), _dev(v, dtype), _i32(table), _i32([0] * len(lengths)), _i32(lengths))
    _check_attend(kv, cache, ref, table, lengths, hq, 1, d, dtype, 0, 0, rng)


def test_reports_on_a_stream_of_its_own():
    """A report cleared, and the next one made at once by a stream that does not wait for the
    default one: none is lost."""
    kv = ra.ra_kv4_plan(1, 16, 1, 1, 64)
    cache = torch.zeros(ra.ra_kv4_cache_size(kv), dtype=torch.uint8, device="cuda")
    x = torch.zeros((1, 1, 1, 64), dtype=torch.bfloat16, device="cuda")
    bad, zero = _i32([[3]]), _i32([0])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(100):
        ra.ra_kv4_write(kv, cache, x, x, bad, zero, stream=side)
        with pytest.raises(ra.RaError):
            ra.ra_kv4_sync_status(kv, side)
    ra.ra_kv4_sync_status(kv, side)
