"""Host-side tests of windowed plans: refusals, tile counts, and the float64 reference's
gradients against differences.  No GPU is needed."""

import ctypes

import numpy as np
import pytest

import oracle

torch = pytest.importorskip("torch")
ra = pytest.importorskip("context_ring_attention_gb300")
from tests import window_ref  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _library():
    import os
    from context_ring_attention_gb300 import build
    if not os.path.exists(ra.library_path()):
        build.build()
    ra.load_library()


def _plan(window, sinks, **kw):
    args = dict(batch=1, seq=512, heads_q=4, heads_kv=2, head_dim=128, n_shards=4)
    args.update(kw)
    return ra.ra_plan_window(window=window, sinks=sinks, **args)


@pytest.mark.parametrize("window,sinks,kw,status", [
    (0, 0, {}, "RA_ERR_INVALID_ARG"),
    (-3, 0, {}, "RA_ERR_INVALID_ARG"),
    (8, -1, {}, "RA_ERR_INVALID_ARG"),
    (8, 0, dict(seq=510), "RA_ERR_INVALID_ARG"),            # uneven shards
    (8, 0, dict(seq=508, layout="zigzag"), "RA_ERR_INVALID_ARG"),
    (8, 0, dict(heads_q=3), "RA_ERR_INVALID_ARG"),
    (8, 0, dict(head_dim=64), "RA_ERR_UNSUPPORTED"),        # bf16 needs d = 128
    (8, 0, dict(head_dim=160, dtype="f32"), "RA_ERR_UNSUPPORTED"),
])
def test_refusals(window, sinks, kw, status):
    with pytest.raises(ra.RaError) as err:
        _plan(window, sinks, **kw)
    assert err.value.name == status


def test_reach_beyond_the_kernels_is_refused():
    """Sequences above 2^30 positions, and windows whose work items would outlast the
    kernels' bounded waits.  (float32 plans have no work lists: building them is quick.)"""
    big = dict(batch=1, heads_q=1, heads_kv=1, n_shards=1, head_dim=64, dtype="f32")
    _plan(4, 0, seq=1 << 30, **big)
    with pytest.raises(ra.RaError) as err:
        _plan(4, 0, seq=(1 << 30) + 1, **big)
    assert err.value.name == "RA_ERR_UNSUPPORTED"
    for window, sinks, heads in ((1 << 24, 1, 1), (1 << 25, 0, 2), (1 << 22, 1, 16), (1, 1 << 25, 1)):
        with pytest.raises(ra.RaError) as err:
            _plan(window, sinks, batch=1, seq=1 << 26, heads_q=heads, heads_kv=1, n_shards=1)
        assert err.value.name == "RA_ERR_UNSUPPORTED"


def test_non_causal_is_refused():
    lib = ra.load_library()
    prob = ra._Problem(1, 512, 4, 2, 128, 4, 0, 0, 1, 0.0)
    h = ctypes.c_void_p()
    assert lib.ra_plan_window(ctypes.byref(prob), 8, 0, ctypes.byref(h)) == 1
    assert not h.value and "causal" in ra.ra_last_error()
    assert lib.ra_plan_window(ctypes.byref(prob), 8, 0, None) == 1
    assert lib.ra_plan_window(None, 8, 0, ctypes.byref(h)) == 1


def test_largest_arguments():
    # window and sinks far beyond the sequence (and 32 bits): the whole causal prefix
    want = ra.ra_plan_tile_counts(ra.ra_plan(1, 512, 4, 2, 128, 4, "striped", True, "bf16"))
    for window, sinks in ((1 << 62, 0), (512, 0), (1, 1 << 62), (1, 512)):
        got = ra.ra_plan_tile_counts(_plan(window, sinks, layout="striped"))
        for g, w in zip(got, want):
            assert np.array_equal(g, w)


@pytest.mark.parametrize("layout", oracle.LAYOUTS)
@pytest.mark.parametrize("seq,n", [(512, 4), (900, 3), (1536, 2), (64, 8), (2048, 1)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (100, 4), (130, 0), (700, 200)])
def test_tile_counts(layout, seq, n, window, sinks):
    """FULL tiles against every (query, key) pair; every tile that holds a visible pair is
    visited, and for runs of consecutive positions no others are."""
    if layout == "zigzag" and seq % (2 * n):
        pytest.skip("zigzag needs 2N | S")
    full, part, skip = ra.ra_plan_tile_counts(_plan(window, sinks, seq=seq, n_shards=n, layout=layout))
    pos = torch.from_numpy(oracle.layout_positions(layout, seq, n))
    vis = window_ref.visible(pos, pos, window, sinks).numpy()
    s_n = seq // n
    tiles = range(0, s_n, 128)
    for p in range(n):
        n_full = n_some = 0
        for q0 in tiles:
            rows = slice(p * s_n + q0, p * s_n + min(q0 + 128, s_n))
            for r in range(n):
                for k0 in tiles:
                    block = vis[rows, r * s_n + k0:r * s_n + min(k0 + 128, s_n)]
                    n_full += bool(block.all())
                    n_some += bool(block.any())
        assert full[p] == n_full
        assert full[p] + part[p] >= n_some
        if layout == "contiguous":
            assert full[p] + part[p] == n_some
        assert full[p] + part[p] + skip[p] == len(tiles) * len(tiles) * n


def test_a_window_reduces_the_tiles():
    whole = ra.ra_plan_tile_counts(ra.ra_plan(1, 32768, 32, 8, 128, 8, "zigzag", True, "bf16"))
    part = ra.ra_plan_tile_counts(_plan(4096, 4, seq=32768, n_shards=8, heads_q=32, heads_kv=8, layout="zigzag"))
    # 33 tiles of the window and 1 of the sinks at most, for each of 32 query tiles
    assert (part[0] + part[1]).max() <= 32 * 34 < (whole[0] + whole[1]).min()


@pytest.mark.parametrize("seq,sinks", [(131072, 65536), (1 << 20, 1 << 19)])
def test_many_sinks_are_planned_with_bounded_scratch(seq, sinks):
    """Half the sequence sinks, the window one token: the pieces that the sinks' far queries are
    cut into stay as many as balance needs (10000, and the heads' last ones of every tile of
    sinks), each with the sums of 128 rows of dK and dV at most."""
    plan = _plan(1, sinks, seq=seq, n_shards=8, heads_q=32, heads_kv=8, layout="contiguous")
    tiles = 8 * sinks // 128
    scalars = 8 * 32 * seq
    assert ra.ra_bwd_scratch_size(plan) <= scalars + (10000 + tiles * (1 + 4)) * 2 * 128 * 128 * 4


def test_plan_without_a_device_refuses_to_compute():
    if torch.cuda.is_available():
        pytest.skip("a device is present")
    plan = _plan(8, 2)
    lib = ra.load_library()
    buf = ctypes.create_string_buffer(64 + 16)
    a = (ctypes.addressof(buf) + 15) & ~15
    assert lib.ra_fwd(plan.handle, a, a, a, a, None, None, None, None) == 5


@pytest.mark.parametrize("layout,n", [("contiguous", 1), ("zigzag", 3)])
def test_reference_gradients_against_differences(layout, n):
    """The reference's gradients, which the kernels are compared with, against central
    differences of the reference's forward in float64."""
    torch.manual_seed(5)
    b, hq, hk, s, d, window, sinks = 1, 4, 2, 18, 3, 5, 2
    pos = torch.from_numpy(oracle.layout_positions(layout, s, n))
    x = [torch.randn(b, h, s, d, dtype=torch.float64) for h in (hq, hk, hk)]
    do = torch.randn(b, hq, s, d, dtype=torch.float64)
    fwd = lambda *t: window_ref.forward(*t, pos, window, sinks, 0.0)
    o, lse, _, _ = fwd(*x)
    grads, _ = window_ref.backward(*x, o, lse, do, pos, window, sinks, 0.0)
    h = 1e-5
    for n_in in range(3):
        flat = x[n_in].view(-1)
        for at in range(0, flat.numel(), 7):
            keep = flat[at].item()
            vals = []
            for step in (h, -h):
                flat[at] = keep + step
                vals.append((fwd(*x)[0] * do).sum())
            flat[at] = keep
            slope = (vals[0] - vals[1]) / (2 * h)
            # truncation h^2 * third derivative, rounding 2^-53 / h
            assert abs(slope - grads[n_in].view(-1)[at]) < 1e-7
