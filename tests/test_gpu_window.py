"""GPU parity of windowed plans (ra_plan_window) on every path that takes a plan, against
the float64 reference with the bounds derived in window_ref.py."""

import os
import subprocess
import sys

import numpy as np
import pytest

import oracle
from tests.conftest import ROOT

torch = pytest.importorskip("torch")
ra = pytest.importorskip("context_ring_attention_gb300")
from context_ring_attention_gb300 import workloads  # noqa: E402
from tests import window_ref  # noqa: E402
from tests.window_ref import BF16_U, F32_U, assert_within  # noqa: E402

pytestmark = pytest.mark.gpu

# B, S, Hq, Hkv, N: ragged tiles, shards shorter than a tile, odd and unit groups, one token
SHAPES = [(1, 256, 8, 1, 1), (1, 900, 4, 2, 3), (2, 640, 2, 2, 4), (1, 768, 6, 2, 2), (1, 48, 4, 2, 8),
          (1, 16, 2, 1, 8), (1, 1300, 3, 1, 2), (1, 1, 1, 1, 1)]
MASKS = [(1, 0), (7, 3), (130, 4), (300, 200), (1, 1000), (5000, 0)]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ra.load_library()


def _setup(shape, layout, window, sinks, seed, dtype="bf16", d=128, q_scale=1.0):
    b, s, hq, hk, n = shape
    if layout == "zigzag" and s % (2 * n):
        pytest.skip("zigzag needs 2N | S")
    q, k, v = workloads.small_inputs(b, s, hq, hk, d, seed=seed, device="cuda", dtype=dtype, q_scale=q_scale)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    do = torch.randn(q.shape, generator=g, device="cuda").to(q.dtype)
    pos = torch.from_numpy(oracle.layout_positions(layout, s, n)).cuda()
    plan = ra.ra_plan_window(b, s, hq, hk, d, n, window, sinks, layout=layout, dtype=dtype)
    return plan, q, k, v, do, pos


@pytest.mark.parametrize("mask", MASKS, ids=str)
@pytest.mark.parametrize("layout", oracle.LAYOUTS)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_bf16_forward_and_gradients(shape, layout, mask):
    plan, q, k, v, do, pos = _setup(shape, layout, *mask, seed=sum(shape) + mask[0])
    o, lse = ra.ra_fwd(plan, q, k, v)
    grads = ra.ra_bwd(plan, q, k, v, o, lse, do)
    ra.ra_sync_status(plan)
    ow, lw, ob, lb = window_ref.forward(q, k, v, pos, *mask, BF16_U)
    assert_within(o, ow, ob, "O")
    assert_within(lse, lw, lb, "LSE")
    want, bound = window_ref.backward(q, k, v, o, lse, do, pos, *mask, BF16_U)
    for name, g_, w_, b_ in zip(("dQ", "dK", "dV"), grads, want, bound):
        assert_within(g_, w_, b_, name)


@pytest.mark.parametrize("mask", [(7, 3), (300, 200)], ids=str)
@pytest.mark.parametrize("layout", oracle.LAYOUTS)
@pytest.mark.parametrize("shape", [(1, 900, 4, 2, 3), (1, 768, 6, 2, 2), (1, 48, 4, 2, 8), (1, 1300, 3, 1, 2)], ids=str)
def test_bf16_ring_paths(shape, layout, mask):
    """Partials and their merge, per-step launches on passed-on blocks, the ring driver,
    gathered K/V."""
    plan, q, k, v, _, pos = _setup(shape, layout, *mask, seed=sum(shape))
    n = shape[4]
    ow, lw, ob, lb = window_ref.forward(q, k, v, pos, *mask, BF16_U)
    op, lp = ra.ra_fwd(plan, q, k, v, partials=True)
    ra.ra_sync_status(plan)
    # every step alone: attention over the keys of the block met
    s_n = shape[1] // n
    for t in range(n):
        for p in range(n):
            rows = slice(p * s_n, (p + 1) * s_n)
            r = (p - t) % n
            keys = torch.arange(r * s_n, (r + 1) * s_n, device="cuda")
            vis = window_ref.visible(pos[rows], pos[keys], *mask)
            empty = ~vis.any(1)
            assert torch.isneginf(lp[t][:, :, rows][:, :, empty]).all()
            assert (op[t][:, :, rows][:, :, empty] == 0).all()
            assert torch.isfinite(lp[t][:, :, rows][:, :, ~empty]).all()
    o, lse = ra.ra_merge_partials(op, lp)
    assert_within(o, ow, ob, "merged O")
    assert_within(lse, lw, lb, "merged LSE")
    kb, vb = k, v
    for t in range(n):
        o_t, lse_t = ra.ra_fwd_step(plan, t, q, kb, vb)
        ra.ra_sync_status(plan)
        assert torch.equal(o_t, op[t]) and torch.equal(lse_t, lp[t]), f"step {t}"
        if t + 1 < n:
            kb, vb = ra.ra_ring_rotate(plan, kb, vb)
    o, lse = ra.ra_ring_fwd(plan, q, k, v)
    assert_within(o, ow, ob, "ring driver O")
    assert_within(lse, lw, lb, "ring driver LSE")
    o, lse = ra.ra_fwd_gathered(plan, q, *ra.ra_allgather_kv(plan, k, v))
    ra.ra_sync_status(plan)
    assert_within(o, ow, ob, "gathered O")
    assert_within(lse, lw, lb, "gathered LSE")


@pytest.mark.parametrize("layout", oracle.LAYOUTS)
@pytest.mark.parametrize("d", [1, 13, 32, 128])
@pytest.mark.parametrize("mask", [(1, 0), (17, 2), (1, 1000), (1000, 0)], ids=str)
def test_f32_every_path(layout, d, mask):
    shape = (2, 96, 4, 2, 4)
    plan, q, k, v, do, pos = _setup(shape, layout, *mask, seed=d, dtype="f32", d=d)
    ow, lw, ob, lb = window_ref.forward(q, k, v, pos, *mask, F32_U)
    o, lse = ra.ra_fwd(plan, q, k, v)
    assert_within(o, ow, ob, "O")
    assert_within(lse, lw, lb, "LSE")
    want, bound = window_ref.backward(q, k, v, o, lse, do, pos, *mask, F32_U)
    for name, g_, w_, b_ in zip(("dQ", "dK", "dV"), ra.ra_bwd(plan, q, k, v, o, lse, do), want, bound):
        assert_within(g_, w_, b_, name)
    for what, (o, lse) in (("partials", ra.ra_merge_partials(*ra.ra_fwd(plan, q, k, v, partials=True))),
                           ("ring", ra.ra_ring_fwd(plan, q, k, v)),
                           ("gathered", ra.ra_fwd_gathered(plan, q, *ra.ra_allgather_kv(plan, k, v)))):
        assert_within(o, ow, ob, what)
        assert_within(lse, lw, lb, what)
    ra.ra_sync_status(plan)


def test_large_logits_rescale():
    """Q x 4: the running maximum moves from tile to tile, and few keys carry a row."""
    plan, q, k, v, do, pos = _setup((1, 1024, 4, 2, 2), "zigzag", 400, 4, seed=3, q_scale=4.0)
    o, lse = ra.ra_fwd(plan, q, k, v)
    grads = ra.ra_bwd(plan, q, k, v, o, lse, do)
    ra.ra_sync_status(plan)
    ow, lw, ob, lb = window_ref.forward(q, k, v, pos, 400, 4, BF16_U)
    assert_within(o, ow, ob, "O")
    assert_within(lse, lw, lb, "LSE")
    want, bound = window_ref.backward(q, k, v, o, lse, do, pos, 400, 4, BF16_U)
    for name, g_, w_, b_ in zip(("dQ", "dK", "dV"), grads, want, bound):
        assert_within(g_, w_, b_, name)


@pytest.mark.parametrize("layout", oracle.LAYOUTS)
@pytest.mark.parametrize("shape,mask", [((1, 1024, 8, 2, 4), (512, 4)), ((2, 810, 4, 1, 1), (253, 1)),
                                        ((1, 2048, 4, 1, 2), (2048, 0)), ((1, 1500, 6, 1, 3), (400, 300)),
                                        ((1, 2048, 16, 8, 2), (300, 5))], ids=str)
def test_bf16_gradients_of_cut_tiles(shape, layout, mask):
    """Few key tiles with long chains of queries, which are cut into pieces by heads and by
    queries, with and without sinks; and passes side by side in more than one wave."""
    plan, q, k, v, do, pos = _setup(shape, layout, *mask, seed=sum(shape) + mask[0])
    o, lse = ra.ra_fwd(plan, q, k, v)
    grads = ra.ra_bwd(plan, q, k, v, o, lse, do)
    ra.ra_sync_status(plan)
    want, bound = window_ref.backward(q, k, v, o, lse, do, pos, *mask, BF16_U)
    for name, g_, w_, b_ in zip(("dQ", "dK", "dV"), grads, want, bound):
        assert_within(g_, w_, b_, name)
    for a, b in zip(grads, ra.ra_bwd(plan, q, k, v, o, lse, do)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("shape,mask", [((1, 900, 4, 2, 3), (122, 4)), ((1, 512, 4, 2, 8), (124, 4)),
                                        ((2, 512, 3, 1, 8), (122, 1)), ((1, 512, 2, 2, 4), (126, 1)),
                                        ((1, 600, 3, 1, 100), (150, 30))], ids=str)
def test_first_stripe_of_the_window_holds_the_last_sink(shape, mask):
    """Striped shards walked by position, where a range of keys begins with its stripe: a sink
    in the window's first stripe enters once."""
    plan, q, k, v, do, pos = _setup(shape, "striped", *mask, seed=sum(shape) + mask[0])
    o, lse = ra.ra_fwd(plan, q, k, v)
    grads = ra.ra_bwd(plan, q, k, v, o, lse, do)
    ra.ra_sync_status(plan)
    ow, lw, ob, lb = window_ref.forward(q, k, v, pos, *mask, BF16_U)
    assert_within(o, ow, ob, "O")
    assert_within(lse, lw, lb, "LSE")
    want, bound = window_ref.backward(q, k, v, o, lse, do, pos, *mask, BF16_U)
    for name, g_, w_, b_ in zip(("dQ", "dK", "dV"), grads, want, bound):
        assert_within(g_, w_, b_, name)


@pytest.mark.parametrize("layout,mask", [("zigzag", (300, 4)), ("contiguous", (1, 0)), ("striped", (40, 200)),
                                         ("contiguous", (5000, 1))], ids=str)
def test_steps_in_which_most_items_meet_no_key(layout, mask):
    """Ring steps of a long sequence under a short window: a CTA has long rows of items without
    a key in the step between few with one, or none of these at all."""
    plan, q, k, v, _, pos = _setup((1, 16384, 16, 4, 8), layout, *mask, seed=mask[0])
    n, s_n = 8, 2048
    op, lp = ra.ra_fwd(plan, q, k, v, partials=True)
    ra.ra_sync_status(plan)
    kb, vb = k, v
    for t in range(n):
        o_t = torch.full_like(op[0], 7.0)
        o_t, lse_t = ra.ra_fwd_step(plan, t, q, kb, vb, o_part=o_t)
        ra.ra_sync_status(plan)
        assert torch.equal(o_t, op[t]) and torch.equal(lse_t, lp[t]), f"step {t}"
        for p in range(n):
            rows, r = slice(p * s_n, (p + 1) * s_n), (p - t) % n
            seen = window_ref.visible(pos[rows], pos[r * s_n:(r + 1) * s_n], *mask).any(1)
            assert torch.equal(torch.isneginf(lse_t[0, 0, rows]), ~seen)
        if t + 1 < n:
            kb, vb = ra.ra_ring_rotate(plan, kb, vb)
    o, lse = ra.ra_fwd(plan, q, k, v)
    o2, lse2 = ra.ra_ring_fwd(plan, q, k, v)
    ra.ra_sync_status(plan)
    # both round the weights and the outputs to bf16; the statistics are fp32 sums of the same terms
    assert (o.float() - o2.float()).abs().max() <= 3 * BF16_U * v.abs().max()
    assert (lse - lse2).abs().max() <= 2.0 ** -13


def test_long_window_one_head_pair():
    """32k tokens, 4096-token window: 512 rows spread over the sequence, all of dK and dV of
    the sinks (each gathers every later query)."""
    b, s, hq, hk, n, window, sinks = 1, 32768, 4, 2, 8, 4096, 4
    plan, q, k, v, do, pos = _setup((b, s, hq, hk, n), "zigzag", window, sinks, seed=11)
    o, lse = ra.ra_fwd(plan, q, k, v)
    dq, dk, dv = ra.ra_bwd(plan, q, k, v, o, lse, do)
    ra.ra_sync_status(plan)
    rows = torch.linspace(0, s - 1, 512).long().cuda()
    scale = 128 ** -0.5
    for h in range(hq):
        kk, vv = k[0, h // 2].double(), v[0, h // 2].double()
        x = (q[0, h, rows].double() @ kk.T) * scale
        mag = (q[0, h, rows].double().abs() @ kk.abs().T).amax(-1) * scale
        vis = window_ref.visible(pos[rows], pos, window, sinks)
        x = x.masked_fill(~vis, -torch.inf)
        lw = torch.logsumexp(x, -1)
        p = torch.exp(x - lw[:, None])
        e = 2.0 ** -15 * (1 + mag) + window * 2.0 ** -23
        assert_within(lse[0, h, rows], lw, e, "LSE")
        assert_within(o[0, h, rows], p @ vv, (BF16_U + 2 * e[:, None]) * (p @ vv.abs()) + BF16_U * (p @ vv).abs(), "O")
    sink_rows = (pos < sinks).nonzero()[:, 0]
    for kv in range(hk):
        want_k = torch.zeros((sinks, 128), dtype=torch.float64, device="cuda")
        want_v, bound_k, bound_v = (torch.zeros_like(want_k) for _ in range(3))
        for h in (2 * kv, 2 * kv + 1):
            qq, dd, oo = q[0, h].double(), do[0, h].double(), o[0, h].double()
            p = torch.exp(qq @ k[0, kv, sink_rows].double().T * scale - lse[0, h].double()[:, None])
            p = p.masked_fill(~window_ref.visible(pos, pos[sink_rows], window, sinks), 0.0)
            mag = (qq.abs() @ k[0, kv, sink_rows].double().abs().T) * scale
            inner = dd.abs() @ v[0, kv, sink_rows].double().abs().T + (dd * oo).abs().sum(-1, keepdim=True)
            ds = p * (dd @ v[0, kv, sink_rows].double().T - (dd * oo).sum(-1, keepdim=True))
            e = BF16_U + 2.0 ** -15 * (1 + mag) + 2 * s * 2.0 ** -23
            want_k += scale * ds.T @ qq
            want_v += p.T @ dd
            bound_k += scale * (e * ds.abs() + 2.0 ** -15 * p * inner).T @ qq.abs()
            bound_v += (e * p).T @ dd.abs()
        assert_within(dk[0, kv, sink_rows], want_k, bound_k + BF16_U * want_k.abs(), "dK of the sinks")
        assert_within(dv[0, kv, sink_rows], want_v, bound_v + BF16_U * want_v.abs(), "dV of the sinks")


def test_whole_prefix_window_agrees_with_the_causal_plan():
    plan, q, k, v, _, pos = _setup((1, 900, 4, 2, 3), "striped", 900, 0, seed=21)
    causal = ra.ra_plan(1, 900, 4, 2, 128, 3, "striped", True, "bf16")
    o, lse = ra.ra_fwd(plan, q, k, v)
    o2, lse2 = ra.ra_fwd(causal, q, k, v)
    ra.ra_sync_status(plan)
    ra.ra_sync_status(causal)
    _, _, ob, _ = window_ref.forward(q, k, v, pos, 900, 0, BF16_U)
    assert_within(o, o2.double(), 2 * ob, "O")
    # the causal plan's LSE holds its rows' bf16 rounding of the largest weight
    assert (lse - lse2).abs().max() <= BF16_U * 1.01


def test_repeatable_and_on_another_stream():
    plan, q, k, v, do, _ = _setup((1, 2048, 8, 2, 4), "zigzag", 500, 130, seed=31)
    o, lse = ra.ra_fwd(plan, q, k, v)
    grads = ra.ra_bwd(plan, q, k, v, o, lse, do)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    o2, lse2 = ra.ra_fwd(plan, q, k, v, stream=side)
    side.synchronize()
    grads2 = ra.ra_bwd(plan, q, k, v, o2, lse2, do, stream=side)
    ra.ra_sync_status(plan, side)
    for a, b in zip((o, lse) + grads, (o2, lse2) + grads2):
        assert torch.equal(a, b)


def test_captured_step_replays():
    """A forward and backward captured into a graph, while eager results of the same inputs
    live, replayed on new inputs."""
    plan, q, k, v, do, pos = _setup((1, 900, 4, 2, 3), "contiguous", 100, 4, seed=41)
    _, q2, k2, v2, do2, _ = _setup((1, 900, 4, 2, 3), "contiguous", 100, 4, seed=43)
    eager = [ra.ra_fwd(plan, *x) for x in ((q, k, v), (q2, k2, v2))]
    eager = [(o, lse) + ra.ra_bwd(plan, *x, o, lse, g) for (o, lse), x, g in
             zip(eager, ((q, k, v), (q2, k2, v2)), (do, do2))]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = ra.ra_fwd(plan, q, k, v)
        out = (o, lse) + ra.ra_bwd(plan, q, k, v, o, lse, do)
    for want, src in ((eager[0], None), (eager[1], (q2, k2, v2, do2))):
        if src is not None:
            for dst, s in zip((q, k, v, do), src):
                dst.copy_(s)
        graph.replay()
        ra.ra_sync_status(plan)
        for a, b in zip(out, want):
            assert torch.equal(a, b)


def bounds_outputs():
    """Outputs of every windowed bf16 path on shapes that stress the index arithmetic (also
    run by the child process on the debug library)."""
    out = {}
    for n_case, (shape, layout, mask) in enumerate([((1, 900, 4, 2, 3), "striped", (100, 4)),
                                                    ((1, 768, 6, 2, 2), "zigzag", (130, 200)),
                                                    ((1, 320, 2, 1, 8), "zigzag", (7, 0)),
                                                    ((2, 640, 2, 2, 4), "contiguous", (300, 3)),
                                                    ((1, 16, 4, 2, 16), "contiguous", (2, 1))]):
        plan, q, k, v, do, _ = _setup(shape, layout, *mask, seed=600 + n_case)
        o, lse = ra.ra_fwd(plan, q, k, v)
        ts = [o, lse, *ra.ra_bwd(plan, q, k, v, o, lse, do), *ra.ra_fwd(plan, q, k, v, partials=True),
              *ra.ra_ring_fwd(plan, q, k, v), *ra.ra_fwd_gathered(plan, q, *ra.ra_allgather_kv(plan, k, v))]
        ra.ra_sync_status(plan)
        for n, t in enumerate(ts):
            out[f"{n_case}/{n}"] = t.float().cpu().numpy()
    return out


def test_debug_library_passes_its_bounds_checks(tmp_path):
    path = str(tmp_path / "out.npz")
    env = dict(os.environ, RA_LIBRARY_VARIANT="debug")
    code = ("import numpy as np, sys; from tests import test_gpu_window as t; "
            "np.savez(sys.argv[1], **t.bounds_outputs())")
    res = subprocess.run([sys.executable, "-c", code, path], cwd=ROOT, env=env, capture_output=True, text=True,
                         timeout=300)
    assert res.returncode == 0, res.stderr[-2000:]
    here = bounds_outputs()
    with np.load(path) as debug:
        assert set(debug.files) == set(here)
        for name, a in here.items():
            assert np.array_equal(a, debug[name], equal_nan=True), name
