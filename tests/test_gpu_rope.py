"""GPU tests of the rotary positions against the plain form in paged_ref.py."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
ra = pytest.importorskip("context_ring_attention_gb300")
from tests import paged_ref  # noqa: E402
from tests.paged_ref import DT, U  # noqa: E402
from tests.window_ref import assert_within  # noqa: E402

pytestmark = pytest.mark.gpu

SCALED = {"none": dict(), "linear": dict(scaling="linear", factor=4.0), "base": dict(scaling="base", factor=8.0),
          "bands": dict(scaling="bands", factor=8.0, original=512, base=500000.0, low=1.0, high=4.0),
          "ramp": dict(scaling="ramp", factor=16.0, original=512, low=1.0, high=32.0)}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ra.load_library()


def _x(rng, shape, dtype):
    return torch.from_numpy(rng.normal(size=shape)).to(DT[dtype])


def _check(got, x, pos, dtype, rot, **kw):
    y, b = paged_ref.rotate(x.double().numpy(), pos, rot, **kw)
    y = torch.from_numpy(y)
    assert_within(got.cpu(), y, torch.from_numpy(b) + U[dtype] * y.abs(), "rotated")
    assert torch.equal(got[..., rot:].cpu(), x[..., rot:])  # copied


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("scaling", list(SCALED))
@pytest.mark.parametrize("b,s,hq,hk,d,rot,layout,n", [
    (1, 1, 1, 1, 128, 128, "contiguous", 1), (2, 96, 4, 2, 64, 64, "striped", 3), (1, 300, 6, 2, 128, 64, "zigzag", 2),
    (3, 17, 3, 1, 80, 32, "contiguous", 1), (2, 10, 2, 2, 24, 10, "striped", 5), (1, 8, 5, 1, 7, 2, "contiguous", 2),
    (2, 33, 9, 3, 256, 96, "contiguous", 3)])
def test_forward_and_gradient(dtype, interleaved, scaling, b, s, hq, hk, d, rot, layout, n):
    """Every layout, odd sizes, part of the head, one row; both directions, and both as one map
    and its transpose."""
    rng = np.random.default_rng(s + d)
    args = dict(interleaved=interleaved, **SCALED[scaling])
    rope = ra.ra_rope_plan(d, rot, dtype=dtype, amplitude=1.25, **args)
    q, k = _x(rng, (b, hq, s, d), dtype), _x(rng, (b, hk, s, d), dtype)
    pos = ra.ra_layout_index(layout, s, n)
    for call, transposed in ((ra.ra_rope, False), (ra.ra_rope_bwd, True)):
        out = call(rope, q.cuda(), k.cuda(), layout=layout, n_shards=n)
        for got, x in zip(out, (q, k)):
            _check(got, x, pos, dtype, rot, amplitude=1.25, transposed=transposed, **args)
    assert torch.equal(ra.ra_rope(rope, q.cuda(), layout=layout, n_shards=n), ra.ra_rope(rope, q.cuda(), k.cuda(),
                                                                                        layout=layout, n_shards=n)[0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rot", [64, 30])
def test_far_and_negative_positions(dtype, rot):
    """Angles are exact modulo a turn at every int32 position."""
    rng = np.random.default_rng(rot)
    pos = np.array([[0, 1, -1, 4095, 4096, 1 << 20, (1 << 20) + 1, 123456789, (1 << 31) - 1, -(1 << 31), 1 << 30, 99999]], np.int64)
    rope = ra.ra_rope_plan(64, rot, dtype=dtype)
    q = _x(rng, (1, 3, 12, 64), dtype)
    got = ra.ra_rope(rope, q.cuda(), position=torch.from_numpy(pos).int().cuda())
    _check(got, q, pos[:, None], dtype, rot)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lead", [0, 1])
def test_strides(dtype, lead):
    """Projections' order, unaligned rows, rows read more than once, in place, parts of a larger
    tensor: the same numbers, and nothing beside the rows is written."""
    rng = np.random.default_rng(lead)
    b, h, s, d = 2, 3, 21, 64
    rope = ra.ra_rope_plan(d, 48, dtype=dtype)
    x = _x(rng, (b, h, s, d), dtype)
    want = ra.ra_rope(rope, x.cuda(), layout="striped", n_shards=3)
    wide = torch.zeros((b, s, h + 2, d + 8), dtype=DT[dtype], device="cuda")
    view = wide[:, :, 1:1 + h, lead:lead + d].transpose(1, 2)  # (lead 1: no row is 16-byte aligned)
    view.copy_(x)
    out = torch.full((b, s, h + 2, d + 8), 7.0, dtype=DT[dtype], device="cuda")
    to = out[:, :, 1:1 + h, lead:lead + d].transpose(1, 2)
    assert ra.ra_rope(rope, view, layout="striped", n_shards=3, q_out=to) is to
    assert torch.equal(to, want)
    to.fill_(7.0)
    assert (out == 7).all()
    assert ra.ra_rope(rope, view, layout="striped", n_shards=3, q_out=view) is view  # in place
    assert torch.equal(view, want)
    view.fill_(0.0)
    assert (wide == 0).all()
    one = x[:1, :1].cuda().expand(b, h, s, d)
    assert torch.equal(ra.ra_rope(rope, one, layout="striped", n_shards=3)[1, 2],
                       ra.ra_rope(rope, x[:1, :1].cuda(), layout="striped", n_shards=3)[0, 0])
    with pytest.raises(ra.RaError):
        ra.ra_rope(rope, x.cuda(), q_out=torch.empty((1, h, s, d), dtype=DT[dtype], device="cuda").expand(b, h, s, d))


def test_other_streams_and_graphs():
    rng = np.random.default_rng(2)
    rope = ra.ra_rope_plan(128)
    q, k = _x(rng, (1, 4, 256, 128), "bf16").cuda(), _x(rng, (1, 2, 256, 128), "bf16").cuda()
    pos = torch.arange(256, dtype=torch.int32, device="cuda")[None].contiguous()
    want = ra.ra_rope(rope, q, k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ra.ra_rope(rope, q, k, stream=side)
    side.synchronize()
    assert all(torch.equal(a, e) for a, e in zip(got, want))
    out = torch.empty_like(q), torch.empty_like(k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ra.ra_rope(rope, q, k, position=pos, q_out=out[0], k_out=out[1])
    for shift in (0, 1000):
        pos.copy_(torch.arange(256, device="cuda")[None] + shift)
        graph.replay()
        want = ra.ra_rope(rope, q, k, position=pos)
        torch.cuda.synchronize()
        assert all(torch.equal(a, e) for a, e in zip(out, want))
    ra.ra_rope_destroy(rope)


def test_refused_tensors():
    rope = ra.ra_rope_plan(64)
    q = torch.zeros((1, 2, 8, 64), dtype=torch.bfloat16, device="cuda")
    for bad in (q.cpu(), q.float(), q[0], q[..., ::2].repeat(1, 1, 1, 2)[..., ::2]):
        with pytest.raises(ValueError):
            ra.ra_rope(rope, bad)
    with pytest.raises(ValueError):
        ra.ra_rope(rope, q, position=torch.zeros((1, 8), dtype=torch.int32))
    for kw in (dict(layout="zigzag", n_shards=3), dict(n_shards=0), dict(layout=9)):
        with pytest.raises(ra.RaError):
            ra.ra_rope(rope, q, **kw)


def test_ring_with_rotated_queries_and_keys():
    """Projections rotated into a zigzag ring, its gradients rotated back: the same attention and
    gradients as float64 autograd's."""
    torch.manual_seed(0)
    b, s, hq, hk, d, n = 1, 256, 4, 2, 128, 4
    rope = ra.ra_rope_plan(d, base=500.0)
    plan = ra.ra_plan(b, s, hq, hk, d, n, layout="zigzag", causal=True)
    x = [torch.randn((b, s, h, d)).bfloat16() for h in (hq, hk, hk)]
    order = torch.from_numpy(np.asarray(ra.ra_layout_index("zigzag", s, n)).astype(np.int64))
    q, k, v = (t[:, order].cuda().transpose(1, 2) for t in x)  # the shards' rows, in the projections' order
    v = v.contiguous()
    q2, k2 = ra.ra_rope(rope, q, k, layout="zigzag", n_shards=n)
    o, lse = ra.ra_fwd(plan, q2, k2, v)
    do = torch.randn((b, hq, s, d)).bfloat16()
    dq2, dk2, dv = ra.ra_bwd(plan, q2, k2, v, o, lse, do.cuda())
    dq, dk = ra.ra_rope_bwd(rope, dq2, dk2, layout="zigzag", n_shards=n)
    ra.ra_sync_status(plan)

    leaf = [t.double().transpose(1, 2).requires_grad_() for t in x]
    c, sn = (torch.from_numpy(f(np.arange(s)[:, None] * paged_ref.speeds(d, base=500.0))) for f in (np.cos, np.sin))
    turn = lambda t: torch.cat([t[..., :64] * c - t[..., 64:] * sn, t[..., :64] * sn + t[..., 64:] * c], -1)
    g = hq // hk
    kk, vv = turn(leaf[1]).repeat_interleave(g, 1), leaf[2].repeat_interleave(g, 1)
    w = (turn(leaf[0]) @ kk.transpose(-1, -2) * d ** -0.5).masked_fill(torch.ones(s, s).triu(1).bool(), -torch.inf).softmax(-1)
    out = w @ vv
    natural = torch.empty_like(do)
    natural[:, :, order] = do
    (out * natural.double()).sum().backward()
    rms = lambda a, e: ((a.cpu().double() - e).pow(2).mean() / e.pow(2).mean()).sqrt()
    assert rms(o, out[:, :, order].detach()) < 1e-2
    # four roundings to bf16 on the way (2^-8 each at most, a third of that in the mean), two of them in both factors
    for got, t in zip((dq, dk, dv), leaf):
        assert rms(got, t.grad[:, :, order]) < 1.5e-2
