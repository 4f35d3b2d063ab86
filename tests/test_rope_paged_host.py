"""Host-side tests of the rotary positions and the paged cache: refusals, sizes, the binding's
checks, and the plain forms themselves.  No GPU is needed."""

import ctypes
import os

import numpy as np
import pytest

torch = pytest.importorskip("torch")
ra = pytest.importorskip("context_ring_attention_gb300")
from tests import paged_ref  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _library():
    from context_ring_attention_gb300 import build
    if not os.path.exists(ra.library_path()):
        build.build()
    ra.load_library()


END = 1 if torch.cuda.is_available() else 5  # a call whose arguments are fine: host pointers, or no device


def _kv(**kw):
    return ra.ra_paged_plan(**{**dict(pages=6, page_rows=32, heads_q=4, heads_kv=2, head_dim=128), **kw})


@pytest.mark.parametrize("kw", [
    dict(head_dim=0), dict(head_dim=1), dict(rotary_dim=3), dict(rotary_dim=130), dict(rotary_dim=-2), dict(dtype=2),
    dict(base=1.0), dict(base=float("inf")), dict(base=float("nan")), dict(scaling=5), dict(scaling=-1),
    dict(scaling="linear", factor=0.5), dict(scaling="base", factor=float("inf")), dict(scaling="bands", factor=8.0),
    dict(scaling="bands", factor=8.0, original=8192, low=4.0, high=4.0), dict(scaling="ramp", factor=8.0, original=8192, low=0.0),
    dict(scaling="ramp", factor=float("nan"), original=8192), dict(amplitude=float("inf"))])
def test_refused_rotations(kw):
    with pytest.raises(ra.RaError) as err:
        ra.ra_rope_plan(**{**dict(head_dim=128), **kw})
    assert err.value.name == "RA_ERR_INVALID_ARG"


def test_unsupported_rotation_and_amplitude():
    with pytest.raises(ra.RaError) as err:
        ra.ra_rope_plan(1026)
    assert err.value.name == "RA_ERR_UNSUPPORTED"
    ra.ra_rope_plan(1024)
    for bad in (0.0, -1.0, float("nan")):
        with pytest.raises(ValueError):
            ra.ra_rope_plan(64, amplitude=bad)


@pytest.mark.parametrize("kw,status", [
    (dict(pages=0), "RA_ERR_INVALID_ARG"), (dict(page_rows=0), "RA_ERR_INVALID_ARG"),
    (dict(page_rows=24), "RA_ERR_INVALID_ARG"), (dict(page_rows=65552), "RA_ERR_INVALID_ARG"),
    (dict(heads_q=3), "RA_ERR_INVALID_ARG"), (dict(heads_kv=0), "RA_ERR_INVALID_ARG"),
    (dict(window=-1), "RA_ERR_INVALID_ARG"), (dict(sinks=-1), "RA_ERR_INVALID_ARG"),
    (dict(scale=float("inf")), "RA_ERR_INVALID_ARG"), (dict(scale=-1.0), "RA_ERR_INVALID_ARG"),
    (dict(scale=float("nan")), "RA_ERR_INVALID_ARG"), (dict(scale=2.0 ** -101), "RA_ERR_INVALID_ARG"), (dict(dtype=7), "RA_ERR_INVALID_ARG"),
    (dict(head_dim=0), "RA_ERR_INVALID_ARG"), (dict(head_dim=96), "RA_ERR_UNSUPPORTED"),
    (dict(head_dim=256), "RA_ERR_UNSUPPORTED"), (dict(heads_q=65536, heads_kv=65536), "RA_ERR_UNSUPPORTED"),
    (dict(pages=1 << 24, page_rows=64), "RA_ERR_UNSUPPORTED")])
def test_refused_caches(kw, status):
    with pytest.raises(ra.RaError) as err:
        _kv(**kw)
    assert err.value.name == status


def test_shape_and_scratch():
    kv = _kv()
    assert ra.ra_paged_cache_shape(kv) == (6, 2, 2, 32, 128)
    assert ra.ra_paged_attend_scratch_size(kv, 1, 1, 1) == 0  # one share
    n = ra.ra_paged_attend_scratch_size(kv, 1, 1, 4096)
    assert n > 0 and n % 16 == 0
    assert ra.ra_paged_attend_scratch_size(_kv(window=64, sinks=4), 1, 1, 4096) == 0  # the window bounds the keys
    assert ra.ra_paged_attend_scratch_size(_kv(window=1 << 62, sinks=1 << 62), 1, 1, 4096) == n
    for args, status in (((0, 1, 1), "RA_ERR_INVALID_ARG"), ((1, 0, 1), "RA_ERR_INVALID_ARG"),
                         ((1, 1, 0), "RA_ERR_INVALID_ARG"), ((4097, 1, 1), "RA_ERR_UNSUPPORTED"),
                         ((1, 1 << 28, 1), "RA_ERR_UNSUPPORTED"), ((1, 1, (1 << 30) // 32 + 1), "RA_ERR_UNSUPPORTED")):
        for size in (ra.ra_paged_attend_scratch_size, ra.ra_paged_weigh_scratch_size):
            with pytest.raises(ra.RaError) as err:
                size(kv, *args)
            assert err.value.name == status
    # chunks: parts of every share; float32 and few rows need none for the weights
    assert ra.ra_paged_weigh_scratch_size(kv, 1, 100, 64) > 0 and ra.ra_paged_attend_scratch_size(kv, 1, 100, 64) % 16 == 0
    assert ra.ra_paged_weigh_scratch_size(kv, 100, 100, 64) == ra.ra_paged_weigh_scratch_size(_kv(dtype="f32"), 1, 100, 64) == 0


def _buffer():
    buf = ctypes.create_string_buffer(4096 + 16)
    return buf, (ctypes.addressof(buf) + 15) & ~15


def _s(*x):
    return (ctypes.c_int64 * len(x))(*x)


def test_refused_rope_calls():
    lib, (buf, a) = ra.load_library(), _buffer()
    rope = ra.ra_rope_plan(64, dtype="f32")
    h = rope.handle
    good = dict(b=1, s=2, hq=2, hk=1, layout=0, n=1, pos=a, q=a, qs=_s(256, 128, 64), k=a, ks=_s(128, 128, 64), qo=a,
                qos=_s(256, 128, 64), ko=a, kos=_s(128, 128, 64))

    def call(handle=h, fn=lib.ra_rope, **kw):
        x = {**good, **kw}
        return fn(handle, x["b"], x["s"], x["hq"], x["hk"], x["layout"], x["n"], x["pos"], x["q"], x["qs"], x["k"], x["ks"],
                  x["qo"], x["qos"], x["ko"], x["kos"], None)

    assert call() == END and call(fn=lib.ra_rope_bwd) == END
    assert call(hk=0, k=None, ks=None, ko=None, kos=None) == END
    assert call(qs=_s(0, 0, 0)) == END  # rows read more than once
    assert call(q=a + 4, qs=_s(257, 129, 65)) == END  # unaligned rows
    for kw in (dict(handle=None), dict(b=0), dict(s=0), dict(hq=0), dict(hk=-1), dict(layout=3), dict(n=0), dict(n=3, pos=None),
               dict(layout=2, n=2, pos=None), dict(pos=a + 2), dict(q=None), dict(k=None), dict(qo=None), dict(ko=None),
               dict(qs=None), dict(kos=None), dict(q=a + 2), dict(qs=_s(256, -128, 64)), dict(qos=_s(0, 0, 0)),
               dict(qos=_s(256, 64, 64)), dict(qos=_s(256, 128, 63)), dict(kos=_s(128, 128, 0)),
               dict(qs=_s(1 << 60, 128, 64), b=2)):
        assert call(**kw) == 1, kw
    assert call(s=1 << 32) == 2 and call(hq=(1 << 20) + 1, qos=_s(0, 64, 1 << 27), qs=_s(0, 0, 0)) == 2


def test_refused_paged_calls():
    """Bad pointers, sizes and strides are refused before anything is launched."""
    lib, (buf, a), kv = ra.load_library(), _buffer(), _kv()
    h, q4, kv2 = kv.handle, _s(512, 128), _s(256, 128)
    rope, other = ra.ra_rope_plan(128), ra.ra_rope_plan(64)
    f32 = ra.ra_rope_plan(128, dtype="f32")

    def append(kv=h, rope=rope.handle, cache=a, b=1, t=2, k=a, ks=kv2, v=a, vs=kv2, q=a, qs=q4, qo=a, qos=q4, tab=a, w=1, off=a,
               ln=a, pos=a):
        return lib.ra_paged_append(kv, rope, cache, b, t, k, ks, v, vs, q, qs, qo, qos, tab, w, off, ln, pos, None)

    def attend(kv=h, cache=a, b=1, t=2, q=a, qs=q4, tab=a, w=1, off=a, ln=a, o=a, os=q4, lse=a, scratch=a):
        return lib.ra_paged_attend(kv, cache, b, t, q, qs, tab, w, off, ln, o, os, lse, scratch, None)

    def weigh(kv=h, cache=a, b=1, t=2, q=a, qs=q4, lse=a, tab=a, w=1, off=a, ln=a, win=a, wout=a, ww=8, scratch=a):
        return lib.ra_paged_weigh(kv, cache, b, t, q, qs, lse, tab, w, off, ln, win, wout, ww, scratch, None)

    def evict(kv=h, cache=a, b=1, tab=a, w=1, ln=a, win=a, wout=a, ww=8, keep=4, first=1, recent=1, new=a, nw=1, kept=a,
              nl=a + 16):
        return lib.ra_paged_evict(kv, cache, b, tab, w, ln, win, wout, ww, keep, first, recent, new, nw, kept, nl, None)

    assert append() == append(q=None, qo=None, qs=None, qos=None) == append(pos=None) == END
    assert append(rope=None, q=None, qo=None, pos=None) == END
    assert attend() == attend(lse=None) == attend(scratch=None) == weigh() == weigh(win=None) == END
    assert evict() == evict(wout=None) == evict(keep=2) == evict(first=0, recent=0) == END
    shared = [dict(kv=None), dict(cache=None), dict(cache=a + 8), dict(b=0), dict(tab=None), dict(tab=a + 2), dict(w=0),
              dict(ln=None), dict(ln=a + 1)]
    packed = [dict(t=0), dict(off=None), dict(off=a + 2), dict(q=a + 8), dict(qs=_s(512, 124)), dict(qs=_s(-512, 128))]
    for kw in shared + packed + [
            dict(k=None), dict(v=None), dict(ks=None), dict(vs=_s(256, 4)), dict(k=a + 4), dict(q=None), dict(qo=None),
            dict(qos=_s(256, 128)), dict(qos=_s(512, 64)), dict(qos=None), dict(pos=a + 2), dict(rope=None),
            dict(rope=None, q=None, qo=None), dict(rope=other.handle), dict(rope=f32.handle)]:
        assert append(**kw) == 1, kw
    for kw in shared + packed + [dict(q=None), dict(o=None), dict(o=a + 8), dict(os=_s(0, 128)), dict(os=None), dict(lse=a + 2),
                                 dict(w=4096, scratch=None), dict(w=4096, scratch=a + 8),
                                 dict(t=20, scratch=None), dict(t=20, scratch=a + 4), dict(qs=_s(512, 0))]:
        assert attend(**kw) == 1, kw
    for kw in shared + packed + [dict(q=None), dict(lse=None), dict(wout=None), dict(win=a + 2), dict(ww=0), dict(ww=1 << 31),
                                 dict(t=20, scratch=None), dict(t=20, scratch=a + 4), dict(qs=_s(0, 128))]:
        assert weigh(**kw) == 1, kw
    for kw in shared + [dict(win=None), dict(wout=a + 2), dict(ww=0), dict(keep=0), dict(first=-1), dict(recent=-1),
                        dict(first=3, recent=2), dict(first=5), dict(keep=1 << 31), dict(new=None), dict(nw=0),
                        dict(nw=1 << 26), dict(kept=None), dict(nl=None), dict(nl=a)]:
        assert evict(**kw) == 1, kw
    for call in (append, attend, weigh):
        assert call(t=1 << 28) == call(b=4097) == call(w=1 << 26) == 2
    assert evict(b=4097) == evict(w=1 << 26) == 2
    assert lib.ra_paged_sync_status(None, None) == 1
    if END == 5:
        assert lib.ra_paged_sync_status(h, None) == 5
    assert lib.ra_paged_destroy(None) == lib.ra_rope_destroy(None) == 0


class _OnDevice(torch.Tensor):
    """A host tensor that passes for a CUDA tensor."""
    is_cuda = True


def _fake(shape, dtype):
    return torch.zeros(shape, dtype=dtype).as_subclass(_OnDevice)


class _Library:
    """Every entry point succeeds and does nothing."""

    def __getattr__(self, name):
        return lambda *args: 0


def _tensors():
    bf, i32 = torch.bfloat16, torch.int32
    return dict(cache=_fake((6, 2, 2, 32, 128), bf), q=_fake((3, 4, 128), bf), k=_fake((3, 2, 128), bf), v=_fake((3, 2, 128), bf),
                table=_fake((2, 3), i32), offset=_fake((3,), i32), length=_fake((2,), i32), position=_fake((3,), i32),
                lse=_fake((3, 4), torch.float32), weight=_fake((2, 2, 96), torch.float32),
                x=_fake((1, 4, 8, 128), bf), y=_fake((1, 2, 8, 128), bf))


def _binding_calls(kv, rope, t, stream=None):
    return dict(
        append=lambda **kw: ra.ra_paged_append(**{**dict(kv=kv, cache=t["cache"], k=t["k"], v=t["v"], page_table=t["table"],
                                                         offset=t["offset"], length=t["length"], rope=rope, q=t["q"],
                                                         position=t["position"], stream=stream), **kw}),
        attend=lambda **kw: ra.ra_paged_attend(**{**dict(kv=kv, cache=t["cache"], q=t["q"], page_table=t["table"],
                                                         offset=t["offset"], length=t["length"], stream=stream), **kw}),
        weigh=lambda **kw: ra.ra_paged_weigh(**{**dict(kv=kv, cache=t["cache"], q=t["q"], lse=t["lse"], page_table=t["table"],
                                                       offset=t["offset"], length=t["length"], weight=t["weight"],
                                                       stream=stream), **kw}),
        evict=lambda **kw: ra.ra_paged_evict(**{**dict(kv=kv, cache=t["cache"], page_table=t["table"], length=t["length"],
                                                       weight=t["weight"], keep=4, stream=stream), **kw}),
        rope=lambda **kw: ra.ra_rope(**{**dict(rope=rope, q=t["x"], k=t["y"], stream=stream), **kw}))


def test_the_binding_checks_every_tensor(monkeypatch):
    kv, rope, t = _kv(), ra.ra_rope_plan(128), _tensors()
    calls = _binding_calls(kv, rope, t)
    monkeypatch.setattr(ra, "load_library", lambda: _Library())
    monkeypatch.setattr(ra, "_stream", lambda s: 0)
    monkeypatch.setattr(ra, "_on_current_device", lambda *a: None)
    wrong = dict(
        append=dict(cache=t["cache"][:5], k=t["k"][:, :1], v=t["v"][:2], q=t["q"][:, :2], q_out=t["q"].float(),
                    page_table=t["table"][0], offset=t["offset"][:2], length=t["length"][:1], position=t["position"].long()),
        attend=dict(cache=t["cache"].float(), q=t["q"].transpose(1, 2), o=t["q"][:2], lse=t["lse"].double(),
                    scratch=torch.zeros(1 << 20, dtype=torch.float64), offset=t["offset"].long(), length=t["length"][:1],
                    page_table=t["table"].t()),
        weigh=dict(scratch=torch.zeros(1 << 20, dtype=torch.float64), lse=t["lse"][:2], weight=t["weight"][:1], weight_in=t["weight"][:, :, :5], q=t["x"], cache=t["cache"][:, :1]),
        evict=dict(weight=t["weight"][0], weight_out=t["weight"].bfloat16(), new_table=t["table"][:1], kept=t["lse"],
                   new_length=t["offset"], length=t["offset"], page_table=t["table"].long()),
        rope=dict(q=t["x"][0], k=t["y"][:, :, :4], q_out=t["x"][:, :2], k_out=t["y"].transpose(2, 3), position=t["position"]))
    for name, call in calls.items():
        call()
        for arg, bad in wrong[name].items():
            with pytest.raises(ValueError):
                call(**{arg: bad})
    with pytest.raises(ValueError):
        calls["rope"](k=None, k_out=t["y"])
    with pytest.raises(ValueError):
        calls["append"](q=None, q_out=t["q"])


@pytest.mark.parametrize("name", ["append", "attend", "weigh", "evict", "rope"])
def test_buffers_are_made_on_the_calls_stream(monkeypatch, name):
    inside, made = [], []

    class _Context:
        def __enter__(self):
            inside.append(True)

        def __exit__(self, *exc):
            inside.pop()

    stream = object()
    kv, rope, t = _kv(), ra.ra_rope_plan(128), _tensors()
    monkeypatch.setattr(ra, "load_library", lambda: _Library())
    monkeypatch.setattr(ra, "_alloc_on", lambda s: _Context() if s is stream else pytest.fail("another stream"))
    monkeypatch.setattr(ra, "_stream", lambda s: 0)
    monkeypatch.setattr(ra, "_on_current_device", lambda *a: None)
    for size in ("ra_paged_attend_scratch_size", "ra_paged_weigh_scratch_size"):
        monkeypatch.setattr(ra, size, lambda *a: 4096)
    for fn in ("empty", "empty_like"):
        real = getattr(torch, fn)
        monkeypatch.setattr(torch, fn, lambda *a, real=real, **kw: (made.append(bool(inside)), real(*a, **kw))[1])
    _binding_calls(kv, rope, t, stream)[name]()
    assert made and all(made)


# ------------------------------------------------------------------- the plain forms --
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("scaled", [dict(), dict(scaling="linear", factor=4.0), dict(scaling="base", factor=8.0),
                                    dict(scaling="bands", factor=8.0, original=512, base=500000.0),
                                    dict(scaling="ramp", factor=8.0, original=512, low=1.0, high=32.0)],
                         ids=lambda s: s.get("scaling", "none"))
def test_rotation_gradient_by_differences(interleaved, scaled):
    rng = np.random.default_rng(3)
    x, g, pos = rng.normal(size=(5, 12)), rng.normal(size=(5, 12)), np.array([0, 1, 7, 1000, -3])
    f = lambda x: (paged_ref.rotate(x, pos, 10, interleaved, 1.3, **scaled)[0] * g).sum()
    grad = paged_ref.rotate(g, pos, 10, interleaved, 1.3, transposed=True, **scaled)[0]
    for at in np.ndindex(x.shape):
        step = np.zeros(x.shape)
        step[at] = 1e-3
        # f is linear: the difference is the derivative but for the sums' rounding, 1e-13 / 1e-3
        assert abs((f(x + step) - f(x - step)) / 2e-3 - grad[at]) < 1e-9


def test_rotation_keeps_relative_positions():
    """q at n and k at m: the product depends on n - m alone, in every pairing."""
    rng = np.random.default_rng(4)
    q, k = rng.normal(size=16), rng.normal(size=16)
    for inter in (False, True):
        dot = lambda n, m: paged_ref.rotate(q, n, 16, inter)[0] @ paged_ref.rotate(k, m, 16, inter)[0]
        assert abs(dot(10, 3) - dot(1007, 1000)) < 1e-10


def test_speeds_at_the_ends():
    w = paged_ref.speeds(64, base=10000.0)
    bands = paged_ref.speeds(64, base=10000.0, scaling="bands", factor=8.0, original=4096, low=1.0, high=4.0)
    ramp = paged_ref.speeds(64, base=10000.0, scaling="ramp", factor=8.0, original=4096, low=1.0, high=32.0)
    for s in (bands, ramp):
        assert s[0] == w[0] and np.isclose(s[-1], w[-1] / 8, rtol=1e-15) and (np.diff(s) < 0).all()
    assert np.isclose(paged_ref.speeds(64, scaling="base", factor=8.0)[-1], w[-1] / 8, rtol=1e-12)


def test_weights_sum_to_the_rows():
    """Over all slots a row's weights sum to one; the plain attention of one visible slot is it."""
    rng = np.random.default_rng(5)
    k, v = (torch.from_numpy(rng.normal(size=(2, 9, 8))) for _ in range(2))
    q, slot, j = torch.from_numpy(rng.normal(size=(4, 6, 8))), torch.arange(5, 9), torch.arange(9)
    for window, sinks in ((0, 0), (3, 2), (1, 0)):
        o, lse, _, _ = paged_ref.attend(k, v, q, slot, j, window, sinks, 0.0)
        w, _ = paged_ref.weigh(k, q, lse, slot, j, window, sinks)
        assert torch.allclose(w.sum(-1), torch.full((2,), 12.0, dtype=torch.float64))
        if window == 1:
            assert torch.allclose(o, v.repeat_interleave(3, 0).transpose(0, 1)[5:9])


def test_eviction_order():
    nan, inf = float("nan"), float("inf")
    assert list(paged_ref.evict([5, 1, 1, 1, 2, 0], 6, 4, 1, 1)) == [0, 1, 4, 5]
    assert list(paged_ref.evict([1, nan, -inf, 0, 0.0, -0.0], 6, 3, 0, 0)) == [0, 3, 4]
    assert list(paged_ref.evict([nan, nan, -inf, nan], 4, 2, 0, 0)) == [0, 2]
    assert list(paged_ref.evict([3, 2, 1], 3, 3, 0, 3)) == [0, 1, 2]
    assert list(paged_ref.evict([3, 9, 1, 4], 4, 2, 1, 1)) == [0, 3]
