"""Buffers that the binding makes for a call belong to the stream the call runs on.

The caching allocator hands a block on in the order of the stream it was made for: an
output of the current stream's, written by kernels on another one, may be memory that the
current stream's queued work still uses."""

import types

import pytest

torch = pytest.importorskip("torch")
ra = pytest.importorskip("context_ring_attention_gb300")

B, H, S, D, N = 1, 4, 8, 128, 2
PROBLEM = dict(batch=B, seq=S, heads_q=H, heads_kv=H, head_dim=D, n_shards=N, dtype=1)


class _Library:
    """Every entry point succeeds and does nothing."""

    def __getattr__(self, name):
        return lambda *args: 0


class _OnDevice(torch.Tensor):
    """A host tensor that passes for a CUDA tensor."""
    is_cuda = True


def _calls(make):
    """(name, call with an explicit stream) for everything that makes a buffer of its own."""
    plan = types.SimpleNamespace(problem=PROBLEM, handle=None, _bwd_scratch=256)
    q, k, v, o, do = (make((B, H, S, D), torch.bfloat16) for _ in range(5))
    lse = make((B, H, S), torch.float32)
    parts, lse_parts = make((N, B, H, S, D), torch.float32), make((N, B, H, S), torch.float32)
    return [
        ("fwd", lambda s: ra.ra_fwd(plan, q, k, v, stream=s)),
        ("partials", lambda s: ra.ra_fwd(plan, q, k, v, partials=True, stream=s)),
        ("merge", lambda s: ra.ra_merge_partials(parts, lse_parts, stream=s)),
        ("perm", lambda s: ra.ra_layout_perm(q, "zigzag", N, stream=s)),
        ("static", lambda s: ra.ra_fwd_static(B, S, H, H, N, "zigzag", True, q, k, v, stream=s)),
        ("step", lambda s: ra.ra_fwd_step(plan, 0, q, k, v, stream=s)),
        ("rotate", lambda s: ra.ra_ring_rotate(plan, k, v, stream=s)),
        ("ring", lambda s: ra.ra_ring_fwd(plan, q, k, v, stream=s, comm_stream=s)),
        ("bwd", lambda s: ra.ra_bwd(plan, q, k, v, o, lse, do, stream=s)),
        ("allgather", lambda s: ra.ra_allgather_kv(plan, k, v, stream=s)),
        ("gathered", lambda s: ra.ra_fwd_gathered(plan, q, k, v, stream=s)),
        ("ulysses", lambda s: ra.ra_ulysses_a2a(q, "zigzag", N, 0, stream=s)),
    ]


NAMES = [name for name, _ in _calls(lambda shape, dtype: None)]


@pytest.mark.parametrize("name", NAMES)
def test_buffers_are_made_on_the_calls_stream(monkeypatch, name):
    inside, made = [], []

    class _Context:
        def __enter__(self):
            inside.append(True)

        def __exit__(self, *exc):
            inside.pop()

    stream = object()
    monkeypatch.setattr(ra, "load_library", lambda: _Library())
    monkeypatch.setattr(ra, "_alloc_on", lambda s: _Context() if s is stream else pytest.fail("another stream"))
    monkeypatch.setattr(ra, "_stream", lambda s: 0)
    for check in ("_check_qkv", "_need", "_need_like", "_same_device", "_on_current_device"):
        monkeypatch.setattr(ra, check, lambda *a, **kw: None)
    calls = dict(_calls(lambda shape, dtype: torch.zeros(shape, dtype=dtype).as_subclass(_OnDevice)))
    for fn in ("empty", "empty_like"):
        real = getattr(torch, fn)
        monkeypatch.setattr(torch, fn, lambda *a, real=real, **kw: (made.append(bool(inside)), real(*a, **kw))[1])
    calls[name](stream)
    assert made and all(made)


@pytest.mark.gpu
def test_outputs_do_not_take_the_current_streams_memory():
    """A block freed on the current stream is not an output of a call on another."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    plan = ra.ra_plan(1, 512, 4, 2, 128, 2, "zigzag", True, "bf16")
    win = ra.ra_plan_window(1, 512, 4, 2, 128, 2, 100, 4, layout="zigzag")
    q, k, v, do = (torch.randn((1, h, 512, 128), device="cuda").bfloat16() for h in (4, 2, 2, 4))
    o, lse = ra.ra_fwd(plan, q, k, v)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for p in (plan, win):
        free = [torch.empty_like(q) for _ in range(8)] + [torch.empty_like(k) for _ in range(8)] + \
               [torch.empty_like(lse) for _ in range(8)]
        blocks = {t.data_ptr() for t in free}
        del free
        outs = ra.ra_fwd(p, q, k, v, stream=side) + ra.ra_bwd(p, q, k, v, o, lse, do, stream=side)
        assert not blocks & {t.data_ptr() for t in outs}
        side.synchronize()
        del outs
        ra.ra_sync_status(p, side)
