"""Host-side tests of the 4-bit cache: refusals, sizes, and the reference's own format.
No GPU is needed."""

import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")
ra = pytest.importorskip("context_ring_attention_gb300")
from tests import kv4_ref  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _library():
    import os
    from context_ring_attention_gb300 import build
    if not os.path.exists(ra.library_path()):
        build.build()
    ra.load_library()


def _kv(**kw):
    args = dict(pages=6, page_rows=32, heads_q=4, heads_kv=2, head_dim=128)
    args.update(kw)
    return ra.ra_kv4_plan(**args)


@pytest.mark.parametrize("kw,status", [
    (dict(pages=0), "RA_ERR_INVALID_ARG"), (dict(page_rows=0), "RA_ERR_INVALID_ARG"),
    (dict(page_rows=24), "RA_ERR_INVALID_ARG"), (dict(page_rows=65552), "RA_ERR_INVALID_ARG"),
    (dict(heads_q=3), "RA_ERR_INVALID_ARG"), (dict(heads_kv=0), "RA_ERR_INVALID_ARG"),
    (dict(window=-1), "RA_ERR_INVALID_ARG"), (dict(sinks=-1), "RA_ERR_INVALID_ARG"),
    (dict(scale=float("inf")), "RA_ERR_INVALID_ARG"), (dict(scale=-1.0), "RA_ERR_INVALID_ARG"),
    (dict(dtype=7), "RA_ERR_INVALID_ARG"), (dict(head_dim=0), "RA_ERR_INVALID_ARG"),
    (dict(head_dim=96), "RA_ERR_UNSUPPORTED"), (dict(head_dim=256), "RA_ERR_UNSUPPORTED"),
    (dict(pages=1 << 31), "RA_ERR_UNSUPPORTED"),
    (dict(pages=(1 << 31) - 1, page_rows=65536, heads_q=1 << 20, heads_kv=1 << 20), "RA_ERR_UNSUPPORTED"),
])
def test_refused_descriptions(kw, status):
    with pytest.raises(ra.RaError) as err:
        _kv(**kw)
    assert err.value.name == status


def test_sizes():
    assert ra.ra_kv4_cache_size(_kv()) == 6 * 2 * 32 * 160          # 5 bits a channel, K and V
    assert ra.ra_kv4_cache_size(_kv(head_dim=64)) == 6 * 2 * 32 * 80
    big = _kv(pages=(1 << 31) - 1, page_rows=4096, heads_q=64, heads_kv=64)
    assert ra.ra_kv4_cache_size(big) == ((1 << 31) - 1) * 64 * 4096 * 160


def test_attention_scratch():
    kv = _kv()
    # one split: no scratch; a long table: parts of 8 rows of d floats and two statistics
    assert ra.ra_kv4_attend_scratch_size(kv, 1, 1, 1) == 0
    n = ra.ra_kv4_attend_scratch_size(kv, 1, 1, 4096)
    assert n > 0 and n % (8 * 130 * 4) == 0
    # the window bounds the keys, so also the split
    assert ra.ra_kv4_attend_scratch_size(_kv(window=64, sinks=4), 1, 1, 4096) == 0
    # a window beyond any sequence does not
    assert ra.ra_kv4_attend_scratch_size(_kv(window=1 << 62, sinks=1 << 62), 1, 1, 4096) == n
    for args, status in (((0, 1, 1), "RA_ERR_INVALID_ARG"), ((1, 0, 1), "RA_ERR_INVALID_ARG"),
                         ((1, 1, 0), "RA_ERR_INVALID_ARG"), ((65536, 1, 1), "RA_ERR_UNSUPPORTED"),
                         ((1, 1 << 20, 1), "RA_ERR_UNSUPPORTED"), ((1, 1, (1 << 30) // 32 + 1), "RA_ERR_UNSUPPORTED")):
        with pytest.raises(ra.RaError) as err:
            ra.ra_kv4_attend_scratch_size(kv, *args)
        assert err.value.name == status


def test_refused_calls():
    """Bad pointers and sizes are refused before anything is launched; without a device the
    rest is RA_ERR_NO_DEVICE (with one, a host pointer is RA_ERR_INVALID_ARG)."""
    lib = ra.load_library()
    kv = _kv()
    h = kv.handle
    buf = ctypes.create_string_buffer(4096 + 16)
    a = (ctypes.addressof(buf) + 15) & ~15
    end = 1 if torch.cuda.is_available() else 5
    write = lambda cache=a, b=1, t=1, k=a, v=a, tab=a, w=1, f=a, c=a: lib.ra_kv4_write(h, cache, b, t, k, v, tab, w, f, c, None)
    read = lambda cache=a, b=1, t=1, k=a, v=a, tab=a, w=1, f=a, c=a: lib.ra_kv4_read(h, cache, b, t, tab, w, f, c, 0, k, v, None)
    attend = lambda cache=a, b=1, t=1, q=a, tab=a, w=1, n=a, o=a, lse=a, s=a: lib.ra_kv4_attend(
        h, cache, b, t, q, tab, w, n, o, lse, s, None)
    for call in (write, read):
        assert call() == end and call(c=None) == end
        for bad in (dict(cache=None), dict(k=None), dict(v=None), dict(tab=None), dict(f=None), dict(b=0), dict(t=0),
                    dict(w=0), dict(cache=a + 4), dict(k=a + 8), dict(v=a + 2), dict(tab=a + 2), dict(f=a + 1),
                    dict(c=a + 1)):
            assert call(**bad) == 1, bad
        for big in (dict(t=1 << 31), dict(b=1 << 16, t=1 << 15), dict(w=(1 << 30) // 32 + 1)):
            assert call(**big) == 2, big
    assert attend() == end and attend(lse=None) == end and attend(s=None) == end
    for bad in (dict(cache=None), dict(q=None), dict(tab=None), dict(n=None), dict(o=None), dict(b=0), dict(t=0),
                dict(w=0), dict(q=a + 8), dict(o=a + 4), dict(lse=a + 4), dict(tab=a + 1),
                dict(w=4096, s=None)):  # a long table needs scratch
        assert attend(**bad) == 1, bad
    for big in (dict(b=65536), dict(t=1 << 20), dict(w=(1 << 30) // 32 + 1)):
        assert attend(**big) == 2, big
    for fn in (lib.ra_kv4_cache_size, ):
        assert fn(None, a) == 1 and fn(h, None) == 1
    assert lib.ra_kv4_plan(None, ctypes.byref(ctypes.c_void_p())) == 1
    assert lib.ra_kv4_sync_status(None, None) == 1
    if not torch.cuda.is_available():
        assert lib.ra_kv4_sync_status(h, None) == 5
    assert lib.ra_kv4_destroy(None) == 0


def test_binding_checks_tensors():
    kv = _kv()
    cache = torch.zeros(ra.ra_kv4_cache_size(kv), dtype=torch.uint8)
    table = torch.zeros((1, 2), dtype=torch.int32)
    n = torch.ones(1, dtype=torch.int32)
    k = torch.zeros((1, 2, 3, 128), dtype=torch.bfloat16)
    for call in (lambda: ra.ra_kv4_write(kv, cache, k, k, table, n),             # not CUDA tensors
                 lambda: ra.ra_kv4_write(kv, cache[:-1], k, k, table, n),
                 lambda: ra.ra_kv4_write(kv, cache, k.float(), k, table, n),
                 lambda: ra.ra_kv4_write(kv, cache, k, k, table.long(), n),
                 lambda: ra.ra_kv4_write(kv, cache, k, k, table[0], n),
                 lambda: ra.ra_kv4_read(kv, cache, table, n, 3),
                 lambda: ra.ra_kv4_attend(kv, cache, k[0], table, n)):
        with pytest.raises(ValueError):
            call()


def test_reference_format():
    """The reference on a group worked out by hand, and its error bound: half a step, and
    the bf16 rounding of the two parameters."""
    x = np.zeros((1, 64))
    x[0, :32] = np.arange(32) / 31 * 15  # low 0, scale 1
    codes, scale, low = kv4_ref.quantise(x)
    assert low[0].tolist() == [0, 0] and scale[0].tolist() == [1, 0]
    assert codes[0, 0] == 0 and codes[0, 31] == 15 and codes[0, 1] == 0 and codes[0, 2] == 1
    assert (codes[0, 32:] == 0).all()
    kb, par = kv4_ref.row_bytes(x, True)
    assert par[0].tolist() == [0x80, 0x3f, 0, 0, 0, 0, 0, 0]
    # key channel 9 (code 4): word (9 % 32 // 8) * 2 + 0 = 2, nibble 1 -> byte 8, high half
    assert kb[0, 8] >> 4 == codes[0, 9] == 4
    vb, _ = kv4_ref.row_bytes(x, False)
    # value channel 9: 16-bit word (9 // 4) * 2 + 0 = 4, nibble 1 -> byte 8, high half
    assert vb[0, 8] >> 4 == 4
    rng = np.random.default_rng(3)
    y = rng.normal(size=(50, 128)) * np.exp(rng.normal(size=(50, 1))) + 3
    g = y.reshape(50, 4, 32)
    step = (g.max(-1) - g.min(-1)) / 15
    err = np.abs(kv4_ref.values(y) - y).reshape(g.shape).max(-1)
    assert (err <= step * (0.5 + 15 * 2.0 ** -8) + np.abs(g).max(-1) * 2.0 ** -8 * 2).all()
