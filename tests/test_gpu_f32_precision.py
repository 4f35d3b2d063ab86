"""What float32 plans and float32 caches keep of their inputs' 24 bits.

The bounds of window_ref.py and kv4_ref.py are those of bf16 kernels with a smaller
rounding of the outputs; these are the float32 kernels' own, and inputs are chosen so that
a bf16 term too few (2^-17 of a query or a weight) lies far outside of them.

Roundings: u = 2^-24 each; ex2.approx and expf are off by 2^-22 at most, logarithms by as much.
"""

import numpy as np
import pytest

import oracle

torch = pytest.importorskip("torch")
ra = pytest.importorskip("context_ring_attention_gb300")
from context_ring_attention_gb300 import workloads  # noqa: E402
from tests import window_ref  # noqa: E402
from tests.window_ref import assert_within  # noqa: E402

pytestmark = pytest.mark.gpu
LOG2E, U = 1.4426950408889634, 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ra.load_library()


def _two_terms(x):
    """float64 -> what two bf16 terms of it hold."""
    x = torch.as_tensor(x, dtype=torch.float32)
    a = x.bfloat16().float()
    return (a + (x - a).bfloat16().float()).double()


def _cached(k, v, hq, log2_scale):
    """A float32 cache of one sequence with the rows k, v [tokens, d] and scores in units of
    log2_scale (a power of two, which the kernel's product of scale and log2(e) returns exactly)."""
    scale = np.float32(log2_scale / LOG2E)
    assert np.float32(scale * np.float32(LOG2E)) == np.float32(log2_scale)
    kv = ra.ra_kv4_plan(1, 16, hq, 1, k.shape[1], dtype="f32", scale=float(scale))
    cache = torch.zeros(ra.ra_kv4_cache_size(kv), dtype=torch.uint8, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    rows = [torch.as_tensor(x, dtype=torch.float32, device="cuda")[None, None].contiguous() for x in (k, v)]
    ra.ra_kv4_write(kv, cache, *rows, i32([[0]]), i32([0]))
    back = ra.ra_kv4_read(kv, cache, i32([[0]]), i32([0]), k.shape[0])
    for x, y in zip(rows, back):
        assert torch.equal(x, y)  # the rows are what their codes stand for
    return lambda q: ra.ra_kv4_attend(kv, cache, torch.as_tensor(q, dtype=torch.float32, device="cuda")[None, :, None],
                                      i32([[0]]), i32([k.shape[0]])), kv


@pytest.mark.parametrize("log2_scale", [2.0, 2.0 ** -5])
@pytest.mark.parametrize("hq", [4, 64])
@pytest.mark.parametrize("d", [64, 128])
def test_cache_scores_keep_the_querys_24_bits(d, hq, log2_scale):
    """One key, whose code n meets one channel x of a query: LSE = log2_scale ln(2) x n.

    The score: x n in three products summed in fp32 (two additions, each off by 2^-23 of the
    sum at most), then two roundings (u); the exponential of 0 and the logarithm of 1 add 2^-22
    each and the last product u."""
    n = np.tile(np.arange(16), d // 16)  # groups of 0..15 twice: low 0, scale 1
    attend, kv = _cached(n[None].astype(np.float64), n[None].astype(np.float64), hq, log2_scale)
    rng = np.random.default_rng(hq)
    x = (1 + rng.random(hq)).astype(np.float32).astype(np.float64)
    at = (np.arange(hq) * 5 + 15) % d  # the channel that a head's query holds
    q = np.zeros((hq, d))
    q[np.arange(hq), at] = x
    o, lse = attend(q)
    ra.ra_kv4_sync_status(kv)
    s = log2_scale * x * n[at]
    want = s * np.log(2)
    bound = np.abs(s) * (2 * 2.0 ** -23 + 3 * U) + 2 * 2.0 ** -22
    short = log2_scale * np.abs(_two_terms(x).numpy() - x) * n[at] * np.log(2)
    assert (short > 2 * bound).any()  # two terms would be seen
    assert_within(lse[0, :, 0].cpu(), torch.as_tensor(want), torch.as_tensor(bound), "LSE")
    # the one key's weight is 1: its values, each code times the scale 1 and the centring by 8
    assert_within(o[0, :, 0].cpu(), torch.as_tensor(np.tile(n, (hq, 1))).double(), torch.tensor(2.0 ** -18), "O")


@pytest.mark.parametrize("hq", [4, 16])
@pytest.mark.parametrize("d", [64, 128])
def test_cache_weights_keep_24_bits(d, hq):
    """Two keys, the second one's weight p = 2^-(5 h / 16) of the first's, whose values are zeros
    (a group of scale 0, no products): at channels whose code is 0, 8 below the middle, which
    is 0, O = -8 p / (1 + p).

    The exponents' arguments are exact (small multiples of 1/16); p is off by 2^-22 in the sum
    of the products and in that of the weights; -8 times its three terms is exact in fp32; the
    weights' sum, the quotient and the outcome add three roundings."""
    k = np.zeros((2, d))
    k[0] = np.arange(d) % 16
    k[1] = np.where(np.arange(d) % 32 == 7, 2, np.arange(d) % 16)  # channel 7: code 7, then 2
    v = np.zeros((2, d))
    v[1] = np.arange(d) % 16 - 8
    attend, kv = _cached(k, v, hq, 2.0 ** -4)
    h = np.arange(1, hq + 1)
    q = np.zeros((hq, d))
    q[:, 7] = h
    o, lse = attend(q)
    ra.ra_kv4_sync_status(kv)
    p = 2.0 ** (-5 * h / 16)
    want = -8 * p / (1 + p)
    bound = np.abs(want) * (2 * 2.0 ** -22 + 3 * U)
    p32 = p.astype(np.float32).astype(np.float64)
    short = np.abs(_two_terms(p32).numpy() - p32) / p * np.abs(want)
    assert (short > 2 * bound).any()  # two terms would be seen
    code0 = (np.arange(d) % 16 == 0).nonzero()[0]
    assert_within(o[0, :, 0, torch.as_tensor(code0)].cpu(), torch.as_tensor(np.repeat(want[:, None], len(code0), 1)),
                  torch.as_tensor(bound)[:, None], "O")
    ln = (7 * h / 16 + np.log2(1 + p)) * np.log(2)
    assert_within(lse[0, :, 0].cpu(), torch.as_tensor(ln), torch.as_tensor(np.abs(ln) * 3 * U + 4 * 2.0 ** -22), "LSE")


@pytest.mark.parametrize("tokens,t,hq", [(2, 1, 3), (16, 3, 8), (700, 1, 4), (700, 9, 2)])
@pytest.mark.parametrize("d", [64, 128])
def test_cache_attention_in_float32(d, tokens, t, hq):
    """Ordinary inputs, the values being those that the cache reads back.

    A score: 3 d products and d / 32 group sums, each addition off by 2^-23 of the magnitudes,
    which are those of codes times the scale and of low, up to three times a group's largest value;
    the weights' arguments round by u of the score's range; a weight by 2^-22 and (three terms) u;
    the sums of O over blocks of 16 tokens and of their 5 products, with the offset of 8 codes."""
    rng = np.random.default_rng(tokens + t)
    page = 64
    kv = ra.ra_kv4_plan(-(-tokens // page), page, hq, 1, d, dtype="f32")
    cache = torch.zeros(ra.ra_kv4_cache_size(kv), dtype=torch.uint8, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    k, v = (torch.as_tensor(rng.normal(size=(1, 1, tokens, d)), dtype=torch.float32, device="cuda") for _ in range(2))
    table = i32([list(range(-(-tokens // page)))])
    ra.ra_kv4_write(kv, cache, k, v, table, i32([0]))
    k, v = (x[0].double() for x in ra.ra_kv4_read(kv, cache, table, i32([0]), tokens))  # (values exact in float32)
    q = torch.as_tensor(rng.normal(size=(1, hq, t, d)), dtype=torch.float32, device="cuda")
    o, lse = ra.ra_kv4_attend(kv, cache, q, table, i32([tokens]))
    ra.ra_kv4_sync_status(kv)
    vis = window_ref.visible(torch.arange(tokens - t, tokens), torch.arange(tokens), 1 << 40, 0).cuda()
    x = (q[0].double() @ k.transpose(-1, -2) * d ** -0.5).masked_fill(~vis, -torch.inf)
    lw = torch.logsumexp(x, -1)
    p = torch.exp(x - lw[..., None])
    reach = lambda y: (3 * y.abs().unflatten(-1, (-1, 32)).amax(-1, keepdim=True)).expand(*y.shape[:-1], d // 32, 32).flatten(-2)
    mag = (q[0].double().abs() @ reach(k).transpose(-1, -2) * d ** -0.5).masked_fill(~vis, 0.0).amax(-1)
    # Additions by magnitude: the products of a score are added 16 at a time (exactly but for the
    # sum's 2^-23), 12 sums a group, then the groups' and the low's: 60 of 2^-23 at most.
    e = mag * 60 * 2.0 ** -23 + 2 * U * mag + 2 * 2.0 ** -22 + tokens / 16 * U
    assert_within(lse[0], lw, e + 3 * U * lw.abs(), "LSE")
    assert_within(o[0], p @ v, (2 * e + 2 * U)[..., None] * (p @ v.abs())
                  + (5 * tokens / 16 + 16) * 2.0 ** -23 * (p @ reach(v)), "O")


@pytest.mark.parametrize("layout", oracle.LAYOUTS)
@pytest.mark.parametrize("d", [13, 32, 128])
@pytest.mark.parametrize("window,sinks", [(1, 0), (17, 2), (1, 1000), (1000, 0)])
def test_windowed_plans_in_float32(layout, d, window, sinks):
    """Forward (fused, gathered, partials and their merge) and gradients, each sum bounded by its
    own number of fp32 roundings: d products of a score, n keys of a row (and n / 32 rescales)."""
    b, s, hq, hk, n = 2, 96, 4, 2, 4
    q, k, v = workloads.small_inputs(b, s, hq, hk, d, seed=d, device="cuda", dtype="f32")
    do = torch.randn(q.shape, generator=torch.Generator(device="cuda").manual_seed(d), device="cuda")
    pos = torch.from_numpy(oracle.layout_positions(layout, s, n)).cuda()
    plan = ra.ra_plan_window(b, s, hq, hk, d, n, window, sinks, layout=layout, dtype="f32")
    vis, scale, g = window_ref.visible(pos, pos, window, sinks), d ** -0.5, hq // hk
    q64, do64 = q.double(), do.double()
    k64, v64 = (x.double().repeat_interleave(g, 1) for x in (k, v))
    x = q64 @ k64.transpose(-1, -2) * scale
    mag = (q64.abs() @ k64.abs().transpose(-1, -2) * scale).masked_fill(~vis, 0.0).amax(-1, keepdim=True)
    lw = torch.logsumexp(x.masked_fill(~vis, -torch.inf), -1)
    p = torch.exp(x - lw[..., None]).masked_fill(~vis, 0.0)
    ow = p @ v64
    # a score: d fused products and the scale's product and own rounding; the exponent's argument:
    # up to 2 mag, two roundings; the row sum: n terms and 3 roundings at each of n / 32 rescales
    e = U * ((d + 2) * mag + 4 * mag) + 2 * 2.0 ** -22 + (s + 3 * s / 32) * U
    # (a merge of n partials: the same sums again, each with an exponential and a logarithm)
    for what, more, (o, lse) in (
            ("fused", 0.0, ra.ra_fwd(plan, q, k, v)),
            ("gathered", 0.0, ra.ra_fwd_gathered(plan, q, *ra.ra_allgather_kv(plan, k, v))),
            ("merged", 4 * 2.0 ** -22 + n * U + 4 * U * lw.abs()[..., None],
             ra.ra_merge_partials(*ra.ra_fwd(plan, q, k, v, partials=True)))):
        assert_within(lse, lw, (e + more)[..., 0] + 2 * U * lw.abs(), what + " LSE")
        assert_within(o, ow, (2 * (e + more) + (s + 2) * U) * (p @ v64.abs()) + 2 * U * ow.abs(), what + " O")
    o, lse = ra.ra_fwd(plan, q, k, v)
    grads = ra.ra_bwd(plan, q, k, v, o, lse, do)
    ra.ra_sync_status(plan)
    o64, l64 = o.double(), lse.double()[..., None]
    p = torch.exp(x - l64).masked_fill(~vis, 0.0)
    delta = (o64 * do64).sum(-1, keepdim=True)
    ds = p * (do64 @ v64.transpose(-1, -2) - delta)
    # 2^(score * scale log2(e) - LSE log2(e)): the factors' and the products' roundings and the sum's
    e = U * ((d + 2) * mag + 4 * (mag + l64.abs())) + 2 * 2.0 ** -22
    inner = do64.abs() @ v64.abs().transpose(-1, -2) + (o64 * do64).abs().sum(-1, keepdim=True)
    ds_err = (e + 2 * U) * ds.abs() + (d + 2) * U * p * inner
    m = g * s * U
    per_kv = lambda t: t.view(b, hk, g, s, d).sum(2)
    want = scale * ds @ k64, per_kv(scale * ds.transpose(-1, -2) @ q64), per_kv(p.transpose(-1, -2) @ do64)
    bound = (scale * (ds_err + m * ds.abs()) @ k64.abs(), per_kv(scale * (ds_err + m * ds.abs()).transpose(-1, -2) @ q64.abs()),
             per_kv(((e + m) * p).transpose(-1, -2) @ do64.abs()))
    for name, got, w, b_ in zip(("dQ", "dK", "dV"), grads, want, bound):
        assert_within(got, w, b_ + 3 * U * w.abs(), name)
