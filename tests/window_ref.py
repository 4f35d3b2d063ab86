"""Windowed attention and its gradients in float64, with the error bounds of the kernels.

visible(i, j) = j <= i and (j > i - window or j < sinks) on natural positions; tensors
are [B, H, S, d] in any row order, ``pos`` gives each row's position.

Bounds, element by element, from the arithmetic of the bf16 kernels (u = 2^-8, the
relative error of one rounding to bf16; inputs are exact):
- a score or a dP entry is a sum of 128 exact products accumulated in fp32: off by at
  most 128 * 2^-23 = 2^-16 of the sum of the products' magnitudes (truncating adders);
- P = 2^(..) is then off by a relative e = 2^-15 * (1 + largest sum of magnitudes of the
  row): twice the score's error and the exponential's and the row sum's few 2^-22;
- O = sum P v / l: P enters rounded (u), the output is rounded (u);
- the LSE (fp32) is off by e;
- dV = sum P dO: P rounded (u + e), the output rounded (u);
- dS = P (dP - D) is rounded once (u + e), and dP - D is off by 2^-15 of the magnitudes
  in it; dQ and dK sum it with exact K and Q and are rounded (u);
- the fp32 accumulation of n terms: n * 2^-23 of their magnitudes.
float32 kernels: u = 2^-24 and the same sums (their exponential is off by a few 2^-24).
"""

import torch

BF16_U = 2.0 ** -8
F32_U = 2.0 ** -24


def visible(pos_q, pos_k, window, sinks):
    gap = pos_q[:, None] - pos_k[None, :]
    return (gap >= 0) & ((gap < window) | (pos_k[None, :] < sinks))


def _expand(x, group):
    return x.repeat_interleave(group, 1)


def forward(q, k, v, pos, window, sinks, u):
    """(O, LSE, bound of O, bound of LSE) in float64."""
    g = q.shape[1] // k.shape[1]
    q, k, v = q.double(), _expand(k.double(), g), _expand(v.double(), g)
    scale = q.shape[-1] ** -0.5
    vis = visible(pos, pos, window, sinks)
    s = (q @ k.transpose(-1, -2) * scale).masked_fill(~vis, -torch.inf)
    mag = (q.abs() @ k.abs().transpose(-1, -2) * scale).masked_fill(~vis, 0.0).amax(-1)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse[..., None])
    o = p @ v
    e = 2.0 ** -15 * (1 + mag) + s.shape[-1] * 2.0 ** -23
    o_bound = (u + 2 * e[..., None]) * (p @ v.abs()) + u * o.abs()
    return o, lse, o_bound, e


def backward(q, k, v, o, lse, do, pos, window, sinks, u):
    """(dQ, dK, dV) and their bounds in float64, from the forward's own O and LSE."""
    hk = k.shape[1]
    g = q.shape[1] // hk
    b, hq, s_len, d = q.shape
    q, o, do, lse = q.double(), o.double(), do.double(), lse.double()
    k, v = _expand(k.double(), g), _expand(v.double(), g)
    scale = d ** -0.5
    vis = visible(pos, pos, window, sinks)
    s = q @ k.transpose(-1, -2) * scale
    mag = (q.abs() @ k.abs().transpose(-1, -2) * scale).masked_fill(~vis, 0.0).amax(-1, keepdim=True)
    p = torch.exp(s - lse[..., None]).masked_fill(~vis, 0.0)
    delta = (o * do).sum(-1, keepdim=True)
    ds = p * (do @ v.transpose(-1, -2) - delta)
    e = 2.0 ** -15 * (1 + mag) + s_len * 2.0 ** -23
    inner = do.abs() @ v.abs().transpose(-1, -2) + (o * do).abs().sum(-1, keepdim=True)
    ds_err = (u + e) * ds.abs() + 2.0 ** -15 * p * inner
    p_err = (u + e) * p
    per_kv = lambda x: x.view(b, hk, g, s_len, d).sum(2)
    dq = scale * ds @ k
    dk = per_kv(scale * ds.transpose(-1, -2) @ q)
    dv = per_kv(p.transpose(-1, -2) @ do)
    n = g * s_len * 2.0 ** -23
    dq_b = scale * (ds_err + n * ds.abs()) @ k.abs() + u * dq.abs()
    dk_b = per_kv(scale * (ds_err + n * ds.abs()).transpose(-1, -2) @ q.abs()) + u * dk.abs()
    dv_b = per_kv((p_err + n * p).transpose(-1, -2) @ do.abs()) + u * dv.abs()
    return (dq, dk, dv), (dq_b, dk_b, dv_b)


def assert_within(got, want, bound, what):
    """|got - want| <= bound everywhere, infinities equal."""
    got = got.double()
    assert torch.equal(torch.isneginf(got), torch.isneginf(want)), f"{what}: -inf pattern differs"
    fin = torch.isfinite(want)
    assert torch.isfinite(got[fin]).all(), f"{what}: non-finite values"
    over = (got - want).abs()[fin] - bound.expand_as(want)[fin]
    if over.numel():
        assert over.max() <= 1e-30, f"{what}: off by {over.max().item():.3e} more than its bound"
