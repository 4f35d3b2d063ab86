"""The 4-bit cache's format and the attention over it in plain form: float64 and byte
arithmetic of its own, written from the definition in include/ra.h."""

import numpy as np
import torch

from tests.window_ref import BF16_U, F32_U, visible


def bf16(x):
    """float64 -> the nearest bf16 by way of float32, as float64 (both roundings to even)."""
    with np.errstate(over="ignore", invalid="ignore"):
        return torch.from_numpy(np.asarray(x, np.float64).astype(np.float32)).bfloat16().double().numpy()


def quantise(x):
    """x [..., d] float64 -> codes [..., d], scale and low [..., d/32]."""
    g = x.reshape(x.shape[:-1] + (-1, 32))
    with np.errstate(over="ignore", invalid="ignore"):
        low = bf16(g.min(-1))
        span = (g.max(-1) - low).astype(np.float32)
        scale = bf16(span * (np.float32(1) / np.float32(15)))  # a float32 product
        bad = ~(np.isfinite(g).all(-1) & np.isfinite(scale) & np.isfinite(low))
        scale = np.where(bad | (scale < 2.0 ** -100), 0.0, scale)
        codes = np.zeros(g.shape, np.int64)
        for n in range(15):  # the borders, each one exact in float64
            codes += (g - low[..., None] >= (n + 0.5) * scale[..., None]) & (scale[..., None] > 0)
    codes[bad] = 0
    low = np.where(bad, np.nan, low)
    return codes.reshape(x.shape), scale, low


def row_bytes(x, key):
    """The code bytes [..., d/2] and parameter bytes [..., d/8] of rows x [..., d]."""
    codes, scale, low = quantise(x)
    d = x.shape[-1]
    c = np.arange(d)
    if key:
        nibble = (c % 32 // 8 * (d // 32) + c // 32) * 8 + c % 8
    else:
        nibble = (c % 32 // 4 * (d // 32) + c // 32) * 4 + c % 4
    out = np.zeros(x.shape[:-1] + (d // 2,), np.uint8)
    for ch in range(d):
        out[..., nibble[ch] // 2] |= (codes[..., ch] << (4 * (nibble[ch] % 2))).astype(np.uint8)
    par = np.stack([scale, low], -1).astype(np.float32).view(np.uint32) >> 16
    par = np.where(np.isnan(np.stack([scale, low], -1)), 0x7fff, par).astype("<u2")
    return out, np.ascontiguousarray(par).view(np.uint8).reshape(x.shape[:-1] + (d // 8,))


def values(x):
    codes, scale, low = quantise(x)
    return np.repeat(low, 32, -1) + np.repeat(scale, 32, -1) * codes


class Cache:
    """A cache of bytes and what it stands for, filled row by row."""

    def __init__(self, pages, page_rows, heads, d, fill=0xAB):
        self.shape = (pages, page_rows, heads, d)
        self.bytes = np.full((pages, heads, page_rows // 16, 20 * d), fill, np.uint8)
        self.k = np.full((pages, heads, page_rows, d), np.nan)
        self.v = np.full((pages, heads, page_rows, d), np.nan)

    def write(self, k, v, table, first, count):
        d = self.shape[3]
        cut = (0, 8 * d, 10 * d, 18 * d, 20 * d)
        for n, (x, key, store) in enumerate(((k, True, self.k), (v, False, self.v))):
            codes, par = row_bytes(x, key)
            vals = values(x)
            for b in range(x.shape[0]):
                for t in range(int(count[b])):
                    pos = int(first[b]) + t
                    page, row = int(table[b][pos // self.shape[1]]), pos % self.shape[1]
                    blk = self.bytes[page, :, row // 16]
                    blk[:, cut[2 * n]:cut[2 * n + 1]].reshape(-1, 16, d // 2)[:, row % 16] = codes[b, :, t]
                    at = cut[2 * n + 1] + row % 16 * (d // 8)
                    blk[:, at:at + d // 8] = par[b, :, t]
                    store[page, :, row] = vals[b, :, t]

    def rows(self, table_row, positions):
        """(k, v) [heads, n, d] of one sequence's positions."""
        pages = np.asarray(table_row)[positions // self.shape[1]]
        rows = positions % self.shape[1]
        return self.k[pages, :, rows].transpose(1, 0, 2), self.v[pages, :, rows].transpose(1, 0, 2)




def attend(k, v, q, length, window, sinks, u, scale=None):
    """One sequence: q [Hq, T, d], k and v [Hkv, n, d] (the values, positions 0..n-1) ->
    O, LSE and their bounds.

    Bounds (see window_ref.py): a score is a sum over groups of scale * (q . codes) plus
    (low + 8 scale) * (sum of q), each in fp32: off by 2^-16 of the magnitudes in it, where
    a code's magnitude is up to 8 scales and the middle's another 8 (at most the group's
    span and its offset); P times a scale is rounded to bf16 (u), so O is off by u times the
    sum of P * |scale * (code - 8)|, at most P * (span + |v|), and by u of its own.  float32: three
    terms leave 2^-24, and the exponent, of magnitude up to 2^7, is off by 2^-24 of itself.
    """
    hq, t, d = q.shape
    g = hq // k.shape[0]
    k, v, q = (torch.as_tensor(np.asarray(x, np.float64)) for x in (k, v, q))
    k, v = k.repeat_interleave(g, 0), v.repeat_interleave(g, 0)
    scale = d ** -0.5 if scale is None else scale
    pos_q = torch.arange(length - t, length)
    vis = visible(pos_q, torch.arange(k.shape[1]), window or 1 << 40, sinks)
    s = (q @ k.transpose(-1, -2) * scale).masked_fill(~vis, -torch.inf)

    def reach(x):  # per row and channel: the span and offset of its group
        y = x.abs().unflatten(-1, (-1, 32)).amax(-1, keepdim=True)
        return (3 * y).expand(*y.shape[:-1], 32).flatten(-2)

    mag = (q.abs() @ reach(k).transpose(-1, -2) * scale).masked_fill(~vis, 0.0)
    mag = mag.amax(-1) if mag.shape[-1] else mag.sum(-1)
    lse = torch.logsumexp(s, -1) if s.shape[-1] else torch.full((hq, t), -torch.inf, dtype=torch.float64)
    p = torch.where(vis, torch.exp(s - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[..., None]), 0.0)
    o = p @ v
    e = 2.0 ** -15 * (1 + mag) + s.shape[-1] * 2.0 ** -23
    o_bound = (u + 2 * e[..., None]) * (p @ reach(v)) + u * o.abs()
    return o, lse, o_bound, e


U = {"bf16": BF16_U, "f32": F32_U}
