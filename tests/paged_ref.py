"""Rotary positions, the paged cache and what is done with it in plain float64 form, written from
the definitions in include/ra.h, with the error bounds of the kernels.

Bounds, element by element (u: half a step of the dtype, 2^-8 bf16, 2^-24 float32; inputs exact):
- a rotation's cosine and sine are off by 2^-21 of the amplitude: the angle by 2^-33 of a turn
  and by half a step of a float below pi/4 (2^-25), the functions by a step or two (2^-23), the
  amplitude's product by half a one; the two products and their sum add 2^-23 of their magnitudes;
  the result is rounded (u); far positions: the float64 angle here and the speed there are each
  off by 2^-52 of the angle;
- a score is a sum of d exact products in fp32 (bf16) or of d fused steps (float32): off by at
  most 128 * 2^-23 = 2^-16 of the magnitudes, and its product by the scale by 2^-23 more;
- P is then off by a relative e = 2^-15 * (1 + largest sum of magnitudes of the row) and by the
  exponential's and the sum's 2^-23 a term;
- O = sum P v / l: P enters rounded (u), the output is rounded (u); the LSE is off by e;
- a slot's weight, a sum over n rows of e^(score - LSE): off by e and n * 2^-23 of itself, and by
  half a step of |LSE| and |score| in the exponent, which e holds.
"""

import math

import numpy as np
import torch

from tests.window_ref import BF16_U, F32_U

U = {"bf16": BF16_U, "f32": F32_U}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------- rotary positions --
def speeds(rot, base=10000.0, scaling="none", factor=1.0, original=0, low=1.0, high=4.0):
    j = np.arange(rot // 2, dtype=np.float64)
    if scaling == "base" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    w = base ** (-2 * j / rot)
    if scaling == "linear":
        return w / factor
    if scaling == "bands":
        t = np.clip((original * w / (2 * np.pi) - low) / (high - low), 0, 1)
        return t * w + (1 - t) * w / factor
    if scaling == "ramp":
        at = lambda turns: rot * math.log(original / (2 * np.pi * turns)) / (2 * math.log(base))
        j0, j1 = max(math.floor(at(high)), 0), min(math.ceil(at(low)), rot - 1)
        t = np.clip((j - j0) / (j1 - j0 if j1 != j0 else 0.001), 0, 1)
        return (1 - t) * w + t * w / factor
    return w


def rotate(x, pos, rot, interleaved=False, amplitude=1.0, transposed=False, **scaled):
    """x [..., d] at positions pos [...] (broadcast against x[..., 0]) -> (y, bound without the
    output's rounding), float64."""
    x = np.asarray(x, np.float64)
    a = np.asarray(pos, np.float64)[..., None] * speeds(rot, **scaled)
    c, s = amplitude * np.cos(a), amplitude * np.sin(a)
    if transposed:
        s = -s
    one, two = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    y, b = x.copy(), np.zeros(x.shape)
    x1, x2 = x[..., one], x[..., two]
    y[..., one], y[..., two] = x1 * c - x2 * s, x1 * s + x2 * c
    b[..., one] = b[..., two] = amplitude * (np.abs(x1) + np.abs(x2)) * (2.0 ** -21 + 2.0 ** -23 + 2.0 ** -51 * np.abs(a))
    return y, b


# ------------------------------------------------------------------ the paged cache --
class Cache:
    """A pool of pages with scattered page tables for sequences of the given lengths.  Entries of
    the tables behind the last page name one outside the pool, and everything that no sequence
    wrote is NaN."""

    def __init__(self, rng, lengths, page_rows, heads_kv, d, dtype, spare=2, extra=1, junk=None):
        used = [-(-n // page_rows) for n in lengths]
        self.pages = sum(used) + spare
        self.width = max(1, max(used) + extra)
        self.page_rows, self.heads_kv, self.d, self.dtype = page_rows, heads_kv, d, dtype
        order = rng.permutation(self.pages)
        self.table = np.full((len(lengths), self.width), self.pages + 5)
        at = 0
        for b, n in enumerate(used):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.free = order[at:]
        self.data = torch.full((self.pages, 2, heads_kv, page_rows, d), math.nan if junk is None else junk, dtype=DT[dtype])
        for b, n in enumerate(lengths):
            self.put(b, np.arange(n), *(self.random(rng, n) for _ in range(2)))

    def random(self, rng, n):
        """Rows [n, heads_kv, d] whose channels have sizes and offsets of their own."""
        x = rng.normal(size=(n, self.heads_kv, self.d)) * np.exp(0.3 * rng.normal(size=self.d)) + 0.3 * rng.normal(size=self.d)
        return torch.from_numpy(x).to(DT[self.dtype])

    def place(self, b, slots):
        slots = np.asarray(slots, np.int64)
        return torch.from_numpy(self.table[b][slots // self.page_rows].astype(np.int64)), torch.from_numpy(slots % self.page_rows)

    def put(self, b, slots, k, v):
        page, row = self.place(b, slots)
        self.data[page, 0, :, row], self.data[page, 1, :, row] = k, v

    def rows(self, b, slots, which):
        """[heads_kv, n, d] float64."""
        page, row = self.place(b, slots)
        return self.data[page, which, :, row].transpose(0, 1).double()


def sees(slot, j, window, sinks):
    """[tokens, slots]: j <= slot and (no window, or j > slot - window, or j < sinks)."""
    slot, j = torch.as_tensor(slot)[:, None], torch.as_tensor(j)[None]
    return (j <= slot) & ((j > slot - window) | (j < sinks)) if window else j <= slot


def _scores(k, q, slot, j, window, sinks, scale):
    """Scores [Hq, T, n] (-inf unseen), which are seen, largest sum of magnitudes per row."""
    t, hq, d = q.shape
    k = k.repeat_interleave(hq // k.shape[0], 0)
    q = q.double().transpose(0, 1)
    vis = sees(slot, j, window, sinks)
    s = (q @ k.transpose(-1, -2) * scale).masked_fill(~vis, -math.inf)
    mag = (q.abs() @ k.abs().transpose(-1, -2) * scale).masked_fill(~vis, 0.0)
    return s, vis, mag.amax(-1) if mag.shape[-1] else mag.sum(-1)


def attend(k, v, q, slot, j, window, sinks, u, scale=None):
    """One sequence: q [T, Hq, d] at slots `slot`, rows k, v [Hkv, n, d] float64 of the slots j ->
    O [T, Hq, d], LSE [T, Hq] and their bounds."""
    t, hq, d = q.shape
    s, vis, mag = _scores(k, q, slot, j, window, sinks, d ** -0.5 if scale is None else scale)
    v = torch.where(vis.any(0)[:, None], v, 0.0).repeat_interleave(hq // v.shape[0], 0)
    lse = torch.logsumexp(s, -1) if s.shape[-1] else torch.full((hq, t), -math.inf, dtype=torch.float64)
    p = torch.exp(s - torch.where(torch.isinf(lse), 0.0, lse)[..., None])
    o = p @ v
    e = 2.0 ** -15 * (1 + mag) + s.shape[-1] * 2.0 ** -23
    bound = (u + 2 * e[..., None]) * (p @ v.abs()) + u * o.abs()
    return tuple(x.transpose(0, 1) for x in (o, lse, bound, e))


def weigh(k, q, lse, slot, j, window, sinks, scale=None):
    """Weights [Hkv, n] that the slots j receive from q [T, Hq, d] with lse [T, Hq], and their bound."""
    t, hq, d = q.shape
    s, vis, mag = _scores(k, q, slot, j, window, sinks, d ** -0.5 if scale is None else scale)
    l = lse.double().transpose(0, 1)[..., None]
    p = torch.where(vis, torch.exp(s - torch.where(vis, l, 0.0)), 0.0)
    e = 2.0 ** -15 * (1 + mag[..., None]) + (t * hq // k.shape[0]) * 2.0 ** -23 + 2.0 ** -22 * torch.where(vis, l.abs(), 0.0)
    per_kv = lambda x: x.unflatten(0, (k.shape[0], -1)).sum((1, 2))
    return per_kv(p), per_kv(p * e)


def evict(weight, length, keep, first, recent):
    """Slots that stay, in order: weight [n] as the kernel takes it."""
    if length <= keep:
        return np.arange(length)
    w = np.asarray(weight, np.float64)[:length]
    w = np.where(np.isnan(w), -np.inf, w)
    nan = np.isnan(np.asarray(weight, np.float64)[:length])
    middle = np.arange(first, length - recent)
    # heaviest first, NaN behind -inf, then the lowest slot
    order = sorted(middle, key=lambda j: (nan[j], -w[j], j))[:keep - first - recent]
    return np.sort(np.concatenate([np.arange(first), order, np.arange(length - recent, length)]).astype(np.int64))
