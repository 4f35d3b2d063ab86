"""GPU tests of the attention of chunks over caches larger than the L2, whose keys are walked in rounds: a CTA then has
more than one share, and an item's parts lie in several rounds."""

import os
import subprocess
import sys

import numpy as np
import pytest

from tests.conftest import ROOT

torch = pytest.importorskip("torch")
ra = pytest.importorskip("context_ring_attention_gb300")
from tests.test_gpu_paged import _i32, _same_bits  # noqa: E402
from tests.window_ref import BF16_U, assert_within  # noqa: E402

gpu = pytest.mark.gpu
ROUND = 44 << 20  # bytes of keys and values of a round
# counts, lengths, hq, hk, d, window, sinks, rounds on 152 SMs: the sequences' query tiles are pairs of 2 * (128 / group)
# tokens, each as long as its key tiles of 128; rounds are of ROUND bytes of what more than one pair reads, and of 100
# key tiles a CTA at least.
CASES = [
    ([2048], [36000], 32, 8, 128, 0, 0, 3),
    ([1500, 1, 1, 0, 1, 3], [27000, 20000, 1, 77, 9001, 3], 32, 8, 128, 0, 0, 2),  # beside the row kernel, on some of the SMs
    ([1111, 900], [22000, 18001], 32, 8, 128, 0, 0, 2),                           # two chunks
    ([4000], [30001], 16, 16, 64, 0, 0, 2),                                       # D 64, groups of one
    ([3000], [40000], 32, 8, 128, 12000, 4, 2),                                   # a window
]


class Chunks:
    def __init__(self, counts, lengths, hq, hk, d, window, sinks, rounds):
        torch.manual_seed(len(counts) + hq + d)
        self.counts, self.lengths, self.hq, self.hk, self.d, self.window, self.sinks = counts, lengths, hq, hk, d, window, sinks
        pr, b = 64, len(counts)
        used = [-(-n // pr) for n in lengths]
        pages = sum(used) + 2
        self.kv = ra.ra_paged_plan(pages, pr, hq, hk, d, window=window, sinks=sinks)
        shape = ra.ra_paged_cache_shape(self.kv)
        self.cache = (torch.randn(shape, device="cuda") * torch.exp(0.3 * torch.randn(d, device="cuda"))).bfloat16()
        order, table, at = torch.randperm(pages), torch.full((b, max(used)), -1, dtype=torch.int64), 0
        for i, n in enumerate(used):
            table[i, :n] = order[at:at + n]
            at += n
        self.table = table.int().cuda()
        self.first = np.concatenate([[0], np.cumsum(counts)])
        self.offset, self.length = _i32(self.first), _i32(lengths)
        self.q = torch.randn((sum(counts), hq, d), device="cuda").bfloat16()

    def attend(self, **kw):
        out = ra.ra_paged_attend(self.kv, self.cache, self.q, self.table, self.offset, self.length, **kw)
        ra.ra_paged_sync_status(self.kv)
        return out

    def check(self, o, lse):
        """Every row in float64 on the GPU, with the bounds of paged_ref.py."""
        g, scale = self.hq // self.hk, self.d ** -0.5
        for b, (count, length) in enumerate(zip(self.counts, self.lengths)):
            if not count:
                continue
            j = torch.arange(length, device="cuda")
            pages = self.table[b].long()[j // 64]
            for h in range(self.hk):
                k, v = (self.cache[pages, w, h, j % 64].double() for w in (0, 1))
                for t0 in range(0, count, 512):
                    t1 = min(count, t0 + 512)
                    rows = slice(int(self.first[b]) + t0, int(self.first[b]) + t1)
                    slot = torch.arange(length - count + t0, length - count + t1, device="cuda")[:, None]
                    seen = j[None] <= slot
                    if self.window:
                        seen &= (j[None] > slot - self.window) | (j[None] < self.sinks)
                    for e in range(h * g, h * g + g):
                        q = self.q[rows, e].double()
                        s = ((q @ k.T) * scale).masked_fill(~seen, -torch.inf)
                        mag = ((q.abs() @ k.abs().T) * scale).masked_fill(~seen, 0.0).amax(-1)
                        lw = torch.logsumexp(s, -1)
                        p = torch.exp(s - lw[:, None])
                        err = 2.0 ** -15 * (1 + mag) + length * 2.0 ** -23
                        ow = p @ v
                        bound = (BF16_U + 2 * err[:, None]) * (p @ v.abs()) + BF16_U * ow.abs()
                        assert_within(lse[rows, e], lw, err, f"LSE of sequence {b}, head {e}")
                        assert_within(o[rows, e], ow, bound, f"O of sequence {b}, head {e}")


@pytest.mark.parametrize("counts,lengths,hq,hk,d,window,sinks,rounds", CASES)
def test_the_cases_have_rounds(counts, lengths, hq, hk, d, window, sinks, rounds):
    """By the rule that the file's head states."""
    per_item, units, again = 2 * (128 // (hq // hk)), 0, 0
    for n, length in zip(counts, lengths):
        if n * hq // hk <= 16:
            continue
        again += length if n > per_item else 0
        for t0 in range(0, n, per_item):
            s0, s1 = length - n + t0, length - n + min(n, t0 + per_item) - 1
            lo = max(0, s0 - window + 1) if window else 0
            tiles = set(range(lo // 128, s1 // 128 + 1)) | set(range(-(-min(sinks, lo) // 128)))
            units += len(tiles)
    assert min(8, units * hk // (100 * 152), again * hk * d * 4 // ROUND) == rounds


@gpu
@pytest.mark.parametrize("case", CASES, ids=lambda c: str(c[:2]))
def test_rounds(case):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    t = Chunks(*case)
    need = ra.ra_paged_attend_scratch_size(t.kv, len(t.counts), t.q.shape[0], t.table.shape[1])
    scratch = torch.full((need // 4 + 1024,), float("nan"), device="cuda")
    o, lse = t.attend(scratch=scratch)
    assert torch.isnan(scratch[need // 4:]).all()
    t.check(o, lse)
    again = t.attend(scratch=scratch)
    assert _same_bits(o, again[0]) and _same_bits(lse, again[1])


def rounds_outputs():
    out = {}
    for n, case in enumerate(CASES[1:4]):
        o, lse = Chunks(*case).attend()
        out[f"{n}/o"], out[f"{n}/lse"] = o.float().cpu().numpy(), lse.cpu().numpy()
    return out


@gpu
def test_debug_library_passes_its_bounds_checks(tmp_path):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    path = str(tmp_path / "out.npz")
    code = "import numpy as np, sys; from tests import test_gpu_paged_rounds as t; np.savez(sys.argv[1], **t.rounds_outputs())"
    res = subprocess.run([sys.executable, "-c", code, path], cwd=ROOT, env=dict(os.environ, RA_LIBRARY_VARIANT="debug"),
                         capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr[-2000:]
    here = rounds_outputs()
    with np.load(path) as debug:
        assert set(debug.files) == set(here)
        for name, a in here.items():
            assert np.array_equal(a, debug[name]), name
