"""The debug build's bounds checks of the 4-bit cache's kernels, whose addresses come from
page tables, lengths and counts on the device."""

import os
import re
import subprocess
import sys

import numpy as np
import pytest

from tests.conftest import ROOT

torch = pytest.importorskip("torch")
ra = pytest.importorskip("context_ring_attention_gb300")

CSRC = os.path.join(ROOT, "context_ring_attention_gb300", "csrc")


@pytest.mark.parametrize("name", ["kv4_rows.cu", "kv4_attend.cu"])
def test_addresses_are_checked(name):
    """Each kernel file checks what it reads and what it writes, at sites of its own."""
    sites = {}
    for other in sorted(os.listdir(CSRC)):
        if other.endswith(".cu"):
            with open(os.path.join(CSRC, other)) as f:
                sites[other] = [int(x) for x in re.findall(r"RA_BOUNDS\(.*?,\s*(\d+)\);", f.read(), re.S)]
    assert len(sites[name]) >= 5
    others = {x for other, v in sites.items() if other != name for x in v}
    assert not others & set(sites[name]) and max(sites[name]) < 256


def cache_outputs():
    """Bytes written, rows read back and attention for each type, head size and split: one
    sequence, one CTA a sequence, sequences in a row; few rows and several tiles; a window."""
    out = {}
    rng = np.random.default_rng(31)
    dev = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")
    for n, (dtype, d, lengths, t, hq, hk, window, sinks) in enumerate([
            ("bf16", 128, [1900], 1, 4, 1, 0, 0), ("bf16", 64, [70, 0, 33], 3, 6, 2, 20, 3),
            ("f32", 128, [300, 16, 1], 9, 3, 3, 0, 0), ("bf16", 128, [2300, 0, 1801, 40], 5, 16, 2, 1500, 20),
            ("f32", 64, [1700, 2], 1, 4, 2, 0, 0)]):
        dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        page_rows = 48
        used = [-(-x // page_rows) for x in lengths]
        pages, width = sum(used) + 2, max(used) + 1
        order, table = rng.permutation(pages), np.full((len(lengths), width), pages + 7)
        for b, x in enumerate(used):
            table[b, :x] = order[sum(used[:b]):sum(used[:b]) + x]
        kv = ra.ra_kv4_plan(pages, page_rows, hq, hk, d, dtype=dtype, window=window, sinks=sinks)
        cache = torch.full((ra.ra_kv4_cache_size(kv),), 0xAB, dtype=torch.uint8, device="cuda")
        k, v, q = (torch.from_numpy(rng.normal(size=(len(lengths), h, x, d))).to(dt).cuda()
                   for h, x in ((hk, max(lengths)), (hk, max(lengths)), (hq, t)))
        tab, first = dev(table), dev([0] * len(lengths))
        ra.ra_kv4_write(kv, cache, k, v, tab, first, dev(lengths))
        back = ra.ra_kv4_read(kv, cache, tab, first, max(lengths), dev(lengths))
        o = ra.ra_kv4_attend(kv, cache, q, tab, dev(lengths))
        ra.ra_kv4_sync_status(kv)
        for name, x in zip("ckvol", (cache, *back, *o)):
            out[f"{n}/{name}"] = x.float().cpu().numpy()
    return out


@pytest.mark.gpu
def test_debug_library_passes_its_bounds_checks(tmp_path):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    path = str(tmp_path / "out.npz")
    code = "import numpy as np, sys; from tests import test_kv4_bounds as t; np.savez(sys.argv[1], **t.cache_outputs())"
    res = subprocess.run([sys.executable, "-c", code, path], cwd=ROOT, env=dict(os.environ, RA_LIBRARY_VARIANT="debug"),
                         capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr[-2000:]
    here = cache_outputs()
    with np.load(path) as debug:
        assert set(debug.files) == set(here)
        for name, a in here.items():
            assert np.array_equal(a, debug[name]), name
