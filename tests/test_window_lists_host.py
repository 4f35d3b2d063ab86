"""The work lists of windowed plans: every visible (query, key) pair enters each sum once.

tests/window_lists.cc is the planner's own source with a main() that expands the lists as the
kernels do; it needs a C++ compiler and the CUDA headers, and no GPU."""

import itertools
import os
import random
import shutil
import subprocess

import pytest

from tests.conftest import ROOT

LAYOUTS = {"contiguous": 0, "striped": 1, "zigzag": 2}


@pytest.fixture(scope="module")
def expand(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    cxx = shutil.which("g++")
    headers = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    if cxx is None or not os.path.exists(os.path.join(headers, "cuda_runtime.h")):
        pytest.skip("needs g++ and the CUDA headers")
    exe = str(tmp_path_factory.mktemp("lists") / "window_lists")
    # (the planner's file also holds the C ABI, which main() does not reach: the linker drops it,
    # and with it the calls of CUDA and of the kernels)
    subprocess.run([cxx, "-std=c++17", "-O2", "-w", "-x", "c++", os.path.join(ROOT, "tests", "window_lists.cc"), "-o", exe,
                    "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "context_ring_attention_gb300", "csrc"),
                    "-I", headers, "-ffunction-sections", "-fdata-sections", "-Wl,--gc-sections"], check=True)

    def run(cases):
        text = "".join("{} {} {} {} {} {} {} {}\n".format(*c) for c in cases)
        res = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=600)
        assert res.returncode == 0, res.stdout[-4000:] + res.stderr[-2000:]
        assert res.stdout.split()[-1] == str(len(cases))

    return run


def _cases(layout, seqs, shards, masks, heads=(2, 1)):
    return [(1, s, *heads, n, LAYOUTS[layout], w, k) for s, n, (w, k) in itertools.product(seqs, shards, masks)
            if s % (2 * n if layout == "zigzag" else n) == 0]


@pytest.mark.parametrize("layout", LAYOUTS)
def test_small_masks(expand, layout):
    """Windows and sinks around each other and around the stripes and tiles."""
    masks = [(w, k) for w in (1, 2, 7, 63, 64, 65, 122, 126, 127, 128, 129, 200, 300) for k in (0, 1, 4, 5, 66, 140)]
    expand(_cases(layout, (192, 300, 320), (1, 2, 3, 5, 8, 16), masks))


def test_first_stripe_of_the_window_holds_the_last_sink(expand):
    """Striped shards walked by position, where a range begins with its stripe: the window's
    first stripe is the sinks' last one."""
    expand([(1, 900, 4, 2, 3, 1, 122, 4), (1, 512, 4, 2, 8, 1, 124, 4), (1, 512, 4, 2, 8, 1, 122, 1),
            (1, 512, 4, 2, 4, 1, 126, 1), (1, 512, 4, 2, 4, 1, 127, 1), (1, 600, 3, 1, 100, 1, 150, 30)])


@pytest.mark.parametrize("layout", LAYOUTS)
def test_heads_batches_and_cut_tiles(expand, layout):
    masks = [(1, 0), (100, 4), (500, 3), (253, 130), (1000, 0)]
    cases = [(2, 256, 3, 1, 2, LAYOUTS[layout], *m) for m in masks]
    cases += [(1, 768, 6, 2, 2, LAYOUTS[layout], *m) for m in masks]
    cases += [(1, 1024, 4, 1, 1, LAYOUTS[layout], *m) for m in masks]
    cases += [(1, 1040, 2, 1, 130, LAYOUTS[layout], *m) for m in masks]  # stripes above a tile
    expand(cases)


def test_drawn_masks(expand):
    rng = random.Random(5)
    cases = []
    while len(cases) < 300:
        layout, n = rng.choice(list(LAYOUTS)), rng.choice([1, 2, 3, 4, 6, 7, 8, 12, 16, 31, 33, 65])
        unit = n * (2 if layout == "zigzag" else 1)
        s = max(1, rng.randrange(8, 420) // unit) * unit
        hq, hk = rng.choice([(1, 1), (2, 1), (3, 1), (2, 2)])
        cases.append((1, s, hq, hk, n, LAYOUTS[layout], rng.randrange(1, s + 40), rng.choice([0, 1, 3, 4, 9, 40, s // 2])))
    expand(cases)
