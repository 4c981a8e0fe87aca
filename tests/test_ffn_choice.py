"""Every kernel that the feed-forward products can choose has a test (CPU): the choice is built
from its header with the host's compiler and asked about sizes over the whole range."""
from __future__ import annotations

import collections
import ctypes
import math
import os
import random
import subprocess

import pytest

from ffn_sizes import KERNELS, KINDS, MANY, NAMES

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "block_scaled_precision_bf16tofp4row_amd", "csrc")
ASK = """
#include "ffn_choice.h"
extern "C" int choice(int kind, int fp8, int32_t G, int64_t M_cap, int64_t N, int64_t K)
{
    using namespace mxfp4;
    const Which w = choose((Kind)kind, fp8, G, M_cap, N, K);
    return 2 * w + (w > kRows32 && feature_runs(kind == kGated ? 2 : 1, kCost[w].TM, G, M_cap, N));
}
extern "C" int size(int w, int columns) { return columns ? mxfp4::kCost[w].TN : mxfp4::kCost[w].TM; }
extern "C" int kernels() { return mxfp4::kKernels; }
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("choice")
    (d / "ask.cpp").write_text(ASK)
    subprocess.check_call(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-fPIC", "-shared", "-I", CSRC, "-o",
                           str(d / "ask.so"), str(d / "ask.cpp")])
    lib = ctypes.CDLL(str(d / "ask.so"))
    lib.choice.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int32] + [ctypes.c_int64] * 3
    return lib


def choice(lib, kind, fp8, G, M_cap, N, K):
    v = lib.choice(KINDS.index(kind), int(fp8), G, M_cap, N, K)
    return NAMES[v // 2], bool(v % 2)


def test_the_names(lib):
    assert lib.kernels() == len(NAMES)
    for i, name in enumerate(NAMES):
        rows = name.removeprefix("rows")
        tm, tn = (int(rows), 32) if rows != name else (int(v) for v in name.rstrip("splitar").split("x"))
        assert (lib.size(i, 0), lib.size(i, 1)) == (tm, tn), name


def test_listed_sizes_reach_their_kernels(lib):
    for kind, fp8, name, runs, *sizes in KERNELS + MANY:
        assert choice(lib, kind, fp8, *sizes) == (name, runs), (kind, fp8, sizes)
    seen = [k[:4] for k in KERNELS]
    assert len(set(seen)) == len(seen)


def test_no_kernel_without_a_size(lib):
    r = random.Random(11)
    log = lambda lo, hi: int(round(math.exp(r.uniform(math.log(lo), math.log(hi)))))      # noqa: E731
    listed, found = {k[:4] for k in KERNELS}, collections.Counter()
    for _ in range(300000):
        kind, fp8 = r.choice([("gated", False), ("gated", True), ("gradient", False), ("gradient", True),
                              ("dense", False)])
        n = 8 * log(1, 2048) if not fp8 else 16 * log(1, 1024) if kind == "gated" else 128 * log(1, 64)
        key = (kind, fp8, *choice(lib, kind, fp8, 1 if r.random() < 0.3 else log(2, 300), log(1, 30000), n, 16 * log(1, 1024)))
        found[key] += 1
    assert not set(found) - listed, {k: found[k] for k in set(found) - listed}
    assert len(found) > 0.9 * len(listed)         # (and the search is no small part of the range)
