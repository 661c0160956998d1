"""The tokens that a thread of qr_kv_plan's kernel goes over, on the host: the
kernel's own header, compiled as plain C++.  Every token number that a thread
reaches lies in its CTA's range, in its chunk and below 2^31 - 1, wherever the
chunk begins."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_quantized_all_gb300", "csrc")
SOURCE = """
#include "qr_kv_plan_range.h"
extern "C" void plan_range(long long lo, long long hi, long long chunk_lo, long long chunk_hi, int thread, long long *out) {
    const qrk::PlanTokens t = qrk::plan_tokens(lo, hi, chunk_lo, chunk_hi);
    out[0] = t.from, out[1] = t.to, out[2] = qrk::plan_first(t, thread);
}
extern "C" int plan_threads() { return qrk::kPlanThreads; }
extern "C" int plan_wide() { return qrk::kPlanWide; }
"""
MOST = 2 ** 31 - 1


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    where = tmp_path_factory.mktemp("plan_range")
    src, so = str(where / "plan.cpp"), str(where / "plan.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run([gxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-Wall", "-Werror", "-I", CSRC, src, "-o", so], check=True)
    L = ctypes.CDLL(so)
    L.plan_range.argtypes = [ctypes.c_longlong] * 4 + [ctypes.c_int, ctypes.POINTER(ctypes.c_longlong)]
    L.plan_range.restype = None
    return L


def _check(L, lo, hi, chunk_lo, chunk_hi):
    want = range(max(lo, chunk_lo), min(hi, chunk_hi, MOST))
    got = (ctypes.c_longlong * 3)()
    wide, threads = L.plan_wide(), L.plan_threads()
    for thread in (0, 1, 2, threads // 2, threads - 1):
        L.plan_range(lo, hi, chunk_lo, chunk_hi, thread, got)
        first = got[2]
        assert first == got[0] + wide * thread and first >= max(lo, chunk_lo)
        if first < got[1]:
            assert first in want and got[1] - 1 == want[-1]
        if not want:
            assert first >= got[1]


@pytest.mark.parametrize("chunk_lo", [0, 5, MOST - 1021, MOST - 1020, MOST - 3, MOST - 1, MOST, MOST + 1, 2 ** 31 + 5000, 2 ** 40, 2 ** 47])
@pytest.mark.parametrize("brings", [0, 1, 1000, 2 ** 31, 2 ** 42])
@pytest.mark.parametrize("lo,hi", [(0, MOST), (0, 256), (1000, MOST), (MOST - 500, MOST), (MOST + 7, MOST + 9)])
def test_chunks_at_and_past_the_last_token(host, chunk_lo, brings, lo, hi):
    _check(host, lo, hi, chunk_lo, chunk_lo + brings)


def test_random_ranges(host):
    rng = random.Random(0)
    for _ in range(3000):
        lo = rng.randrange(1 << rng.randint(1, 32))
        a = rng.randrange(1 << rng.randint(1, 48))
        _check(host, lo, lo + rng.randrange(1 << 31), a, a + rng.randrange(1 << rng.randint(1, 44)))
