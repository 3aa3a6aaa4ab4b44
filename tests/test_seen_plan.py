"""Which kernel a call with trees or sinks launches: the host's rule, compiled by itself."""
import ctypes
import os
import subprocess

import pytest

from conftest import ROOT

SOURCE = r"""
#include "kv4_plan.h"
extern "C" int plan(long long heads, long long seqs, long long pages, int dim, long long share, long long tokens,
                    long long max_new, long long window, long long sinks, long long* out) {
  const dcc::AttnPlan p = dcc::seen_plan(heads, seqs, pages, dim, share, tokens, max_new, window, sinks, 152);
  out[0] = p.tiles, out[1] = p.small;
  return p.prompt;
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "driven_collective_communication_gb300", "csrc"), "-o", str(d / "plan.so"),
                    str(d / "plan.cpp")], check=True)
    f = ctypes.CDLL(str(d / "plan.so")).plan
    f.argtypes = [ctypes.c_longlong] * 3 + [ctypes.c_int] + [ctypes.c_longlong] * 5 + [ctypes.c_void_p]

    def call(heads=8, seqs=1, pages=128, dim=128, share=8, tokens=4, max_new=4, window=0, sinks=0):
        out = (ctypes.c_longlong * 2)()
        return bool(f(heads, seqs, pages, dim, share, tokens, max_new, window, sinks, out)), out[0], bool(out[1])
    return call


@pytest.mark.parametrize("dim,most", [(128, 16), (64, 24)])
def test_rows(plan, dim, most):
    for rows in range(1, 200):
        for pages in (10, 100000):
            many, tiles, _ = plan(dim=dim, share=1, tokens=rows, max_new=rows, pages=pages)
            assert many == (rows > 2 * most or (rows > most and pages == 10))
            assert many or tiles * 8 * -(-rows // most) >= rows


def test_the_measured_crossings(plan):
    assert plan()[0] and plan(seqs=16, pages=32, tokens=64)[0] and not plan(pages=1024)[0]
    assert not plan(heads=32, seqs=16, pages=64, tokens=64)[0]
    assert plan(pages=1024, window=1024, sinks=4)[0] and plan(seqs=16, pages=128, tokens=64, window=1024, sinks=4)[0]
    assert plan(pages=1024, tokens=6, max_new=6)[0]


def test_idle_slots_change_nothing(plan):
    for pages in (10, 128, 1024):
        for new in (1, 4, 30):
            alone = plan(pages=pages, tokens=new, max_new=new)
            for seqs in (2, 64, 1000):
                many, tiles, _ = plan(seqs=seqs, pages=pages, tokens=new, max_new=new)
                assert (many, tiles) == alone[:2]


# what the tests of these kernels name by their shapes: (ranks x kv heads, lengths, new tokens, share, window, sinks)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,lens,news,share,window,sinks", [
    (2, [700, 300], [130, 100], 4, 100, 4), (2, [900], [257], 3, 300, 130), (8, [600], [64], 8, 128, 1),
    (1, [500, 64, 0, 33], [200, 64, 0, 33], 8, 33, 64), (1, [4096], [40], 8, 2000, 300), (2, [700, 300, 64], [63, 32, 33], 4, 0, 0),
    (2, [900], [70], 8, 0, 0), (8, [2000], [32], 8, 0, 0), (1, [300, 256], [256, 256], 2, 0, 0), (1, [6000], [24], 16, 0, 0)])
def test_tests_of_many_rows_reach_their_kernel(plan, dim, heads, lens, news, share, window, sinks):
    assert plan(heads=heads, seqs=len(lens), pages=max(-(-m // 64) for m in lens), dim=dim, share=share, tokens=sum(news),
                max_new=max(news), window=window, sinks=sinks)[0]


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,lens,news,share,window,sinks", [
    (4, [300, 5, 64, 0, 1000], [1] * 5, 4, 100, 4), (2, [400, 200], [3, 5], 2, 130, 66), (1, [641], [1], 16, 127, 192),
    (1, [8], [8], 1, 0, 0), (4, [300, 5, 64, 0, 1000], [7, 5, 1, 0, 8], 2, 0, 0), (8, [200, 200], [2, 2], 8, 0, 0)])
def test_tests_of_few_rows_reach_the_streaming_kernel(plan, dim, heads, lens, news, share, window, sinks):
    assert not plan(heads=heads, seqs=len(lens), pages=max(-(-m // 64) for m in lens), dim=dim, share=share,
                    tokens=sum(news), max_new=max(news), window=window, sinks=sinks)[0]
