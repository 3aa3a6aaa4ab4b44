"""Which attention kernel a call launches: the host's rule, compiled by itself."""
import ctypes
import os
import subprocess

import pytest

from conftest import ROOT

SOURCE = r"""
#include "kv4_plan.h"
extern "C" int plan(long long heads, long long seqs, long long pages, int dim, long long share, long long tokens,
                    long long max_new, long long* out) {
  const dcc::AttnPlan p = dcc::attn_plan(heads, seqs, pages, dim, share, tokens, max_new, 152);
  out[0] = p.wide, out[1] = p.narrow, out[2] = p.tiles, out[3] = p.small;
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
    f.argtypes = [ctypes.c_longlong] * 3 + [ctypes.c_int] + [ctypes.c_longlong] * 3 + [ctypes.c_void_p]

    def call(heads=8, seqs=1, pages=128, dim=128, share=8, tokens=1, max_new=1):
        out = (ctypes.c_longlong * 4)()
        prompt = bool(f(heads, seqs, pages, dim, share, tokens, max_new, out))
        return dict(prompt=prompt, wide=out[0], narrow=out[1], tiles=out[2], small=bool(out[3]))
    return call


def test_the_measured_crossings(plan):
    assert not plan(tokens=64, max_new=64)["prompt"] and plan(tokens=128, max_new=128)["prompt"]
    assert not plan(heads=1, pages=1000, tokens=128, max_new=128)["prompt"]
    assert not plan(seqs=16, pages=64, tokens=16 * 4, max_new=4)["prompt"]
    assert plan(seqs=16, pages=64, tokens=16 * 8, max_new=8)["prompt"]
    assert plan(seqs=16, pages=64, tokens=16 * 128, max_new=128)["prompt"]
    assert plan(tokens=2048, max_new=2048) == dict(prompt=True, wide=57, narrow=14, tiles=0, small=False)


@pytest.mark.parametrize("pages", [32, 1000])
@pytest.mark.parametrize("heads", [1, 8])
@pytest.mark.parametrize("new", [2, 20, 128, 2048])
def test_idle_slots_change_nothing(plan, pages, heads, new):
    """One sequence with new tokens among any number of slots: the same kernel, all of its rows."""
    alone = plan(heads=heads, pages=pages, tokens=new, max_new=new)
    for seqs in (2, 64, 1000):
        p = plan(heads=heads, seqs=seqs, pages=pages, tokens=new, max_new=new)
        assert p["prompt"] == alone["prompt"] and p["tiles"] == alone["tiles"]
        assert not p["prompt"] or 256 * p["wide"] + 128 * p["narrow"] >= new * 8


def test_a_chunk_beside_decoding_sequences(plan):
    """128 new tokens of one sequence, one each of 63 others: no more than two such chunks."""
    for heads, pages in ((1, 1000), (8, 128), (2, 16)):
        two = plan(heads=heads, seqs=2, pages=pages, tokens=256, max_new=128)
        assert plan(heads=heads, seqs=64, pages=pages, tokens=128 + 63, max_new=128)["prompt"] == two["prompt"]
    assert not plan(heads=1, seqs=64, pages=1000, tokens=128 + 63, max_new=128)["prompt"]


def test_single_tokens_stream(plan):
    for share in (1, 8, 16):
        for seqs in (1, 64, 5000):
            assert not plan(seqs=seqs, share=share, tokens=seqs)["prompt"]
    assert plan(pages=13)["small"] and not plan(pages=128)["small"] and not plan(pages=13, share=9)["small"]


def test_row_tiles(plan):
    for dim, most in ((128, 16), (64, 24)):
        for rows in range(1, 200):
            p = plan(heads=1, pages=5000, dim=dim, share=1, tokens=rows, max_new=rows)
            assert not p["prompt"] and 1 <= p["tiles"] <= most // 8
            passes = -(-rows // most)
            assert p["tiles"] * 8 * passes >= rows and (p["tiles"] - 1) * 8 * passes < rows


# what the tests of the attention's kernels name by their shapes: (ranks x kv heads, lengths, new tokens, share)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,lens,news,share,rows_more", [
    (32, [90, 300, 64, 1], [30, 20, 25, 1], 4, 2), (16, [16, 200, 129], [16, 33, 129], 8, 2),
    (8, [2000, 30, 500, 0], [90, 90, 85, 4], 3, 2), (32, [65, 1000], [17, 40], 16, 2),
    (32, [128, 256, 383], [128, 100, 129], 1, 2), (16, [500, 64], [60, 40], 8, 0), (8, [200, 200], [60, 60], 8, 0),
    (8, [300, 300], [100, 100], 8, 0), (1, [150] * 16, [100] * 16, 4, 0), (8, [4096], [512], 8, 0),
    (8, [700, 300], [130, 100], 4, 0)])
def test_prompt_tests_reach_the_prompt_kernel(plan, dim, heads, lens, news, share, rows_more):
    pages = max(-(-m // 64) for m in lens)
    assert plan(heads=heads, seqs=len(lens), pages=pages, dim=dim, share=share, tokens=sum(news) + rows_more,
                max_new=max(news))["prompt"]


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,lens,news,share", [
    (1, [200, 200], [40, 40], 8), (1, [200, 200], [1, 1], 8), (2, [300, 5, 64], [5, 5, 1], 4), (2, [1000], [3], 4),
    (4, [70, 130], [2, 8], 3), (8, [3000, 10, 700], [1, 1, 1], 8)])
def test_streaming_tests_reach_the_streaming_kernel(plan, dim, heads, lens, news, share):
    pages = max(-(-m // 64) for m in lens)
    assert not plan(heads=heads, seqs=len(lens), pages=pages, dim=dim, share=share, tokens=sum(news),
                    max_new=max(news))["prompt"]
