"""The whole-number arithmetic of cache extension (csrc/mla_spans.h), compiled for the host
and run over tables of up to 2^31 - 1 entries: sizes that no GPU test makes."""
import ctypes
import os
import subprocess

import pytest

from split_kv_mla_gb300 import build as mla_build

LAST = (1 << 31) - 1     # entries at most
CODE = r"""
#include "mla_spans.h"
using namespace mla;
extern "C" {
void run_of(uint32_t total, uint32_t warp, uint32_t warps, uint32_t span, int64_t* out)
{
    const Run r = warp_run(total, warp, warps, span);
    out[0] = r.begin;
    out[1] = r.end;
}
// the spans of a run, as the kernel goes through them; how many, at most `room`
int spans_of(uint32_t begin, uint32_t end, uint32_t span, int64_t* out, int room)
{
    int n = 0;
    for (uint32_t i0 = begin; i0 < end && n < room; i0 += span, ++n) {
        out[2 * n] = i0;
        out[2 * n + 1] = span_end(i0, end, span);
    }
    return n;
}
int64_t kept(uint32_t start, uint32_t next, uint32_t length) { return kept_end(start, next, length); }
int64_t place(uint32_t length, uint32_t n) { return token_place(length, n); }
int mid(int lo, int hi) { return middle(lo, hi); }
int has(uint32_t start, uint32_t next, uint32_t p) { return has_place(start, next, p) ? 1 : 0; }
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("spans")
    (d / "spans.cpp").write_text(CODE)
    so = str(d / "spans.so")
    subprocess.run([os.environ.get("CXX", "g++"), "-O1", "-std=c++17", "-fPIC", "-shared",
                    "-I", mla_build.CSRC, str(d / "spans.cpp"), "-o", so], check=True)
    lib = ctypes.CDLL(so)
    lib.kept.restype = ctypes.c_int64
    lib.kept.argtypes = [ctypes.c_uint32] * 3
    lib.place.restype = ctypes.c_int64
    lib.place.argtypes = [ctypes.c_uint32] * 2
    lib.has.argtypes = [ctypes.c_uint32] * 3
    lib.run_of.argtypes = [ctypes.c_uint32] * 4 + [ctypes.c_void_p]
    lib.spans_of.argtypes = [ctypes.c_uint32] * 3 + [ctypes.c_void_p, ctypes.c_int]
    return lib


def run_of(lib, total, warp, warps, span):
    out = (ctypes.c_int64 * 2)()
    lib.run_of(total, warp, warps, span, out)
    return out[0], out[1]


TOTALS = [0, 1, 31, 32, 33, 255, 256, 257, 511, 512, 513, 65536, 4864 * 32 + 1, 2361857, 1 << 30,
          (1 << 31) - 512, (1 << 31) - 511, (1 << 31) - 101, LAST]


@pytest.mark.parametrize("span", [256, 512])
@pytest.mark.parametrize("warps", [16, 33 * 16, 304 * 16])
@pytest.mark.parametrize("total", TOTALS)
def test_the_warps_cover_a_table(lib, total, warps, span):
    at = 0
    for w in range(warps):
        begin, end = run_of(lib, total, w, warps, span)
        if begin >= total:
            assert begin < 1 << 32
            break
        assert begin == at and begin < end <= total
        at = end
    assert at == total


@pytest.mark.parametrize("span", [256, 512])
@pytest.mark.parametrize("total", TOTALS[1:])
def test_spans_end_with_their_run(lib, total, span):
    room = 64
    out = (ctypes.c_int64 * (2 * room))()
    for begin in sorted({max(0, total - d) for d in (1, 2, span - 1, span, span + 1, 3 * span + 7)}):
        n = lib.spans_of(begin, total, span, out, room)
        got = [(out[2 * k], out[2 * k + 1]) for k in range(n)]
        want = [(i, min(i + span, total)) for i in range(begin, total, span)]
        assert got == want


@pytest.mark.parametrize("start,next_,length", [
    (0, 0, 0), (0, 5, 5), (3, 9, 4), (3, 9, 6), (3, 9, 100), (0, LAST, LAST), (LAST, LAST, 0),
    (LAST, LAST, LAST), (1_900_000_000, 2_000_000_000, 400_000_000), (1 << 30, LAST, 1 << 30),
    (LAST - 1, LAST, LAST), (5, 5, LAST)])
def test_what_is_kept_ends_in_the_request(lib, start, next_, length):
    assert lib.kept(start, next_, length) == min(start + length, next_)


@pytest.mark.parametrize("start,entries", [(0, 0), (0, 7), (LAST - 7, 7), (0, LAST), (1 << 30, 1 << 30)])
@pytest.mark.parametrize("length", [0, 3, 6, 7, (1 << 30) - 1, 1 << 30, LAST - 1, LAST])
@pytest.mark.parametrize("n", [0, 1, 2, 1 << 30, LAST - 1])
def test_tokens_without_an_entry(lib, start, entries, length, n):
    # `entries` of the table from start on are the request's: what it keeps, and its tokens,
    # as far as there is room
    assert lib.place(length, n) == length + n
    next_ = min(start + entries, LAST)
    assert lib.has(start, next_, lib.place(length, n)) == int(length + n < next_ - start)


@pytest.mark.parametrize("lo,hi", [(0, 1), (0, 2), (0, LAST), (1 << 30, (1 << 30) + 1), (1 << 30, LAST),
                                   (LAST - 1, LAST), (LAST - 2, LAST)])
def test_a_search_among_many_requests(lib, lo, hi):
    assert lib.mid(lo, hi) == (lo + hi) // 2


def test_every_search_takes_that_middle():
    for name in ("mla_step.cu", "mla_cache.cu"):
        with open(os.path.join(mla_build.CSRC, name)) as f:
            text = f.read()
        assert "middle(lo, hi)" in text and "(lo + hi)" not in text, name
