"""The division of keys into pages, compiled by itself for every page size, and calls whose keys lie far behind."""

import ctypes
import subprocess

import pytest
import torch

SOURCE = r"""
#include "qmv_attend_plan.h"
using namespace qmv::attend;
// keys [0, end), multiples of 8, whose page is wrong; the first of them in *first
extern "C" long long wrong(int page_size, long long end, int step, long long *first)
{
    const uint64_t magic = page_magic(page_size);
    long long n = 0;
    for (long long key = 0; key < end; key += step)
        if (page_of(magic, int(key)) != key / page_size && n++ == 0) *first = key;
    return n;
}
// the same of each page's first and last eight keys
extern "C" long long wrong_at_edges(int page_size, long long end)
{
    const uint64_t magic = page_magic(page_size);
    long long n = 0;
    for (long long key = page_size; key < end; key += page_size)
        n += (page_of(magic, int(key)) != key / page_size) + (page_of(magic, int(key - 8)) != key / page_size - 1);
    return n;
}
"""
END = (1 << 26) + 1024  # (a last unit of keys may end behind the capacity)


@pytest.fixture(scope="module")
def pages(tmp_path_factory):
    from group_quantized_mat_gb300 import build
    d = tmp_path_factory.mktemp("pages")
    (d / "pages.cpp").write_text(SOURCE)
    subprocess.run([build._nvcc(), "-x", "c++", "-O2", "-std=c++17", "-I", build.INCLUDE, "-I", build.CSRC, "-shared", "-Xcompiler", "-fPIC",
                    "-o", str(d / "pages.so"), str(d / "pages.cpp")], check=True, capture_output=True)
    lib = ctypes.CDLL(str(d / "pages.so"))
    lib.wrong.restype = lib.wrong_at_edges.restype = ctypes.c_longlong
    lib.wrong.argtypes = [ctypes.c_int, ctypes.c_longlong, ctypes.c_int, ctypes.POINTER(ctypes.c_longlong)]
    lib.wrong_at_edges.argtypes = [ctypes.c_int, ctypes.c_longlong]
    return lib


@pytest.mark.parametrize("page_size", [8, 16, 24, 40, 56, 200, 1000, 4096, 65528, 65536])
def test_pages_of_all_keys(pages, page_size):
    first = ctypes.c_longlong(-1)
    assert pages.wrong(page_size, END, 8, first) == 0, first.value


def test_pages_of_all_sizes_at_their_edges(pages):
    assert all(pages.wrong_at_edges(size, END) == 0 for size in range(8, 65537, 8))


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [(700, 0), (300, 21), (1, 1)])
@pytest.mark.parametrize("new", [[1, 3], [16, 1], [40, 2]])
def test_keys_at_the_end_of_the_range(new, window, sinks):
    """Pages of 8, room for 2^26 keys: a window behind key 2^25 gives the bits of the same keys near the start (the distances
    are multiples of eight units, so that parts are joined in the same order)."""
    from test_gpu_attend import Problem, same

    p = Problem(new, [3000, 2100], 4, 2, 64, page=8, seed=31)
    near, need = p.table, [-(-k // 8) for k in p.keys]
    p.most = 1 << 23

    def at(shift):
        p.table = torch.full((2, p.most), -1, dtype=torch.int32)
        for b in range(2):
            p.table[b, :-(-sinks // 8)] = near[b, :-(-sinks // 8)]
            p.table[b, shift // 8:shift // 8 + need[b]] = near[b, :need[b]]
        p.keys = [k + shift for k in (3000, 2100)]
        return p.run(window=window, sinks=sinks)

    want = at(0)
    p.check(want, window=window, sinks=sinks)
    for shift in ((1 << 25) - 8192, 1 << 25, (1 << 26) - 8192):
        assert same(at(shift), want), shift
