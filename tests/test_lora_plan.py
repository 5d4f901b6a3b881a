"""The launch plan of qmv_lora_run, compiled by itself: whatever a kernel of such a
plan addresses in shared memory stays where the plan put it, and the shapes that the
GPU tests run are those whose plans differ."""

import ctypes
import os
import random
import subprocess

import pytest

from lora_shapes import FEW_SLOTS, PASSES, THREE_SLOTS

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SOURCE = r"""
#include "qmv_lora_plan.h"
using namespace qmv;
extern "C" int lora_plan(int M, int N, int K, int bits, int gs, int R, int sms, int *out)
{
    lora::Sizes sz;
    lora::LoraShape p = lora::plan(M, N, K, bits, gs, R, sms, sz);
    const int ok = lora::fit(p, bits);
    const lora::Layout l = lora::layout(p, bits, p.nc);
    const int passes = (M + lora::kPass - 1) / lora::kPass, most = (passes + p.grid_passes - 1) / p.grid_passes;
    int inner_end = 0;
    for (int before = 0; before < most; ++before) {
        const int end = lora::inner_at(p, l, before) + l.inner_bytes;
        inner_end = end > inner_end ? end : inner_end;
    }
    const int v[] = {p.slots, p.sb_buffers, p.inner_buffers, p.nseg, p.range * tile::slot_subs(bits), p.rows, p.tiles, p.grid_rows,
                     p.grid_passes, most, int(sz.total / 256), p.piece, p.nc, l.slot, l.x, l.meta, l.sb, l.inner, inner_end, l.bars, l.misc, l.total, lora::kSmem, p.sb.block};
    for (unsigned i = 0; i < sizeof v / sizeof *v; ++i) out[i] = v[i];
    return ok;
}
"""
NAMES = ("slots", "sb_buffers", "inner_buffers", "nseg", "subs", "rows", "tiles", "grid_rows", "grid_passes", "passes", "workspace", "piece", "nc",
         "slot", "x", "meta", "sb", "inner", "inner_end", "bars", "misc", "total", "most", "block")


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    from group_quantized_mat_gb300 import build
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(SOURCE)
    subprocess.run([build._nvcc(), "-x", "c++", "-O1", "-std=c++17", "-D__host__=", "-D__device__=", "-I", build.INCLUDE, "-I", build.CSRC,
                    "-shared", "-Xcompiler", "-fPIC", "-o", str(d / "plan.so"), str(d / "plan.cpp")], check=True, capture_output=True)
    lib = ctypes.CDLL(str(d / "plan.so"))

    def call(M, N, K, bits, gs, R, sms=152):
        out = (ctypes.c_int * len(NAMES))()
        ok = lib.lora_plan(M, N, K, bits, gs, R, sms, out)
        return dict(zip(NAMES, out), ok=ok)
    return call


def check(p):
    assert p["ok"]
    assert p["slots"] % 3 == 0 and p["slots"] >= 3 and p["piece"] >= 1 and 8 <= p["rows"] <= 128 and p["rows"] % 8 == 0
    assert p["slots"] * p["slot"] <= p["x"] and (p["slots"] - 1) * p["slot"] + 128 * 128 <= p["x"]
    assert p["x"] < p["meta"] < p["sb"] and p["sb"] + 2 * p["sb_buffers"] * p["block"] <= p["inner"]
    assert p["inner"] < p["inner_end"] <= p["bars"] < p["misc"] < p["total"] <= p["most"]
    assert p["tiles"] * p["rows"] >= 1 and p["passes"] >= 1


def test_everything_stays_in_its_place(plan):
    rng = random.Random(1)

    def log(lo, hi):
        return int(lo * (hi / lo) ** rng.random() + 0.5)
    for _ in range(30000):
        gs = rng.choice([64, 128])
        check(plan(log(1, 256), log(1, 200000), gs * log(1, 65536 // gs), rng.choice([2, 4]), gs, log(1, 256), rng.choice([152, 152, 148, 132, 1])))


@pytest.mark.parametrize("N,K", [(15360, 3840), (3840, 15360), (14336, 4096), (4096, 14336), (17408, 5120), (5120, 17408), (128256, 4096)])
def test_widths_of_served_models(plan, N, K):
    for M in (1, 2, 4, 8, 16, 17, 32, 33, 64, 200, 256):
        for bits in (2, 4):
            for gs in (64, 128):
                for R in (1, 16, 27, 64, 65, 256):
                    check(plan(M, N, K, bits, gs, R))


def test_gpu_shapes_cover_the_plans(plan):
    """Several passes in a CTA with one set of inner vectors and with two, rings of three
    slots and of more, one buffer of scales and two, one range of K and several."""
    seen = [plan(*s) for s in PASSES]
    several = [p for p in seen if p["passes"] > 1]
    for key, values in (("inner_buffers", (1, 2)), ("sb_buffers", (1, 2))):
        assert {p[key] for p in several} >= set(values), key
    assert {p["slots"] for p in several} >= {3, 6}
    assert any(p["nseg"] == 1 for p in several) and any(p["nseg"] > 1 for p in several)
    assert any(p["slots"] == 3 and p["inner_buffers"] == 1 and p["passes"] > 2 for p in several)
    assert any(p["tiles"] > p["grid_rows"] for p in several)
    for s in THREE_SLOTS:
        assert plan(*s)["slots"] == 3, s
    for s in FEW_SLOTS:
        p = plan(*s)
        assert p["passes"] > 1 and p["nseg"] == 1 and p["subs"] * s[3] < 3 * 16, s


def test_sums_do_not_depend_on_the_card(plan):
    """Ranges of K, which fix the order of sums, are the same whatever the number of SMs, as
    the workspace is, whose size is asked for without a card; and the GPU test of tiles compares different heights over equal ranges."""
    for N, K in ((1000, 1024), (15360, 3840), (3840, 15360), (250, 5120), (128256, 4096)):
        for M in (1, 16, 64):
            assert len({(p["nseg"], p["subs"], p["workspace"]) for p in (plan(M, N, K, 4, 64, 32, sms) for sms in (1, 100, 148, 152))}) == 1
    a, b = plan(5, 1000, 1024, 4, 64, 72), plan(5, 5000, 1024, 4, 64, 72)
    assert a["nseg"] == b["nseg"] == 1 and a["rows"] != b["rows"]
