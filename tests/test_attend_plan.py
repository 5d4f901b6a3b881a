"""The launch plans of qmv_attend_run, compiled by themselves: rings, operands and lists lie in shared memory side by
side and within a block's limit, rings hold what the kernels wait for at once, work items cover what queries may see and
their sums lie within the workspace."""

import ctypes
import random
import subprocess

import pytest

SOURCE = r"""
#include "qmv_attend_plan.h"
using namespace qmv::attend;
extern "C" int attend_plan(int B, int T, int max_new, int heads, int kv_heads, int D, long long capacity, int window, int sinks, long long *out)
{
    const FewPlan f = few_plan(B, max_new, heads, kv_heads, D, capacity, window, sinks);
    const PromptPlan g = prompt_plan(B, T, max_new, heads, kv_heads, D, capacity, window, sinks);
    const long long v[] = {f.columns, f.tokens, f.blocks, f.rows, f.slots, f.key_slots, f.ctas, f.q_sets, f.p_off, f.q_off, f.misc_off, f.smem, f.unit, f.units, f.items,
                           (long long)f.meta_off, (long long)f.parts_off, (long long)f.workspace, few_misc(f.columns),
                           g.tokens, g.streams, g.slots, g.chunk, g.key_slots, g.q_off, g.misc_off, g.smem, g.pieces, g.items,
                           (long long)g.prefix_off, (long long)g.meta_off, (long long)g.parts_off, (long long)g.workspace, kPromptMisc};
    for (unsigned i = 0; i < sizeof v / sizeof *v; ++i) out[i] = v[i];
    return int(sizeof v / sizeof *v);
}
"""
FEW = ("columns", "tokens", "blocks", "rows", "slots", "key_slots", "ctas", "q_sets", "p_off", "q_off", "misc_off", "smem", "unit", "units", "items",
       "meta_off", "parts_off", "workspace", "misc")
PROMPT = ("tokens", "streams", "slots", "chunk", "key_slots", "q_off", "misc_off", "smem", "pieces", "items", "prefix_off", "meta_off", "parts_off",
          "workspace", "misc")
BLOCK = 227 * 1024


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    from group_quantized_mat_gb300 import build
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(SOURCE)
    subprocess.run([build._nvcc(), "-x", "c++", "-O1", "-std=c++17", "-I", build.INCLUDE, "-I", build.CSRC, "-shared", "-Xcompiler", "-fPIC",
                    "-o", str(d / "plan.so"), str(d / "plan.cpp")], check=True, capture_output=True)
    lib = ctypes.CDLL(str(d / "plan.so"))

    def call(B, T, max_new, heads, kv_heads, D, capacity, window, sinks):
        out = (ctypes.c_longlong * 64)()
        n = lib.attend_plan(B, T, max_new, heads, kv_heads, D, ctypes.c_longlong(capacity), window, sinks, out)
        assert n == len(FEW) + len(PROMPT)
        return dict(zip(FEW, out)), dict(zip(PROMPT, out[len(FEW):n]))
    return call


def check_few(f, B, max_new, heads, kv, D, capacity, window, sinks):
    group, most = heads // kv, min(max_new, 16)
    assert f["columns"] in (16, 32, 64) and f["rows"] == f["tokens"] * group <= f["columns"]
    assert f["blocks"] * f["tokens"] >= most > (f["blocks"] - 1) * f["tokens"]
    # shared memory: ring, weights (two bf16 terms of 256 keys), queries, lists; 1024 bytes to align it
    assert f["p_off"] >= f["slots"] * 16384 and f["q_off"] - f["p_off"] >= 256 * f["columns"] * 4
    assert f["misc_off"] - f["q_off"] >= f["q_sets"] * f["columns"] * D * 2
    assert f["smem"] >= 1024 + f["misc_off"] + f["misc"] + B * 16 + (B + 1) * 4
    assert all(f[k] % 1024 == 0 for k in ("p_off", "q_off", "misc_off"))
    assert f["smem"] <= BLOCK and f["ctas"] * (f["smem"] + 1024) <= 228 * 1024
    # the barriers' lists have 16 places; a tile's values have to be there at once
    assert 1 <= f["key_slots"] and f["slots"] - f["key_slots"] >= max(D // 64, 1) and f["slots"] <= 16
    # keys run at most as many leaves ahead of the scores that are being weighed as the list of pages knows
    assert -(-f["key_slots"] // (2 * (D // 64))) + 4 <= 8
    # units: enough for any place of the window and of the first tokens
    assert f["unit"] in (256, 512, 1024) and f["items"] == B * kv * f["blocks"] * f["units"]
    u = f["unit"]
    for end in {1, min(most, capacity), capacity, max(1, capacity - 1), max(1, capacity // 2 + 3)} | {random.randint(1, capacity) for _ in range(20)}:
        first = end - most  # position of the first of `most` tokens
        low = max(first - window + 1, 0) if window else 0
        least = min(sinks, low) if window else 0
        units = {j // u for j in (0, least - 1) if least > 0}
        count = (len(range(0, (least - 1) // u + 1)) if units else 0)
        near = (end - 1) // u - low // u + 1
        overlap = units and (least - 1) // u >= low // u
        assert count + near - bool(overlap) <= f["units"]
    if f["units"] > 1:
        assert f["parts_off"] >= f["meta_off"] + f["items"] * f["rows"] * 8
        assert f["workspace"] >= f["parts_off"] + f["items"] * f["rows"] * D * 4
    assert f["workspace"] > 0 and f["parts_off"] % 16 == 0


def check_prompt(g, B, T, heads, kv, D, capacity):
    group = heads // kv
    assert g["tokens"] * group <= 128 and g["tokens"] >= 1
    assert g["streams"] == (1 if D == 256 else 2)
    assert g["q_off"] >= g["slots"] * g["chunk"] and g["misc_off"] - g["q_off"] >= g["streams"] * 128 * D * 2
    assert g["smem"] >= 1024 + g["misc_off"] + g["misc"] + B * 16 + (B + 1) * 4 and g["smem"] <= BLOCK
    assert g["q_off"] % 1024 == 0 and g["misc_off"] % 1024 == 0 and g["chunk"] % 1024 == 0
    # a tile's keys, and its values, in either ring at once; at most eight tiles of keys from issue to use
    tile = 128 * D * 2 // g["chunk"]
    assert g["key_slots"] >= tile or D == 256 and g["key_slots"] >= 1
    assert g["slots"] - g["key_slots"] >= 1 and g["slots"] <= 12 and -(-g["key_slots"] // tile) + 2 < 8
    assert 1 <= g["pieces"] <= max(1, -(-capacity // 1024))
    # items: of any division of T rows into sequences of more than 16
    each = g["streams"] * g["tokens"]
    worst = 0
    for _ in range(20):
        left, n = T, 0
        for _ in range(B):
            if left <= 16:
                break
            s = random.choice([17, each + 1, left, random.randint(17, left)])
            s = min(max(s, 17), left)
            n += -(-s // each)
            left -= s
        worst = max(worst, n)
    assert g["items"] >= worst * kv * g["pieces"]
    if g["pieces"] > 1:
        rows = g["items"] * g["streams"] * 128
        assert g["meta_off"] >= (B + 1) * 4 and g["parts_off"] >= g["meta_off"] + rows * 8 and g["workspace"] >= g["parts_off"] + rows * D * 4


@pytest.mark.parametrize("D", [64, 128, 256])
def test_plans(plan, D):
    random.seed(D)
    for _ in range(1500):
        kv = random.choice([1, 2, 3, 8, 32, 256])
        heads = kv * random.choice([1, 2, 3, 4, 5, 7, 8, 16, 17, 33, 64])
        B = random.choice([1, 2, 5, 33, 256, 1024])
        max_new = random.choice([1, 2, 5, 15, 16, 17, 31, 100, 1000, 5000])
        T = random.choice([max_new, max_new + 1, B * max_new, max_new * 3])
        capacity = random.choice([8, 128, 250 * 8, 4096, 70000, 1 << 20, 1 << 26])
        window = random.choice([0, 0, 1, 2, 128, 1000, 4096, 1 << 20, 1 << 30])
        sinks = random.choice([0, 1, 4, 100, 128, 1000, 1 << 30])
        f, g = plan(B, T, max_new, heads, kv, D, capacity, window, sinks)
        check_few(f, B, max_new, heads, kv, D, capacity, window, sinks)
        if max_new > 16:
            check_prompt(g, B, T, heads, kv, D, capacity)
        else:
            assert g["items"] == 0


def test_the_unit_depends_on_room_alone(plan):
    """A token's sums keep their order whatever else is in the call."""
    units = set()
    for B, T, max_new in [(1, 1, 1), (7, 70, 16), (1024, 1024, 1), (3, 5000, 4000)]:
        f, _ = plan(B, T, max_new, 40, 8, 128, 100000, 0, 0)
        units.add((f["unit"],))
    assert len(units) == 1
