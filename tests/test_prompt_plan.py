"""The prompt attention's work plan, run on the CPU by tests/plan_emulator.cpp: every (sequence, KV head, tile of
rows) is found once, whatever the order in which a CTA comes by the indices."""
import os
import random
import shutil
import subprocess

import pytest

from paged_kv_cache_372_b200 import build as b

STUB = """#pragma once
#include <stdint.h>
#include "pa.h"
namespace pa { constexpr unsigned FULL_MASK = 0xffffffffu; }
"""


@pytest.fixture(scope="module")
def emulator(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    shutil.copy(os.path.join(b.CSRC, "pa_prefill_plan.cuh"), d)
    shutil.copy(os.path.join(os.path.dirname(__file__), "plan_emulator.cpp"), d)
    (d / "pa_common.cuh").write_text(STUB)
    exe = str(d / "plan_emulator")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wno-unused-function", "-I", str(d), "-I", b.INCLUDE,
                    str(d / "plan_emulator.cpp"), "-o", exe], check=True)
    return exe


def ask(exe, what, paged, cu, ctx, H, Hkv, limit, sms, order):
    T = cu[-1]
    head = [int(paged), len(ctx), T, H, Hkv, limit, sms, len(order)]
    text = " ".join([what] + [str(x) for x in head + cu + ctx + order]) + "\n"
    res = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=120)
    assert res.returncode == 0, f"the plan ended with {res.returncode}: {res.stderr}"
    lines = res.stdout.split("\n")
    assert lines[-2] == "end"
    return [[int(x) for x in line.split()] for line in lines[:-2]]


def boundaries(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def tiles_of(lens, H, Hkv):
    TM = 256 // (H // Hkv)
    return {(s, t * TM, h) for s, n in enumerate(lens) for t in range(-(-n // TM)) for h in range(Hkv)}


LENS = [[1], [1, 7, 16, 33], [0, 31, 0, 0, 32, 65, 0], [700, 5, 2049, 300], [40 * i % 173 for i in range(70)]]


@pytest.mark.parametrize("lens", LENS, ids=lambda x: f"{len(x)}x{max(x)}")
@pytest.mark.parametrize("H,Hkv", [(2, 2), (8, 2), (8, 1)])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("way", ["rising", "falling", "any", "repeated"])
def test_items_do_not_depend_on_the_order_of_the_indices(emulator, lens, H, Hkv, paged, way):
    rng = random.Random(len(lens) + H)
    ctx = [n + rng.randrange(0, 900) for n in lens] if paged else lens
    want = tiles_of(lens, H, Hkv)
    order = list(range(len(want) + 3))  # and some past the last item
    if way == "falling":
        order.reverse()
    elif way != "rising":
        rng.shuffle(order)
        if way == "repeated":
            order += order[:5]
    got = ask(emulator, "find", paged, boundaries(lens), ctx, H, Hkv, max(ctx + [1]), 148, order)
    of = {}
    for k, found, s, tok0, kvh, row0, n, keys in got:
        assert bool(found) == (k < len(want))
        if found:
            assert (row0, n, keys) == (boundaries(lens)[s], lens[s], ctx[s])
            assert of.setdefault(k, (s, tok0, kvh)) == (s, tok0, kvh)
    assert set(of.values()) == want and len(of) == len(want)
    # the longest first, up to the width of a level
    TM = 256 // (H // Hkv)
    far = [(max(ctx[s] - lens[s], 0) // TM * TM + tok0) // TM for s, tok0, _ in (of[k] for k in sorted(of))]
    assert all(b <= a + 7 for a, b in zip(far, far[1:]))
