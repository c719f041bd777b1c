"""The prompt attention's work plan, run on the CPU by tests/plan_emulator.cpp: every (sequence, KV head, tile of
rows) is found once, whatever the order in which a CTA comes by the indices; where contexts are split, every key
tile is walked once, and each part has a place of its own within the workspace, where the join looks for it."""
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


def ask(exe, what, paged, cu, ctx, H, Hkv, limit, sms, order, tokens=None):
    T, B = cu[-1] if tokens is None else tokens, len(ctx)
    slots = (T // (256 // (H // Hkv)) + min(B, T)) * Hkv + sms  # as the host sizes the workspace
    head = [int(paged), B, T, H, Hkv, limit, sms, slots, len(order)]
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


@pytest.mark.parametrize("lens,more", [([5], 0), ([5], 3000), ([300, 1, 0, 64, 65], 700), ([1] * 40, 2000),
                                       ([40 * i % 173 for i in range(50)], 500), ([700], 0), ([9, 4], -6)])
@pytest.mark.parametrize("H,Hkv", [(2, 2), (8, 2), (8, 1)])
@pytest.mark.parametrize("ctas", [1, 7, 148])
def test_a_deal_covers_every_key_tile_and_no_two_parts_share_a_place(emulator, lens, more, H, Hkv, ctas):
    rng = random.Random(len(lens) + H + ctas)
    ctx = [max(0, n + (rng.randrange(more) if more > 0 else more)) for n in lens]
    cu, T = boundaries(lens), sum(lens)
    TM, group = 256 // (H // Hkv), H // Hkv
    lines = ask(emulator, "deal", True, cu, ctx, H, Hkv, max(ctx + [1]), ctas, [])
    slots = (T // TM + min(len(lens), T)) * Hkv + ctas
    chains, walked = {}, [0] * ctas
    for line in lines:
        if line[0] == 1:
            cta, s, tok0, kvh, j0, j1, slot, parts = line[1:]
            chains.setdefault((s, tok0, kvh), []).append((j0, j1, slot, parts))
            walked[cta] += j1 - j0
    assert set(chains) == tiles_of(lens, H, Hkv)
    tiles = [max(-(-c // 128), 1) for c in ctx]
    for (s, _, _), pieces in chains.items():
        pieces.sort()
        assert pieces[0][0] == 0 and pieces[-1][1] == tiles[s]
        assert all(a[1] == b[0] and a[2] + 1 == b[2] for a, b in zip(pieces, pieces[1:]))
        assert all(p[3] == len(pieces) for p in pieces)
    places = [p[2] for pieces in chains.values() for p in pieces]
    assert len(set(places)) == len(places) and 0 <= min(places) and max(places) < slots
    sum_tiles = sum(walked)
    longest = max(t for t, n in zip(tiles, lens) if n)
    assert max(walked) == min(sum_tiles, max(-(-sum_tiles // ctas), min(longest, 4)))
    seen = set()
    for line in lines:
        if line[0] == 2:
            s, i, h, slot, parts, row = line[1:]
            pieces = chains[(s, i // TM * TM, h // group)]
            assert (slot, parts) == (pieces[0][2], len(pieces))
            assert row == i % TM * group + h % group < 256
            seen.add((s, i, h))
    assert len(seen) == T * H


def test_a_deal_of_overlapping_boundaries_stays_within_the_workspace(emulator):
    # 5 sequences that each claim all 1000 rows: flagged, and more chains than the workspace has places for
    cu = [0, 1000] * 5 + [0]
    lines = ask(emulator, "deal", True, cu, [2000] * 10, 8, 2, 2000, 7, [], tokens=1000)
    slots = (1000 // 64 + 10) * 2 + 7
    places = [line[7] for line in lines if line[0] == 1] + [line[4] for line in lines if line[0] == 2]
    assert max(places) == slots - 1 and min(places) >= 0
