"""The planner of the products grouped by rows: whatever rows the groups turn out to have, the grid covers their
tiles, the workspace their pieces, and no piece of K starts past the end (group_plan_check.cpp prints the plans
of the built library)."""

import json
import os
import random
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
PKG = os.path.join(os.path.dirname(HERE), "gemv_layers_amd")
CUS = (80, 228, 256, 304)
WS_FLOATS, WS_COUNTERS = 8 << 20, 1 << 16

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="no host C++ compiler")


def cdiv(a, b):
    return -(-a // b)


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    """plans([(kind, rows, groups, M, N, K, summed, pairs, strided, cus), ...]) -> [{"plan", "counters", "tail", "fits"}, ...]"""
    exe = str(tmp_path_factory.mktemp("plan") / "group_plan_check")
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", f"-I{os.path.join(PKG, 'csrc')}",
                    os.path.join(HERE, "group_plan_check.cpp"), os.path.join(PKG, "libgemm_bf16.so"), f"-Wl,-rpath,{PKG}",
                    "-Wl,--allow-shlib-undefined", "-o", exe], check=True)

    def run(asked):
        text = "".join(" ".join(str(int(x) if not isinstance(x, str) else x) for x in a) + "\n" for a in asked)
        r = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=120, check=True)
        out = [json.loads(line) for line in r.stdout.splitlines()]
        assert len(out) == len(asked)
        return out

    return run


def size(rng, lo, hi):
    return int(lo * (hi / lo) ** rng.random())


def parts(rng, rows, groups):
    """Rows of each group, and of none before and after them: a few offsets at random, many, or all in one."""
    n = rng.choice([0, 1, groups])
    cuts = sorted([rng.randint(0, rows) for _ in range(n)] + rng.choices([0, rows], k=groups + 1 - n))
    return [b - a for a, b in zip([0, *cuts], [*cuts, rows])]


def test_tile_plans_hold_whatever_rows_groups_have(plans):
    rng = random.Random(1)
    asked = []
    for _ in range(4000):
        rows, groups, summed, pairs = size(rng, 1, 20000), size(rng, 1, 300), rng.random() < 0.3, rng.random() < 0.5
        if not summed and rng.random() < 0.2:
            groups = 0                                     # all rows are one's
        asked.append(("tile", rows, groups, size(rng, 1, 12000), size(rng, 1, 12000), size(rng, 1, 30000), summed,
                      pairs and not summed, not pairs and not summed and rng.random() < 0.5, rng.choice(CUS)))
    seen = set()
    for a, got in zip(asked, plans(asked)):
        _, rows, groups, M, N, K, summed, pairs, strided, cus = a
        p, kt = got["plan"], cdiv(K, 32)
        bm, splits, per = p["bm"], p["splits"], p["kt_per_split"]
        assert p["tiles_n"] == cdiv(N, bm), a
        if summed:
            tiles = groups * cdiv(M, bm) * p["tiles_n"]
            assert p["tiles"] == tiles, a
        else:
            tiles = 0
            for _ in range(3):
                cut = parts(rng, rows, groups) if groups else [rows]
                tiles = max(tiles, sum(cdiv(r, bm) for r in cut) * p["tiles_n"])
            assert tiles <= p["tiles"] == p["tiles_m"] * p["tiles_n"], a
            if groups == 0:
                assert tiles == p["tiles"], a
            assert per * splits >= kt and per * (splits - 1) < max(kt, 1), (a, p)   # all of K, and no empty piece
            assert not pairs or per % 2 == 0, a
        slots = WS_FLOATS // 65536
        tail = got["tail"] > 1                             # 256 x 256: tiles of a last round in pieces
        assert not tail or (bm == 256 and splits == 1 and not summed and got["tail"] <= 8 and got["tail"] ** 2 <= kt // (4 if pairs else 8)), (a, p)
        extra = slots if tail else 0
        if tail and groups == 0:                           # the tiles are known: as many as there are
            rest = p["tiles"] % cus
            pieces = min(slots // rest, cus // rest, got["tail"])
            assert pieces > 1, (a, p)
            extra = rest * (pieces - 1)
        assert p["grid"] == p["tiles"] * splits + extra, a
        if tail:
            assert p["ws_floats"] == slots * 65536 <= WS_FLOATS and got["counters"] == slots, a
        elif splits > 1:
            assert bm < 256 and p["ws_floats"] == p["grid"] * bm * bm <= WS_FLOATS // (1 if pairs or strided else 2) and got["counters"] == p["tiles"] <= WS_COUNTERS, (a, p)
        else:
            assert p["ws_floats"] == got["counters"] == 0, a
        seen.add((bm, tail or splits > 1, summed))
    assert seen >= {(64, True, False), (64, False, False), (128, False, False), (256, True, False), (256, False, False),
                    (64, False, True), (256, False, True)}, seen


@pytest.mark.parametrize("kt", [1, 2, 3, 5, 31, 33, 63, 95, 255, 256, 257, 511, 513, 1000])
def test_pieces_of_whole_blocks(plans, kt):
    """Pieces rounded up to whole blocks of 128 codes are counted after the rounding."""
    for M, N in ((1, 64), (64, 64), (65, 129), (300, 520), (200, 1000)):
        for K in (32 * kt, 32 * kt - 1, 32 * kt - 31):
            p = plans([("tile", M, 0, M, N, K, False, True, False, 256)])[0]["plan"]
            per, splits = p["kt_per_split"], p["splits"]
            assert per % 2 == 0 and per * splits >= kt and per * (splits - 1) < kt


def test_decode_plans_hold_whatever_rows_groups_have(plans):
    rng = random.Random(2)
    asked = []
    for _ in range(3000):
        groups = rng.choice([0, size(rng, 1, 300)])
        asked.append(("decode", size(rng, 1, 64 if groups == 0 else 16 * groups + 1), groups, 0, size(rng, 1, 40000), size(rng, 1, 100000),
                      False, False, False, rng.choice(CUS)))
    shapes = set()
    for a, got in zip(asked, plans(asked)):
        _, rows, groups, _, N, K, _, _, _, cus = a
        p = got["plan"]
        assert got["fits"] == (rows <= 64 if groups == 0 else rows <= 16 * groups)
        mt, tn, s = p["mtiles"], p["strip"] // 16, p["splits"]
        assert mt in (1, 2, 4) and tn in (1, 2, 4) and p["threads"] == 256 and p["strips"] == cdiv(cdiv(N, 16), tn), a
        assert rows > 1 or (mt == 1 and tn <= 2), a        # one row: the kernels that quantise it
        tiles = max(sum(cdiv(r, 16 * mt) for r in (parts(rng, rows, groups) if groups else [rows])) for _ in range(3)) * p["strips"]
        assert tiles * s <= p["grid"], a
        if s > 1:
            assert p["ws_floats"] == p["grid"] * mt * tn * 256 <= WS_FLOATS and got["counters"] == p["grid"] // s <= WS_COUNTERS, a
            assert s <= cdiv(K, 128) // (10 if mt == 1 else 4), a
        shapes.add((mt, tn))
    assert shapes == {(1, 1), (1, 2), (1, 4), (2, 1), (2, 2), (2, 4), (4, 1), (4, 2), (4, 4)}, shapes


def test_large_grids_take_larger_tiles(plans):
    """A launch holds 2^32 - 1 threads: 2^18 rows of 16384 groups (16 a group in the mean) against 70000 columns would be
    22 million 64 x 64 tiles of 256."""
    for rows, groups, N, pairs in ((1 << 18, 16384, 70000, False), (1 << 18, 16384, 70000, True), ((1 << 24) - 1, 65536, 8192, True)):
        p = plans([("tile", rows, groups, rows, N, 512, False, pairs, False, 256)])[0]["plan"]
        assert p["bm"] > 64 and p["grid"] * p["threads"] < 1 << 32, p
    small = plans([("tile", 1 << 18, 16384, 1 << 18, 64, 512, False, False, False, 256)])[0]["plan"]
    assert small["bm"] == 64 and small["grid"] * small["threads"] < 1 << 32
