"""The planner of the 8-bit and training products, its rules restated here and checked at several sizes of
card (op_plan_check.cpp prints the plans of the built library)."""

import json
import os
import random
import shutil
import subprocess
from math import isqrt

import pytest

import gemv_layers_amd as g

HERE = os.path.dirname(os.path.abspath(__file__))
PKG = os.path.join(os.path.dirname(HERE), "gemv_layers_amd")
CUS = (80, 228, 256, 304)
WS_FLOATS, WS_COUNTERS = 8 << 20, 1 << 16

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="no host C++ compiler")


def cdiv(a, b):
    return -(-a // b)


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    """plans([(kind, M, N, K, cus, glu, contiguous), ...]) -> [{"plan", "counters", "fits"}, ...]"""
    exe = str(tmp_path_factory.mktemp("plan") / "op_plan_check")
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", f"-I{os.path.join(PKG, 'csrc')}",
                    os.path.join(HERE, "op_plan_check.cpp"), os.path.join(PKG, "libgemm_bf16.so"), f"-Wl,-rpath,{PKG}",
                    "-Wl,--allow-shlib-undefined", "-o", exe], check=True)

    def run(asked):
        text = "".join(" ".join(str(int(x) if not isinstance(x, str) else x) for x in a) + "\n" for a in asked)
        r = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=120, check=True)
        out = [json.loads(line) for line in r.stdout.splitlines()]
        assert len(out) == len(asked)
        return out

    return run


def small_tiles(M, W, K, cus):
    """(tiles, pieces, k-steps a piece) where the output takes 64 x 64 tiles, else None."""
    tm, tn, kt = cdiv(M, 64), cdiv(W, 64), cdiv(K, 32)
    tiles = tm * tn
    if tiles > 2 * cus or (tiles * kt > (32768 if tm == 1 else 16384) and tiles > cus // 4):
        return None
    s = min(max(1, isqrt(kt // 6)), max(kt // 28, cus // tiles), 16, 3 * cus // tiles)
    if cus < tiles * s <= cus + cus // 2:
        s = cus // tiles
    s = max(s, 1)
    while s > 1 and tiles * s * 4096 > WS_FLOATS // 2:
        s -= 1
    per = cdiv(kt, s)
    return tiles, cdiv(kt, per), per


def shapes(seed, n, lo=65):
    rng = random.Random(seed)
    size = lambda a, b: int(a * (b / a) ** rng.random())  # noqa: E731
    return [(size(lo, 9000), size(1, 12000), size(1, 24000), rng.choice(CUS), rng.random() < 0.4, rng.random() < 0.5)
            for _ in range(n)]


def test_tile_plans_follow_their_rules(plans):
    asked = shapes(1, 3000)
    seen = set()
    for (M, N, K, cus, glu, contiguous), got in zip(asked, plans([("tile", *a) for a in asked])):
        p, W, kt = got["plan"], 2 * N if glu else N, cdiv(K, 32)
        what = (M, N, K, cus, glu, contiguous, p)
        small = small_tiles(M, W, K, cus)
        if small:
            tiles, splits, per = small
            assert (p["bm"], p["tiles"], p["splits"], p["kt_per_split"]) == (64, tiles, splits, per), what
            assert "cut" not in p
            seen.add(("64", splits > 1))
        else:
            # the plan of the plain bf16 product over the weight's columns, but for one rule
            q = g.gemm_plan_describe(M, W, K, cus)
            splits, per = q["splits"], q["kt_per_split"]
            if q["bm"] == 128 and splits == 2 and 3 * q["tiles"] > 2 * cus:
                if kt < (200 if contiguous else 120):
                    splits, per = 1, kt
                else:
                    per += per % 2
                seen.add(("rule", splits, contiguous))
            assert (p["bm"], p["tiles"], p["splits"], p["kt_per_split"]) == (q["bm"], q["tiles"], splits, per), what
            assert ("cut" in p) == ("cut" in q), what
            if "cut" in p:
                c, d = p["cut"], q["cut"]
                half = 2 if glu and c["axis"] == "n" else 1    # columns of outputs: half those of the weight
                assert c["axis"] == d["axis"] and c["at"] == d["at"] // half, what
                assert c["rest"]["bm"] == 128 and c["rest"]["tiles"] == d["rest"]["tiles"], what
                assert c["at"] % (256 // half) == 0
                seen.add(("cut", c["axis"], glu))
        for r in (p, p["cut"]["rest"]) if "cut" in p else (p,):
            # whole pieces cover K, none is empty, and the grid is theirs
            assert r["splits"] == cdiv(kt, r["kt_per_split"]) and (r["splits"] - 1) * r["kt_per_split"] < kt, what
            assert r["grid"] == r["tiles"] * r["splits"], what
            if r["splits"] > 1:
                assert r["bm"] < 256 and r["ws_floats"] == r["grid"] * r["bm"] ** 2 <= WS_FLOATS, what
        assert got["counters"] <= WS_COUNTERS
    assert seen >= {("64", True), ("64", False), ("rule", 1, True), ("rule", 2, True), ("rule", 1, False), ("rule", 2, False),
                    ("cut", "n", False), ("cut", "m", False), ("cut", "n", True), ("cut", "m", True)}, seen


@pytest.mark.parametrize("cus", CUS)
def test_two_pieces_where_they_pay(plans, cus):
    """128 x 128 tiles on more than two thirds of the CUs: whole below 200 k-steps (120 with a strided
    operand), from there two pieces of even numbers of k-steps."""
    for tiles in (2 * cus // 3 + 1, min(cus, 256)):       # (the workspace holds two pieces of 256 tiles)
        # (a long column of tiles: 64 x 64 ones would be more than two a CU and 16384 k-steps)
        M, N = 128 * tiles, 128
        for kt in (96, 119, 120, 121, 141, 199, 200, 201, 344, 345, 688):
            for contiguous in (False, True):
                p = plans([("tile", M, N, 32 * kt, cus, False, contiguous)])[0]["plan"]
                assert (p["bm"], p["tiles"]) == (128, tiles)
                two = kt >= (200 if contiguous else 120)
                assert p["splits"] == (2 if two else 1), (tiles, kt, contiguous, p)
                if two:
                    assert p["kt_per_split"] % 2 == 0 and 0 <= 2 * p["kt_per_split"] - kt <= 3
                    assert p["ws_floats"] == 2 * tiles * 128 * 128 <= WS_FLOATS


# (row tiles, weight tiles, waves, gated) that launch_i8_decode has: from codes, and from one bf16 row
DECODE = ({(1, tn, nw, False) for tn, nw in ((1, 4), (1, 8), (4, 4))} | {(1, 2, 4, True)} |
          {(mt, tn, nw, False) for mt in (2, 3, 4) for tn, nw in ((1, 4), (1, 8), (2, 4), (4, 8))} |
          {(mt, tn, 4, True) for mt in (2, 3, 4) for tn in (2, 4)})


def test_decode_plans_follow_their_rules(plans):
    rng = random.Random(2)
    asked = [(rng.randint(1, 64) if rng.random() < 0.7 else rng.randint(1, 5), int(200 ** rng.random() * 100) + rng.randint(0, 20),
              int(131071 ** rng.random()), rng.choice(CUS), rng.random() < 0.4, 0) for _ in range(4000)]
    seen = set()
    for (M, N, K, cus, glu, _), got in zip(asked, plans([("decode", *a) for a in asked])):
        p = got["plan"]
        what = (M, N, K, cus, glu, p)
        mt, tiles, steps, weight = cdiv(M, 16), cdiv(N, 16), cdiv(K, 64), (2 if glu else 1) * N * K
        if glu:
            tn = 4 if mt > 1 and weight > 20 << 20 else 2
        elif mt == 1:
            tn = 1 if M <= 4 or tiles <= 2 * cus else 4
        else:
            tn = 1 if weight <= 8 << 20 else 2 if weight <= 20 << 20 else 4
        groups = cdiv(tiles, tn // 2 if glu else tn)
        s = max(1, min(cus // groups, steps // 32))
        while s > 1 and groups * s * tn * mt * 256 > WS_FLOATS:
            s -= 1
        wide = (tn == 1 and groups * s < 2 * cus and steps >= 128) or (not glu and tn == 4 and mt > 1)
        assert (p["mtiles"], p["strip"], p["strips"], p["splits"], p["grid"], p["threads"]) == (
            mt, 16 * tn, groups, s, groups * s, 512 if wide else 256), what
        assert p["ws_floats"] == (groups * s * tn * mt * 256 if s > 1 else 0), what
        assert got["counters"] == (groups if s > 1 else 0) and got["counters"] <= WS_COUNTERS, what
        assert got["fits"] == (groups * M * K <= 22_000_000), what
        if got["fits"]:
            seen.add((mt, tn, 8 if wide else 4, glu))
            if s > 1:
                seen.add("pieces")
    assert "pieces" in seen
    seen.discard("pieces")
    assert seen <= DECODE and DECODE - seen == set(), (seen - DECODE, DECODE - seen)
