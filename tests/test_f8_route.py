"""Where the 8-bit floating-point products of few rows run."""

import os
import subprocess

from test_group_planner import PKG, plans, pytestmark  # noqa: F401


def test_row_tiles_of_a_group_share_an_xcd(plans):  # noqa: F811
    """Neighbouring units are the row tiles of one strip: an XCD's share of them is contiguous. A plain product has one."""
    asked = [("decode", rows, groups, 0, 4096, 4096, False, False, False, 256) for rows, groups in ((64, 8), (128, 8), (64, 64), (1000, 300), (40, 0), (1, 0))]
    for a, got in zip(asked, plans(asked)):
        assert got["plan"]["nxcd"] == (8 if a[2] else 1), a


def test_groups_of_more_rows_in_the_mean_take_tiles(tmp_path):
    """The weight is read once for every 16 rows of a group, and a router may deal all rows to one: 4 rows a group in the mean
    are the most."""
    src, exe = str(tmp_path / "route.cpp"), str(tmp_path / "route")
    with open(src, "w") as f:
        f.write("""#include <stdio.h>
#include "plan.h"
int main() {
    for (int g : {0, 1, 2, 8, 64, 65536}) {
        const long long bound = g ? 4ll * g : 64;
        for (long long rows : {1ll, bound - 1, bound, bound + 1, 2 * bound, 16ll * g + 1, 1ll << 23})
            if (glk::f8_decode_pays(rows, g) != (rows <= bound)) return printf("%lld rows in %d groups\\n", rows, g), 1;
    }
}
""")
    subprocess.run(["g++", "-O1", "-std=c++17", f"-I{os.path.join(PKG, 'csrc')}", src, os.path.join(PKG, "libgemm_bf16.so"),
                    f"-Wl,-rpath,{PKG}", "-Wl,--allow-shlib-undefined", "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
