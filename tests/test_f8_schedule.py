"""The main loop of the 256 x 256 tiles of the 8-bit floating-point products, as the compiler makes it: the copies of the next
steps stay in flight."""

import os
import re
import subprocess

import pytest

from gemv_layers_amd import build as b

pytestmark = pytest.mark.skipif(not os.path.exists(b.HIPCC), reason="no hipcc")


def loop_of(asm, kernel):
    """The instructions of the loop of `kernel` that holds its matrix instructions."""
    body = re.search(r"^_ZN3glk\d+%s\w*:[^\n]*\n(.*?)\.Lfunc_end" % kernel, asm, re.S | re.M).group(1)
    loops, header = {}, None
    for line in body.splitlines():
        label = re.match(r"\.L(BB\w+):(.*)", line)
        if label:
            inside = re.search(r"Header=(BB\w+)", label.group(2))
            header = label.group(1) if "Loop Header" in label.group(2) else inside.group(1) if inside else None
        elif header and line.strip() and line.strip()[0] not in ";.":
            loops.setdefault(header, []).append(line.strip())
    return max(loops.values(), key=lambda v: sum(x.startswith("v_mfma") for x in v))


def test_the_loop_of_256_tiles_keeps_copies_in_flight(tmp_path):
    out = str(tmp_path / "f8_tile.s")
    subprocess.run([b.HIPCC, *b.COMMON, "-x", "hip", "--offload-device-only", "-S", os.path.join(b.CSRC, "f8_tile.hip"), "-o", out],
                   check=True, capture_output=True)
    loop = loop_of(open(out).read(), "f8_pp_kernel")
    assert sum(x.startswith("v_mfma") for x in loop) == 32
    waits = [int(m.group(1)) for x in loop if (m := re.search(r"s_waitcnt.*vmcnt\((\d+)\)", x))]
    assert waits == [4], waits                             # the copies of the step itself
