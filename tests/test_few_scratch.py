"""Scratch of the down product's kernels of the layer for a few tokens (CPU
only: hipcc cross-compiles gfx950): a reload waits for the weights in flight."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = os.path.join(ROOT, "combine_symmetric_memory_amd", "csrc", "moe_few.hip")

pytestmark = pytest.mark.skipif(
    shutil.which("hipcc") is None and not os.path.exists("/opt/rocm/bin/hipcc"),
    reason="hipcc not available")


def test_down_products_of_one_tile_of_columns_have_none(tmp_path):
    from combine_symmetric_memory_amd.build import HIPCC_FLAGS, hipcc
    out = str(tmp_path / "few.s")
    r = subprocess.run([hipcc(), *HIPCC_FLAGS, "-x", "hip", "--cuda-device-only", "-S", SRC, "-o",
                        out], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    sizes = dict(re.findall(r"\.name:\s+(_Z\S+)\n\s+\.private_segment_fixed_size:\s+(\d+)",
                            open(out).read()))
    down = {n: int(s) for n, s in sizes.items() if "few_down_kernel" in n}
    assert len(down) == 8
    # (the last template argument: tiles of 16 rows of weights a wavefront)
    one = [n for n in down if "ELi1E" in n]
    assert len(one) == 4
    for n, size in down.items():
        assert size <= (0 if n in one else 48), "%s uses %d bytes of scratch" % (n, size)
    assert sum("few_tiny_down_kernel" in n and s == "0" for n, s in sizes.items()) == 4
