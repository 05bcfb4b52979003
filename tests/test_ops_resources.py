"""Compile-time checks of the operators' kernels (CPU only: hipcc
cross-compiles gfx950): no register array in scratch memory, except in the
norms' gradient and fused combine for rows of more than 8192 elements, whose
1024 threads have half the registers."""
import concurrent.futures as cf
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "combine_symmetric_memory_amd", "csrc")
FILES = ["route.hip", "block_norm.hip", "group_product.hip", "group_dx.hip", "group_dw.hip"]

pytestmark = pytest.mark.skipif(
    shutil.which("hipcc") is None and not os.path.exists("/opt/rocm/bin/hipcc"),
    reason="hipcc not available")


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    """{file: assembly}, compiled side by side."""
    from combine_symmetric_memory_amd.build import HIPCC_FLAGS, hipcc
    out = tmp_path_factory.mktemp("asm")

    def one(src):
        to = str(out / (src + ".s"))
        r = subprocess.run([hipcc(), *HIPCC_FLAGS, "-x", "hip", "--cuda-device-only", "-S",
                            os.path.join(CSRC, src), "-o", to], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-2000:]
        return open(to).read()

    with cf.ThreadPoolExecutor(max_workers=len(FILES)) as ex:
        return dict(zip(FILES, ex.map(one, FILES)))


@pytest.mark.parametrize("src", FILES)
def test_no_scratch(asm, src):
    kernels = re.findall(r"\.name:\s+(_Z\S+)\n\s+\.private_segment_fixed_size:\s+(\d+)", asm[src])
    assert kernels, "no kernels found in " + src
    for name, size in kernels:
        if re.search(r"(norm_grad|combine_norm)_kernelI.*Li1024E", name):
            continue
        # fp32 rows that end inside a vector fill the gradient's registers
        # (12 of some 270 spill)
        limit = 64 if re.search(r"norm_grad_kernelILNS0_6RowEndE1EfLi2E", name) else 0
        assert int(size) <= limit, "%s uses %s bytes of scratch" % (name, size)


@pytest.mark.parametrize("src", FILES[2:])
def test_tile_loops_stay_in_registers(asm, src):
    # the MFMA loops of the fast kernel: no scratch, no moves between the
    # accumulation registers and the others
    text, seen = asm[src], 0
    for fn in re.findall(r"^(\S*group_tile_kernel\S*):", text, re.M):
        body = text[text.index("\n" + fn + ":"):]
        body = body[:body.index(".Lfunc_end")]
        for b in re.split(r"\n(?=\.LBB\d+_\d+:)", body):
            if b.count("v_mfma") < 32 or "buffer_load_dwordx4" not in b:
                continue
            seen += 1
            assert "scratch_" not in b and "v_accvgpr" not in b, fn
    assert seen >= 10


@pytest.mark.parametrize("src", FILES)
def test_wide_buffer_stores_have_no_scalar_offset(asm, src):
    # Behind a buffer store of more than 8 bytes a lane with a scalar register
    # in its offset the compiler keeps no distance to the next write of the
    # stored registers, and such a write reached what some lanes store.
    bad = re.findall(r"buffer_store_dwordx[34] [^\n]*, s\d+ offen", asm[src])
    assert not bad, bad[:3]
    if src in FILES[2:]:
        assert re.search(r"buffer_store_dwordx4 [^\n]*, 0 offen", asm[src])
