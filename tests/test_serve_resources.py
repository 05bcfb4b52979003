"""Compile-time checks of the kernels of the 8-bit operators and the layer for
a few tokens (CPU only: hipcc cross-compiles gfx950)."""
import concurrent.futures as cf
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "combine_symmetric_memory_amd", "csrc")
FILES = ["quant.hip", "group_i8.hip", "moe_few.hip", "moe_few_shared.hip"]

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


def _bodies(text, kernel):
    for fn in re.findall(r"^(\S*%s\S*):" % kernel, text, re.M):
        body = text[text.index("\n" + fn + ":"):]
        yield fn, body[:body.index(".Lfunc_end")]


@pytest.mark.parametrize("src", FILES)
def test_scratch(asm, src):
    kernels = re.findall(r"\.name:\s+(_Z\S+)\n\s+\.private_segment_fixed_size:\s+(\d+)", asm[src])
    assert kernels, "no kernels found in " + src
    for name, size in kernels:
        # the streams keep 8 KiB in flight in 256 registers; a few values
        # outside their loops may not fit
        limit = 96 if src == "moe_few.hip" else 0
        assert int(size) <= limit, "%s uses %s bytes of scratch" % (name, size)


@pytest.mark.parametrize("kernel", ["few_up_kernel", "few_down_kernel"])
def test_streams_make_global_loads(asm, kernel):
    # flat loads would count as LDS operations, which LDS reads wait for
    for fn, body in _bodies(asm["moe_few.hip"], kernel):
        assert "flat_load" not in body, fn
        assert body.count("global_load_dwordx4") >= 32, fn


def test_the_shared_form_loads_straight_into_lds(asm):
    seen = 0
    for fn, body in _bodies(asm["moe_few_shared.hip"], "few_shared_down_kernel"):
        seen += 1
        assert "flat_load" not in body, fn
        assert re.search(r"buffer_load_dwordx4 [^\n]* lds", body), fn
    assert seen >= 4


def test_tile_loops_stay_in_registers(asm):
    # the 8-bit MFMA loops of the fast kernel: no scratch, no moves between the
    # accumulation registers and the others
    seen = 0
    for fn, body in _bodies(asm["group_i8.hip"], "group_tile_kernel"):
        for b in re.split(r"\n(?=\.LBB\d+_\d+:)", body):
            if b.count("v_mfma_i32_32x32x32_i8") < 32 or "buffer_load_dwordx4" not in b:
                continue
            seen += 1
            assert "scratch_" not in b and "v_accvgpr" not in b, fn
    assert seen >= 10


def test_wide_buffer_stores_have_no_scalar_offset(asm):
    # (an instruction behind such a store may change what it stores)
    text = asm["group_i8.hip"]
    assert not re.findall(r"buffer_store_dwordx[34] [^\n]*, s\d+ offen", text)
    assert re.search(r"buffer_store_dwordx4 [^\n]*, 0 offen", text)
