"""The scales that the FP8 block tile kernels read stay inside their tables (CPU only): the address arithmetic of fp8b.hpp,
enumerated by tests/host_san/fb_scale_reads_driver.cpp."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CLANGXX = "/opt/rocm/llvm/bin/clang++"

pytestmark = pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANGXX)), reason="ROCm toolchain missing")


def test_scale_reads_stay_in_their_tables(tmp_path):
    from moe_grouped_expert_amd import build as b
    exe, obj = str(tmp_path / "fb_scale_reads_driver"), str(tmp_path / "fb_scale_reads_driver.o")
    src = os.path.join(ROOT, "tests", "host_san", "fb_scale_reads_driver.cpp")
    for cmd in ([HIPCC, *b.FLAGS, "-c", src, "-o", obj], [CLANGXX, "-o", exe, obj]):
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "fb_scale_reads ok" in r.stdout, (r.stdout + r.stderr)[-3000:]


def test_kernel_takes_its_resources_from_there():
    """The kernel's scale resources are those that the enumeration covers."""
    with open(os.path.join(ROOT, "moe_grouped_expert_amd", "csrc", "gemm_fb.hip")) as f:
        text = f.read()
    body = text[text.index("auto setup ="):text.index("auto at_slice =")]
    made = [line.strip() for line in body.splitlines() if "o.rS = make_rsrc_n" in line]
    assert len(made) == 3 and sum("sp.at, sp.bytes" in line for line in made) == 2
    assert sum("p.src_rows" in line for line in made) == 1     # the tokens' scales as they come, by source row
