"""The launches of the router choice over its whole range of tokens (CPU only): topk.hip linked with a driver that
records the launches (tests/host_san/topk_launch_driver.cpp)."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CLANGXX = "/opt/rocm/llvm/bin/clang++"

pytestmark = pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANGXX)), reason="ROCm toolchain missing")


def test_launches_cover_any_number_of_tokens(tmp_path):
    from moe_grouped_expert_amd import build as b
    objs = []
    for src in (os.path.join(ROOT, "moe_grouped_expert_amd", "csrc", "topk.hip"),
                os.path.join(ROOT, "tests", "host_san", "topk_launch_driver.cpp")):
        objs.append(str(tmp_path / (os.path.basename(src) + ".o")))
        r = subprocess.run([HIPCC, *b.FLAGS, "-O1", "-c", src, "-o", objs[-1]], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-3000:]
    exe = str(tmp_path / "topk_launch_driver")
    r = subprocess.run([CLANGXX, "-o", exe, *objs], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and "topk_launch_driver ok" in r.stdout, (r.stdout + r.stderr)[-3000:]
