"""The workspace of the norm's gradient lies on 4 bytes, so its vectors may be no more aligned than that in the
code's own terms (CPU; hipcc cross-compiles to LLVM IR).  In the kernels of a bf16 stream the workspace is all that is
stored in fp32."""
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "fp4_grouped_gemm_quantize_amd", "csrc")
HIPCC = "/opt/rocm/bin/hipcc"


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    if not os.path.exists(HIPCC):
        pytest.fail("hipcc is required to compile the kernels")
    out = str(tmp_path_factory.mktemp("ir") / "norm.ll")
    res = subprocess.run([HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "-Xclang", "-target-feature", "-Xclang",
                          "-packed-fp32-ops", "-I", os.path.join(ROOT, "include"), "-I", CSRC, "--cuda-device-only",
                          "-S", "-emit-llvm", os.path.join(CSRC, "norm.hip"), "-o", out],
                         capture_output=True, text=True, timeout=600)
    assert res.returncode == 0, res.stderr[-4000:]
    bodies = re.findall(r"^define [^\n]*@(_Z\w+)\([^\n]*\{\n(.*?)^\}", open(out).read(), re.M | re.S)
    return {n: b for n, b in bodies if "rmsnorm_backward" in n and "Lb0E" in n}


def test_kernels_of_a_bf16_stream(kernels):
    assert len(kernels) == 5, list(kernels)


def test_workspace_stores_take_4_bytes_alignment(kernels):
    for name, body in kernels.items():
        aligns = re.findall(r"store (?:<\d+ x )?float>? [^\n]*addrspace\(1\)[^\n]*align (\d+)", body)
        assert aligns and set(aligns) == {"4"}, (name, aligns)


def test_workspace_loads_take_4_bytes_alignment(kernels):
    """The kernel of long rows keeps its sums in the workspace and reads them back as vectors of their own type."""
    long_rows = [b for n, b in kernels.items() if "long" in n]
    aligns = re.findall(r"load <\d+ x float>, [^\n]*addrspace\(1\)[^\n]*align (\d+)", long_rows[0])
    assert aligns and set(aligns) == {"4"}, aligns
