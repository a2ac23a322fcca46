"""A row_of_slot that names a row twice, where the block-128 scatter writes through it:
refused under MXG_VALIDATE.  The check runs on the CPU under AddressSanitizer and
UndefinedBehaviorSanitizer with host-only stand-ins for the launchers, and on the GPU
through the binding."""
import os
import shutil
import subprocess

import pytest
import torch

import fp4_grouped_gemm_quantize_amd as mxg

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SAN = os.path.join(ROOT, "tests", "sanitize")
CSRC = os.path.join(ROOT, "fp4_grouped_gemm_quantize_amd", "csrc")
HIP_INCLUDE = "/opt/rocm/include"


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir(HIP_INCLUDE),
                    reason="g++ or the HIP headers not installed")
def test_check_under_sanitizers(tmp_path):
    exe = str(tmp_path / "abi_rows_driver")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__", "-I", HIP_INCLUDE, "-I", os.path.join(ROOT, "include"),
           "-I", CSRC, os.path.join(CSRC, "api_moe.cpp"), os.path.join(SAN, "abi_rows_driver.cpp"), "-o", exe]
    res = subprocess.run(cmd, cwd=tmp_path, capture_output=True, text=True, timeout=240)
    assert res.returncode == 0, res.stderr
    res = subprocess.run([exe], cwd=tmp_path, capture_output=True, text=True, timeout=120)
    out = res.stdout + res.stderr
    assert res.returncode == 0 and "fails 0" in out, out[-4000:]
    for marker in ("runtime error", "ERROR: AddressSanitizer", "ERROR: LeakSanitizer"):
        assert marker not in out, out[-4000:]


@pytest.mark.gpu
def test_scatter_of_a_repeated_row(monkeypatch):
    S, k, K, T = 2, 2, 160, 6
    x = torch.randn((S, K), device="cuda").to(torch.bfloat16)
    off = torch.tensor([1, 3, 5], dtype=torch.int32, device="cuda")  # rows 0 and 5 lie in no group
    monkeypatch.setenv("MXG_VALIDATE", "1")

    def scatter(*rows):
        q = torch.full((T, K), 0xA5, dtype=torch.uint8, device="cuda")
        s = torch.full((T, 2), 7.0, device="cuda")
        ros = torch.tensor(rows, dtype=torch.int32, device="cuda")
        try:
            mxg.mx_grouped_quantize_block128_scatter(x, ros, q, s, off)
        finally:
            kept = {r for r in range(T) if torch.all(q[r] == 0xA5) and torch.all(s[r] == 7.0)}
            written.append(set(range(T)) - kept)

    written = []
    scatter(4, 1, -1, 2)
    assert mxg.validation_message() == "" and written.pop() == {1, 2, 4}
    scatter(0, 0, 5, 5)  # dropped as often as they are named
    assert mxg.validation_message() == "" and written.pop() == set()
    for rows in ((4, 1, 4, 2), (1, 3, 1, -1)):
        with pytest.raises(mxg.MxgError) as e:
            scatter(*rows)
        assert e.value.status == mxg.ERROR_INVALID_VALUE and "again" in mxg.validation_message()
        assert written.pop() == set()
