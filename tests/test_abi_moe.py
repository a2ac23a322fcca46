"""The C ABI of the router, the routing plan, the block-128 FP8 format and their
gradients, on the CPU: bad arguments are refused with the documented status
before anything touches the GPU, and empty problems are no-ops.  The layer also
runs under AddressSanitizer and UndefinedBehaviorSanitizer with host-only
stand-ins for its launchers (tests/sanitize/abi_moe_driver.cpp)."""
import ctypes
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

P = ctypes.c_void_p
A = P(0x10000)      # never dereferenced: validation fails before any launch
ODD = P(0x10001)    # misaligned for everything
A4 = P(0x10004)     # aligned to 4 bytes only
A2 = P(0x10002)     # aligned to 2 bytes only
INVALID, UNSUPPORTED, OK = mxg.ERROR_INVALID_VALUE, mxg.ERROR_NOT_SUPPORTED, mxg.SUCCESS
BIG = 2 ** 31 - 1

# name -> (arguments that would launch, [(position, bad value, status)], [(position, value) that make it a no-op])
CASES = {
    "mx_moe_topk": (
        [0, 0, A, A, 4, 64, 8, 1, 1.0, A, A, None],
        [(0, 2, INVALID), (0, -1, INVALID), (1, 2, INVALID), (2, None, INVALID), (2, A2, INVALID), (3, ODD, INVALID),
         (4, -1, INVALID), (5, 0, INVALID), (6, 0, INVALID), (9, None, INVALID), (9, ODD, INVALID),
         (10, None, INVALID), (10, A2, INVALID), (5, 1025, UNSUPPORTED), (6, 65, UNSUPPORTED), (5, 7, UNSUPPORTED),
         (4, BIG // 8 + 1, UNSUPPORTED)],
        [(4, 0)]),
    "mx_moe_topk_backward": (
        [1, 1, A, A, A, 4, 64, 8, 1, 1.0, A, None],
        [(0, 5, INVALID), (1, -1, INVALID), (2, None, INVALID), (2, ODD, INVALID), (3, None, INVALID),
         (3, A2, INVALID), (4, None, INVALID), (4, A2, INVALID), (5, -1, INVALID), (6, 0, INVALID), (7, 0, INVALID),
         (10, None, INVALID), (10, ODD, INVALID), (6, 1025, UNSUPPORTED), (7, 65, UNSUPPORTED),
         (5, BIG // 8 + 1, UNSUPPORTED)],
        [(5, 0)]),
    "mx_moe_sort": (
        [A, 4, 8, 64, A, A, A, None],
        [(0, None, INVALID), (0, A2, INVALID), (1, -1, INVALID), (2, 0, INVALID), (3, 0, INVALID), (4, None, INVALID),
         (4, A2, INVALID), (5, None, INVALID), (5, ODD, INVALID), (6, None, INVALID), (6, ODD, INVALID),
         (3, 1025, UNSUPPORTED), (1, BIG // 8 + 1, UNSUPPORTED)],
        []),
    "mx_moe_permute": (
        [A, 4, 64, A, 8, A, 32, None],
        [(0, None, INVALID), (0, A4, INVALID), (1, -1, INVALID), (2, 0, INVALID), (3, None, INVALID),
         (3, A2, INVALID), (4, 0, INVALID), (5, None, INVALID), (5, A4, INVALID), (6, -1, INVALID),
         (2, 60, UNSUPPORTED), (1, BIG // 8 + 1, UNSUPPORTED)],
        [(1, 0), (6, 0)]),
    "mx_moe_permute_backward": (
        [A, 32, 64, A, 4, 8, A, None],
        [(0, None, INVALID), (0, A4, INVALID), (1, -1, INVALID), (2, -8, INVALID), (3, None, INVALID),
         (3, A2, INVALID), (4, -1, INVALID), (5, 0, INVALID), (6, None, INVALID), (6, A4, INVALID),
         (2, 4, UNSUPPORTED), (4, BIG // 8 + 1, UNSUPPORTED)],
        [(4, 0)]),
    "mx_moe_combine_backward": (
        [A, A, 32, 64, A, A, 4, 8, A, A, None],
        [(0, None, INVALID), (0, A4, INVALID), (1, None, INVALID), (1, A4, INVALID), (2, -1, INVALID),
         (3, 0, INVALID), (4, None, INVALID), (4, A2, INVALID), (5, None, INVALID), (5, A2, INVALID),
         (6, -1, INVALID), (7, 0, INVALID), (8, None, INVALID), (8, A4, INVALID), (9, None, INVALID),
         (9, A2, INVALID), (3, 12, UNSUPPORTED), (6, BIG // 8 + 1, UNSUPPORTED)],
        [(6, 0)]),
    "mx_grouped_quantize_block128": (
        [A, A, A, A, 2, 16, 256, None],
        [(0, None, INVALID), (0, A4, INVALID), (1, None, INVALID), (1, A4, INVALID), (2, None, INVALID),
         (2, A2, INVALID), (3, None, INVALID), (3, A2, INVALID), (4, -1, INVALID), (5, -1, INVALID), (6, 0, INVALID),
         (6, 48, UNSUPPORTED), (4, 1025, UNSUPPORTED), (5, BIG + 1, UNSUPPORTED), (6, 2 ** 31, UNSUPPORTED)],
        [(4, 0), (5, 0)]),
    "mx_grouped_quantize_block128_scatter": (
        [A, 4, A, 8, A, A, A, 2, 32, 256, None],
        [(0, None, INVALID), (0, A4, INVALID), (1, -1, INVALID), (2, None, INVALID), (2, A2, INVALID),
         (3, 0, INVALID), (4, None, INVALID), (4, A4, INVALID), (5, None, INVALID), (5, A2, INVALID),
         (6, None, INVALID), (6, A2, INVALID), (7, -1, INVALID), (8, -1, INVALID), (9, -32, INVALID),
         (9, 33, UNSUPPORTED), (3, 65, UNSUPPORTED), (1, BIG // 8 + 1, UNSUPPORTED), (7, 1025, UNSUPPORTED)],
        [(1, 0), (7, 0), (8, 0)]),
    "mx_quantize_weights_block128": (
        [A, 2, 128, 256, A, A, A, A, None],
        [(0, None, INVALID), (0, A4, INVALID), (1, 0, INVALID), (2, 0, INVALID), (3, 0, INVALID), (4, None, INVALID),
         (4, A4, INVALID), (5, None, INVALID), (5, A2, INVALID), (6, None, INVALID), (6, A4, INVALID),
         (7, None, INVALID), (7, A2, INVALID), (2, 100, UNSUPPORTED), (3, 48, UNSUPPORTED),
         (2, 2 ** 30, UNSUPPORTED), (3, 2 ** 30, UNSUPPORTED)],
        []),
    "mx_grouped_matmul_block128": (
        [A, A, A, A, A, A, A, 2, 4, 16, 256, 256, 0, None],
        [(i, None, INVALID) for i in range(7)] + [(0, A4, INVALID), (1, A2, INVALID), (2, A4, INVALID),
         (3, A2, INVALID), (4, A4, INVALID), (5, A2, INVALID), (6, A2, INVALID), (7, -1, INVALID), (8, 0, INVALID),
         (9, -1, INVALID), (10, 0, INVALID), (11, 0, INVALID), (11, 16, UNSUPPORTED),
         (11, mxg.MAX_K + 32, UNSUPPORTED), (7, 1025, UNSUPPORTED), (10, 2 ** 30, UNSUPPORTED),
         (9, 2 ** 31, UNSUPPORTED)],
        [(7, 0), (9, 0)]),
    "mx_silu_quantize_block128": (
        [A, A, A, A, 2, 16, 256, None],
        [(i, None, INVALID) for i in range(4)] + [(0, A4, INVALID), (1, A4, INVALID), (2, A2, INVALID),
         (3, A2, INVALID), (4, -1, INVALID), (5, -1, INVALID), (6, 0, INVALID), (6, 40, UNSUPPORTED),
         (4, 1025, UNSUPPORTED), (6, 2 ** 29, UNSUPPORTED)],
        [(4, 0), (5, 0)]),
    "mx_silu_backward_block128": (
        [A, A, A, A, A, A, 2, 16, 256, None],
        [(0, None, INVALID), (0, A4, INVALID), (1, None, INVALID), (1, A4, INVALID), (2, A4, INVALID),
         (3, None, INVALID), (3, A4, INVALID), (4, None, INVALID), (4, A2, INVALID), (5, None, INVALID),
         (5, A2, INVALID), (6, -1, INVALID), (7, -1, INVALID), (8, 0, INVALID), (8, 40, UNSUPPORTED),
         (6, 1025, UNSUPPORTED)],
        [(6, 0), (7, 0)]),
}


@pytest.mark.parametrize("name", sorted(CASES))
def test_refusals(name):
    good, bad, empty = CASES[name]
    call = getattr(mxg.lib(), name)
    for at, value, status in bad:
        args = list(good)
        args[at] = value
        assert call(*args) == status, (at, value)
    for at, value in empty:
        args = list(good)
        args[at] = value
        assert call(*args) == OK, (at, value)
        if (name, at) != ("mx_moe_permute", 6):  # without work no pointer is examined (there: only the rows' may be null)
            assert call(*[None if a is A else a for a in args]) == OK, (at, value)


def test_both_gradient_outputs_missing():
    good = list(CASES["mx_silu_backward_block128"][0])
    good[2] = good[3] = good[4] = None
    assert mxg.lib().mx_silu_backward_block128(*good) == INVALID


@pytest.mark.parametrize("name,at", [("mx_moe_permute", 2), ("mx_moe_permute_backward", 2),
                                     ("mx_moe_combine_backward", 3)])
def test_rows_too_long(name, at):
    args = list(CASES[name][0])
    args[at] = 2 ** 31
    assert getattr(mxg.lib(), name)(*args) == UNSUPPORTED


def test_binding_refuses_wrong_tensors():
    """dtype, shape and device are checked before the library is called."""
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    i32 = torch.zeros((4, 2), dtype=torch.int32)
    f32 = torch.zeros((4, 2))
    with pytest.raises(ValueError, match="GPU tensor"):
        mxg.mx_moe_topk(mxg.SCORE_SOFTMAX, x, i32, f32)
    with pytest.raises(TypeError):
        mxg.mx_moe_topk(mxg.SCORE_SOFTMAX, x.half(), i32, f32)
    with pytest.raises(TypeError):
        mxg.mx_moe_sort(f32, i32, i32, i32)
    with pytest.raises(ValueError, match="GPU tensor"):
        mxg.mx_moe_permute(x, i32, x)
    with pytest.raises(TypeError):
        mxg.mx_grouped_quantize_block128(f32, i32, f32, i32)
    with pytest.raises(TypeError):
        mxg.mx_grouped_matmul_block128(x, f32, x, f32, x, i32, i32)


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir(HIP_INCLUDE),
                    reason="g++ or the HIP headers not installed")
def test_abi_layer_under_sanitizers(tmp_path):
    exe = str(tmp_path / "abi_moe_driver")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__", "-I", HIP_INCLUDE, "-I", os.path.join(ROOT, "include"),
           "-I", CSRC, os.path.join(CSRC, "api_moe.cpp"), os.path.join(SAN, "abi_moe_driver.cpp"), "-o", exe]
    res = subprocess.run(cmd, cwd=tmp_path, capture_output=True, text=True, timeout=240)
    assert res.returncode == 0, res.stderr
    res = subprocess.run([exe], cwd=tmp_path, capture_output=True, text=True, timeout=120)
    out = res.stdout + res.stderr
    assert res.returncode == 0 and "fails 0" in out, out[-4000:]
    for marker in ("runtime error", "ERROR: AddressSanitizer", "ERROR: LeakSanitizer"):
        assert marker not in out, out[-4000:]
