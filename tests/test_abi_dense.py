"""The C ABI of the norm, the BF16 products and their gradients, on the CPU: bad arguments are refused
with the documented status before anything touches the GPU, and empty problems are no-ops; which kernel
a product of given sizes runs.  The layer also runs under AddressSanitizer and UndefinedBehaviorSanitizer
with host-only stand-ins for its launchers (tests/sanitize/abi_dense_driver.cpp)."""
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
INVALID, UNSUPPORTED, OK = mxg.ERROR_INVALID_VALUE, mxg.ERROR_NOT_SUPPORTED, mxg.SUCCESS
BIG = 2 ** 31 - 1


def at(i, off=0):
    """Addresses far apart, never dereferenced: validation fails before any launch."""
    return P((i + 1) * 0x1000000 + off)


A, B, C, D, E, F, G, H = (at(i) for i in range(8))
NAN = float("nan")

# name -> (arguments that would launch, [(position, bad value, status)], [(position, value) that make it a no-op])
CASES = {
    # format, stream, x, residual, weight type, weight, offset, eps, tokens, H, h, y, q, scales, stream
    "mx_rmsnorm": (
        [3, 1, A, B, 1, C, 0.0, 1e-6, 4, 64, D, E, F, G, None],
        [(0, 4, INVALID), (0, -1, INVALID), (0, 0, INVALID), (1, 2, INVALID), (2, None, INVALID), (2, at(0, 8), INVALID),
         (3, None, INVALID), (3, at(1, 8), INVALID), (4, 7, INVALID), (5, None, INVALID), (5, at(2, 4), INVALID),
         (7, -1.0, INVALID), (7, NAN, INVALID), (8, -1, INVALID), (9, 0, INVALID), (9, 60, UNSUPPORTED),
         (9, 40, UNSUPPORTED), (9, 2 ** 30, UNSUPPORTED), (8, 2 ** 30, UNSUPPORTED), (10, None, INVALID),
         (10, at(3, 4), INVALID), (11, at(4, 8), INVALID), (12, None, INVALID), (12, at(5, 8), INVALID),
         (13, None, INVALID), (13, at(6, 2), INVALID),
         # outputs on inputs and on each other; h on the weight, or half over the residual
         (11, A, INVALID), (11, B, INVALID), (11, D, INVALID), (12, C, INVALID), (12, E, INVALID), (13, E, INVALID),
         (10, C, INVALID), (10, at(1, 16), INVALID), (10, at(0, 16), INVALID)],
        [(8, 0)]),
    # stream, dy, h, weight type, weight, offset, eps, dh, tokens, H, dx, dx_bf16, dweight, workspace, stream
    "mx_rmsnorm_backward": (
        [0, A, B, 1, C, 0.0, 1e-6, D, 4, 64, E, F, G, H, None],
        [(0, 2, INVALID), (1, None, INVALID), (1, at(0, 4), INVALID), (2, None, INVALID), (2, at(1, 4), INVALID),
         (3, -1, INVALID), (4, None, INVALID), (4, at(2, 8), INVALID), (6, -1.0, INVALID), (7, at(3, 4), INVALID),
         (8, -1, INVALID), (9, -8, INVALID), (9, 12, UNSUPPORTED), (8, 2 ** 30, UNSUPPORTED), (10, at(4, 8), INVALID),
         (11, at(5, 8), INVALID), (12, at(6, 2), INVALID), (13, None, INVALID), (13, at(7, 2), INVALID),
         (10, A, INVALID), (10, B, INVALID), (10, at(3, 16), INVALID), (11, D, INVALID), (11, E, INVALID),
         (12, C, INVALID), (13, F, INVALID)],
        []),
    # act, a, b, bias, residual, c type, c, z, off, ids, groups, experts, rows, N, K, hint, stream
    "mx_grouped_matmul_bf16": (
        [4, A, B, C, D, 0, E, F, G, H, 2, 3, 8, 16, 64, 0, None],
        [(0, 5, INVALID), (0, -1, INVALID), (1, None, INVALID), (1, at(0, 8), INVALID), (2, None, INVALID),
         (2, at(1, 8), INVALID), (3, at(2, 2), INVALID), (4, at(3, 8), INVALID), (5, 2, INVALID), (6, None, INVALID),
         (6, at(4, 4), INVALID), (7, at(5, 8), INVALID), (8, None, INVALID), (8, at(6, 2), INVALID), (9, None, INVALID),
         (9, at(7, 2), INVALID), (10, -1, INVALID), (11, 0, INVALID), (12, -1, INVALID), (13, 0, INVALID),
         (14, 0, INVALID), (14, 20, UNSUPPORTED), (13, 15, UNSUPPORTED), (14, mxg.MAX_K + 8, UNSUPPORTED),
         (10, 1025, UNSUPPORTED), (12, BIG + 1, UNSUPPORTED), (13, 2 ** 30, UNSUPPORTED),
         (6, A, INVALID), (6, B, INVALID), (6, C, INVALID), (6, at(3, 16), INVALID), (7, E, INVALID), (7, A, INVALID)],
        [(10, 0), (12, 0)]),
    # act, dc, b, z, da, off, ids, groups, experts, rows, N, K, hint, stream
    "mx_grouped_matmul_bf16_backward": (
        [3, A, B, C, D, G, H, 2, 3, 8, 16, 64, 0, None],
        [(0, 0, INVALID), (0, 5, INVALID), (1, None, INVALID), (1, at(0, 8), INVALID), (2, None, INVALID),
         (2, at(1, 8), INVALID), (3, None, INVALID), (3, at(2, 8), INVALID), (4, None, INVALID), (4, at(3, 8), INVALID),
         (5, None, INVALID), (6, None, INVALID), (7, -1, INVALID), (8, 0, INVALID), (9, -1, INVALID), (10, 0, INVALID),
         (11, 0, INVALID), (10, 12, UNSUPPORTED), (11, 12, UNSUPPORTED), (10, mxg.MAX_K + 8, UNSUPPORTED),
         (11, mxg.MAX_K + 8, UNSUPPORTED), (7, 1025, UNSUPPORTED), (9, BIG + 1, UNSUPPORTED),
         (4, A, INVALID), (4, B, INVALID), (4, at(2, 16), INVALID)],
        [(7, 0), (9, 0)]),
    # dc, a, dw type, dw, dbias, accumulate, off, ids, groups, experts, rows, N, K, stream
    "mx_grouped_matmul_bf16_backward_weights": (
        [A, B, 0, C, D, 1, G, H, 2, 3, 8, 16, 64, None],
        [(0, None, INVALID), (0, at(0, 8), INVALID), (1, None, INVALID), (1, at(1, 8), INVALID), (2, 2, INVALID),
         (3, None, INVALID), (3, at(2, 8), INVALID), (4, at(3, 2), INVALID), (6, None, INVALID), (7, None, INVALID),
         (8, -1, INVALID), (9, 0, INVALID), (10, -1, INVALID), (11, -8, INVALID), (12, 0, INVALID),
         (11, 12, UNSUPPORTED), (12, 12, UNSUPPORTED), (8, 1025, UNSUPPORTED), (10, BIG + 1, UNSUPPORTED),
         (11, mxg.MAX_K + 8, UNSUPPORTED), (3, A, INVALID), (3, B, INVALID), (4, A, INVALID), (4, C, INVALID)],
        [(8, 0), (10, 0)]),
    # act, dc, z, dz, rows, N, stream
    "mx_activation_backward": (
        [4, A, B, C, 8, 16, None],
        [(0, 0, INVALID), (0, 5, INVALID), (1, None, INVALID), (1, at(0, 8), INVALID), (2, None, INVALID),
         (2, at(1, 8), INVALID), (3, None, INVALID), (3, at(2, 8), INVALID), (4, -1, INVALID), (5, 0, INVALID),
         (5, 12, UNSUPPORTED), (4, BIG + 1, UNSUPPORTED), (5, 2 ** 30, UNSUPPORTED), (3, A, INVALID),
         (3, at(1, 16), INVALID)],
        [(4, 0)]),
}


@pytest.mark.parametrize("name", list(CASES))
def test_bad_arguments(name):
    good, bad, empty = CASES[name]
    call = getattr(mxg.lib(), name)
    for pos, value, status in bad:
        args = list(good)
        args[pos] = value
        assert call(*args) == status, (pos, value)
    pointers = [a for a in good if isinstance(a, P)]
    for pos, value in empty:
        args = list(good)
        args[pos] = value
        assert call(*args) == OK, (pos, value)
        if name != "mx_grouped_matmul_bf16_backward_weights" and "rmsnorm" not in name and pos not in (10, 7):
            # without work no pointer is examined (routing without groups apart)
            assert call(*[None if any(a is p for p in pointers) and a not in (G, H) else a for a in args]) == OK


def test_no_output_and_no_routing():
    L = mxg.lib()
    assert L.mx_rmsnorm(0, 1, A, None, 1, C, 0.0, 1e-6, 4, 64, None, None, None, None, None) == INVALID
    assert L.mx_rmsnorm_backward(1, A, B, 1, C, 0.0, 1e-6, None, 4, 64, None, None, None, None, None) == INVALID
    assert L.mx_rmsnorm_backward(1, A, B, 1, C, 0.0, 1e-6, None, 0, 64, E, None, None, None, None) == OK
    assert L.mx_rmsnorm_workspace_bytes(10, 64) == 10 * 64 * 4
    assert L.mx_rmsnorm_workspace_bytes(0, 64) == 0
    for rows, width in ((-1, 64), (4, 0), (4, 12), (2 ** 30, 64)):
        assert L.mx_rmsnorm_workspace_bytes(rows, width) == -1
    # a dense product is one group of one expert
    good = list(CASES["mx_grouped_matmul_bf16"][0])
    good[8] = good[9] = None
    assert L.mx_grouped_matmul_bf16(*good) == INVALID
    good[10] = 1
    assert L.mx_grouped_matmul_bf16(*good) == INVALID
    # sizes whose bytes no memory holds overlap what lies behind them
    huge = list(CASES["mx_grouped_matmul_bf16"][0])
    huge[11], huge[13], huge[14] = BIG, 2 ** 29, mxg.MAX_K
    assert L.mx_grouped_matmul_bf16(*huge) == INVALID


def test_binding_refuses_wrong_tensors():
    """dtype, shape and device are checked before the library is called."""
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    w = torch.zeros((1, 16, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU tensor"):
        mxg.mx_rmsnorm(x, x[0], y=x)
    with pytest.raises(TypeError):
        mxg.mx_rmsnorm(x.half(), x[0], y=x)
    with pytest.raises(ValueError, match="GPU tensor"):
        mxg.mx_rmsnorm_backward(x, x, x[0], x)
    with pytest.raises(ValueError, match="GPU tensor"):
        mxg.mx_grouped_matmul_bf16(x, w, x)
    with pytest.raises(TypeError):
        mxg.mx_grouped_matmul_bf16(x.float(), w, x)
    with pytest.raises(ValueError, match="GPU tensor"):
        mxg.mx_grouped_matmul_bf16_backward(x, w, x)
    with pytest.raises(TypeError):
        mxg.mx_grouped_matmul_bf16_backward_weights(x.int(), x, w)
    with pytest.raises(ValueError, match="GPU tensor"):
        mxg.mx_activation_backward(mxg.ACT_RELU, x, x, x)


# ---- which kernel a product runs (256 compute units are assumed without a GPU, as an MI355X has)
@pytest.mark.parametrize("product,G,E,T,N,K,hint,tile", [
    (0, 1, 1, 8192, 7168, 4096, 0, (256, 256)),
    (0, 128, 128, 65536, 1536, 4096, 0, (256, 256)),
    (0, 1, 1, 2048, 2048, 2048, 0, (128, 128)),
    (0, 1, 1, 1024, 1024, 1024, 0, (32, 128)),
    (0, 1, 1, 128, 4096, 7168, 128, (64, 64)),
    (0, 1, 1, 16, 4096, 7168, 16, (32, 32)),
    (0, 1, 1, 64, 64, 7168, 64, (16, 32)),
    (1, 64, 64, 32768, 4096, 1536, 0, (256, 256)),
    (1, 1, 1, 128, 4096, 4096, 0, (64, 64)),
    (2, 64, 64, 32768, 1536, 4096, 0, (256, 256)),
    (2, 8, 8, 16384, 256, 2048, 0, (128, 128)),
    (2, 1, 1, 4096, 512, 1024, 0, (64, 64)),
    (2, 1, 1, 6000, 200, 1544, 0, (64, 32)),
])
def test_tile_choice(product, G, E, T, N, K, hint, tile):
    assert mxg.bf16_tile(product, G, E, T, N, K, hint) == tile


def test_tile_of_nothing():
    for args in [(0, 0, 1, 4, 8, 8), (0, 1, 1, 0, 8, 8), (0, 1, 1, 4, 8, 12), (1, 1, 1, 4, 12, 8), (2, 1, 1, 4, 12, 8),
                 (3, 1, 1, 4, 8, 8), (0, 1025, 1, 4, 8, 8), (0, 1, 0, 4, 8, 8)]:
        assert mxg.bf16_tile(*args) == (0, 0)
    for hint in (-5, 0, 1, 100, 1 << 62):
        assert mxg.bf16_tile(0, 4, 4, 100, 8, 8, hint) != (0, 0)


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir(HIP_INCLUDE),
                    reason="g++ or the HIP headers not installed")
def test_abi_layer_under_sanitizers(tmp_path):
    exe = str(tmp_path / "abi_dense_driver")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__", "-I", HIP_INCLUDE, "-I", os.path.join(ROOT, "include"),
           "-I", CSRC, os.path.join(CSRC, "api_dense.cpp"), os.path.join(SAN, "abi_dense_driver.cpp"), "-o", exe]
    res = subprocess.run(cmd, cwd=tmp_path, capture_output=True, text=True, timeout=240)
    assert res.returncode == 0, res.stderr
    res = subprocess.run([exe], cwd=tmp_path, capture_output=True, text=True, timeout=120)
    out = res.stdout + res.stderr
    assert res.returncode == 0 and "fails 0" in out, out[-4000:]
    for marker in ("runtime error", "ERROR: AddressSanitizer", "ERROR: LeakSanitizer"):
        assert marker not in out, out[-4000:]
