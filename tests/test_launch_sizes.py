"""Launch sizes at the largest documented sizes (CPU): a launch may hold fewer than 2^32 threads, whatever
the call asks for; what does not fit is left to the kernels' own loops.  The library runs in a process of
its own under stand-ins for the HIP calls (tests/sanitize/launch_recorder.cpp), which record the
launches; the pointers are numbers, 64 TiB apart, that nothing reads."""
import ctypes
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "fp4_grouped_gemm_quantize_amd", "libmxg.so")
RECORDER = os.path.join(ROOT, "tests", "sanitize", "launch_recorder.cpp")

M30 = 1 << 30
TOP = 2 ** 31 - 1
F32, BF16 = 0, 1


def ptr(i):
    return ctypes.c_void_p((i + 1) << 46)


def i64(n):
    return ctypes.c_int64(n)


def f32(x):
    return ctypes.c_float(x)


def norm(T, H, form=0, stream=BF16):
    coded = form != 0
    return "mx_rmsnorm", [form, stream, ptr(0), None, F32, ptr(1), f32(0), f32(1e-6), i64(T), i64(H), None, ptr(2),
                          ptr(3) if coded else None, ptr(4) if coded else None, None]


CASES = {}
for t, h in ((M30 - 1, 8), (1 << 26, 512), (1 << 26, 2048), (1 << 24, 4096), (1 << 24, 8192), (1 << 22, 8200),
             (1 << 22, 32768), (1 << 22, 65536), (1, M30 - 8)):
    CASES[f"norm_{t}x{h}"] = lambda t=t, h=h: norm(t, h)
CASES["norm_codes"] = lambda: norm(M30 - 1, 32, 2)


def norm_gradient(T, H):
    some = T > 0
    return "mx_rmsnorm_backward", [BF16, ptr(0) if some else None, ptr(1) if some else None, F32,
                                   ptr(2) if some else None, f32(0), f32(1e-6), None, i64(T), i64(H),
                                   ptr(3) if some else None, None, ptr(4), ptr(5) if some else None, None]


for t, h in ((0, M30 - 8), (1, M30 - 8), (M30 - 1, 8), (1 << 20, 1 << 20)):
    CASES[f"norm_gradient_{t}x{h}"] = lambda t=t, h=h: norm_gradient(t, h)


def activation_gradient(act, T, N):
    return "mx_activation_backward", [act, ptr(0), ptr(1), ptr(1), i64(T), i64(N), None]


for a, t, n in ((4, 1 << 24, 1 << 10), (4, 1 << 20, 1 << 18), (3, 1 << 25, 1 << 10), (1, TOP, 32), (2, 1, M30 - 8)):
    CASES[f"activation_gradient_{a}_{t}x{n}"] = lambda a=a, t=t, n=n: activation_gradient(a, t, n)


# The other entry points near the ends of their ranges: a name, the entry point, its arguments but for the stream.
OFF, IDS = ptr(20), ptr(21)


def calls():
    for fmt in (0, 1, 2):
        yield f"quantize_{fmt}", "mx_grouped_quantize", [fmt, ptr(0), ptr(1), ptr(2), OFF, IDS, 8, i64(TOP), i64(32)]
        for t, n, hint in ((1 << 28, 256, 0), (1024, 1 << 22, 1)):
            yield f"matmul_{fmt}_{t}x{n}", "mx_grouped_matmul", [
                fmt, *map(ptr, range(5)), OFF, IDS, 1024, 8, i64(t), i64(n), i64(1024), i64(hint)]
    yield "silu_quantize", "mx_silu_quantize", [ptr(0), ptr(1), ptr(2), OFF, 8, i64(TOP), i64(512)]
    yield "prepare_weights", "mx_prepare_weights_fp8", [ptr(0), 1024, i64(1 << 20), i64(1024), ptr(1)]
    yield "combine", "mx_moe_combine", [ptr(0), i64(TOP), i64(8), ptr(1), ptr(2), i64(TOP), 1, ptr(3)]
    yield "combine_backward", "mx_moe_combine_backward", [ptr(0), ptr(1), i64(TOP), i64(8), ptr(2), ptr(3), i64(TOP), 1,
                                                          ptr(4), ptr(5)]
    yield "topk", "mx_moe_topk", [0, 0, ptr(0), None, i64(TOP), 8, 1, 1, f32(1), ptr(1), ptr(2)]
    yield "topk_backward", "mx_moe_topk_backward", [0, 0, ptr(0), ptr(1), ptr(2), i64(TOP), 8, 1, 1, f32(1), ptr(3)]
    yield "sort", "mx_moe_sort", [ptr(0), i64(TOP), 1, 256, ptr(1), ptr(2), ptr(3)]
    yield "permute", "mx_moe_permute", [ptr(0), i64(TOP), i64(1024), ptr(1), 1, ptr(2), i64(TOP)]
    yield "permute_backward", "mx_moe_permute_backward", [ptr(0), i64(TOP), i64(1024), ptr(1), i64(TOP), 1, ptr(2)]
    yield "quantize_block128", "mx_grouped_quantize_block128", [ptr(0), ptr(1), ptr(2), OFF, 8, i64(TOP), i64(1024)]
    yield "weights_block128", "mx_quantize_weights_block128", [ptr(0), 1 << 20, i64(1024), i64(1024), ptr(1), ptr(2),
                                                               ptr(3), ptr(4)]
    yield "silu_quantize_block128", "mx_silu_quantize_block128", [ptr(0), ptr(1), ptr(2), OFF, 8, i64(TOP), i64(512)]
    yield "silu_backward_block128", "mx_silu_backward_block128", [ptr(0), ptr(1), ptr(2), None, None, OFF, 8, i64(TOP),
                                                                  i64(512)]
    for t, n, hint in ((1, 1 << 24, 0), (1024, 1 << 17, 0), (1024, 1 << 24, 1), (1 << 26, 1 << 20, 0)):
        yield f"matmul_block128_{t}x{n}", "mx_grouped_matmul_block128", [
            *map(ptr, range(5)), OFF, IDS, 1024, 8, i64(t), i64(n), i64(128), i64(hint)]
    for t, n, k, e in ((TOP, 256, 8, 1), (1, M30 - 1, 8, 1), (1 << 26, 1 << 10, 512, 1024), (64, 1 << 26, 64, 64),
                       (1, 1 << 28, 7168, 1), (33, 1 << 22, 4096, 1)):
        routing = [OFF, IDS] if e > 1 else [None, None]
        yield f"matmul_bf16_{t}x{n}", "mx_grouped_matmul_bf16", [
            0, ptr(0), ptr(1), None, None, BF16, ptr(2), None, *routing, e, e, i64(t), i64(n), i64(k), i64(0)]
    for t, n, k, e in ((TOP, 256, 8, 1), (1, 8, 1 << 22, 1), (1 << 26, 1 << 10, 512, 1024), (33, 4096, 1 << 22, 1)):
        routing = [OFF, IDS] if e > 1 else [None, None]
        yield f"matmul_bf16_backward_{t}x{k}", "mx_grouped_matmul_bf16_backward", [
            0, ptr(0), ptr(1), None, ptr(2), *routing, e, e, i64(t), i64(n), i64(k), i64(0)]
    for t, n, k, e in ((TOP, 8, 8, 1), (1, 1 << 20, 1 << 20, 1), (1 << 10, 1 << 10, 64, 1 << 22), (16, 1 << 22, 64, 64),
                       (4, 8, 8, 1 << 30)):
        yield f"matmul_bf16_backward_weights_{n}x{k}x{e}", "mx_grouped_matmul_bf16_backward_weights", [
            ptr(0), ptr(1), BF16, ptr(2), None, 0, OFF if e > 1 else None, IDS if e > 1 else None, min(e, 1024), e,
            i64(t), i64(n), i64(k)]


for name_, fn_, args_ in calls():
    CASES[name_] = lambda fn_=fn_, args_=args_: (fn_, [*args_, None])


def record(name):
    """In the process of its own: (status, launches, threads of the largest)."""
    recorder = ctypes.CDLL(os.environ["MXG_TEST_RECORDER"], mode=ctypes.RTLD_GLOBAL)
    recorder.recorder_reset()
    recorder.recorder_launches.restype = recorder.recorder_most_threads.restype = ctypes.c_uint64
    fn, args = CASES[name]()
    status = getattr(ctypes.CDLL(LIB), fn)(*args)
    return status, recorder.recorder_launches(), recorder.recorder_most_threads()


@pytest.fixture(scope="module")
def results(tmp_path_factory):
    gxx = shutil.which("g++")
    assert gxx and os.path.exists(LIB), "g++ and the built library are required"
    so = str(tmp_path_factory.mktemp("recorder") / "recorder.so")
    subprocess.run([gxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include",
                    RECORDER, "-o", so], check=True, timeout=120)
    res = subprocess.run([sys.executable, os.path.abspath(__file__)], capture_output=True, text=True, timeout=120,
                         env={**os.environ, "MXG_TEST_RECORDER": so})
    assert res.returncode == 0, res.stderr[-2000:]
    return {name: (int(s), int(n), int(t)) for name, s, n, t in map(str.split, res.stdout.splitlines())}


@pytest.mark.parametrize("name", list(CASES))
def test_fewer_than_2_32_threads(results, name):
    status, launches, threads = results[name]
    assert status == 0 and launches >= 1
    assert threads < 2 ** 32, threads


if __name__ == "__main__":
    for case in CASES:
        print(case, *record(case))
