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
