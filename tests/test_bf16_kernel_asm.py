"""Checks on the generated gfx950 assembly of the BF16 products and their gradients (CPU; hipcc
cross-compiles).  Their loads from memory straight into LDS are inline assembly, in front of which the
compiler puts no wait states of its own.  What the hardware asks for, on every path that leads to a load:

* five wait states between a vector instruction's write of a scalar register (a lane read, a spilled
  scalar read back from its lane, a compare) and a load that takes its descriptor or offset from it;
* one between a scalar instruction's write of M0 and a load into LDS, whose address it holds.

Each instruction is one wait state at least, s_nop N is N + 1."""
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "fp4_grouped_gemm_quantize_amd", "csrc")
HIPCC = "/opt/rocm/bin/hipcc"

LOAD = re.compile(r"^buffer_load_dword(?:x3|x4)?\s+v\d+,\s*s\[(\d+):(\d+)\],\s*(\S+)\s.*\blds\b")
BRANCH = re.compile(r"^s_c?branch\S*\s+(\S+)")
NEEDED, NEEDED_M0 = 5, 1


class Kernel:
    """The instructions of a kernel, and from where each is reached."""

    def __init__(self, name, lines):
        self.name, self.code = name, []
        labels, pending = {}, []
        for line in lines:
            s = line.split(";")[0].strip()
            if s.endswith(":"):
                pending.append(s[:-1])
            elif s and not s.startswith("."):
                for label in pending:
                    labels[label] = len(self.code)
                pending = []
                self.code.append(s)
        self.before = [[] for _ in self.code]
        for i, s in enumerate(self.code):
            m = BRANCH.match(s)
            if m and labels.get(m.group(1)) is not None:
                self.before[labels[m.group(1)]].append(i)
            if i + 1 < len(self.code) and not s.startswith(("s_branch", "s_endpgm", "s_setpc")):
                self.before[i + 1].append(i)

    def too_close(self, i, needed, writes):
        """An instruction that `writes` says is one, fewer than `needed` wait states before the i-th; or None."""
        seen, todo = {}, [(j, 0) for j in self.before[i]]
        while todo:
            j, states = todo.pop()  # wait states between j and i
            if states >= needed or seen.get(j, needed) <= states:
                continue
            seen[j] = states
            s = self.code[j]
            if writes(s):
                return f"{s}  ... {states} wait states ...  {self.code[i]}"
            m = re.match(r"s_nop\s+(\w+)", s)
            here = states + (int(m.group(1), 0) + 1 if m else 1)
            todo += [(k, here) for k in self.before[j]]
        return None


def scalars(operand):
    m = re.fullmatch(r"s\[(\d+):(\d+)\]", operand)
    if m:
        return set(range(int(m.group(1)), int(m.group(2)) + 1))
    m = re.fullmatch(r"s(\d+)", operand)
    return {int(m.group(1))} if m else set()


def written_by_vector(s):
    """The scalar registers that a vector instruction writes."""
    if not s.startswith("v_"):
        return set()
    op, _, rest = s.partition(" ")
    operands = [o.strip() for o in re.split(r",(?![^\[]*\])", rest)]
    dst = operands[:1]
    if re.match(r"v_(add|sub|subrev|addc|subb|subbrev)_co_|v_div_scale|v_mad_(u|i)64", op):
        dst = operands[:2]  # and a carry
    return set().union(*(scalars(o) for o in dst)) if dst else set()


def vector_write_hazards(k):
    bad = []
    for i, s in enumerate(k.code):
        m = LOAD.match(s)
        if m:
            reads = set(range(int(m.group(1)), int(m.group(2)) + 1)) | scalars(m.group(3))
            found = k.too_close(i, NEEDED, lambda w: bool(written_by_vector(w) & reads))
            bad += [found] if found else []
    return bad


def m0_hazards(k):
    found = [k.too_close(i, NEEDED_M0, lambda w: bool(re.match(r"s_\S+\s+m0\b", w)))
             for i, s in enumerate(k.code) if LOAD.match(s)]
    return [f for f in found if f]


def loads(k):
    return sum(1 for s in k.code if LOAD.match(s))


SOURCES = ("gemm_bf16.hip", "gemm_bf16_weights.hip")
EXPECTED = {"gemm_bf16.hip": 16, "gemm_bf16_weights.hip": 8}  # kernels with such loads


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    if not os.path.exists(HIPCC):
        pytest.fail("hipcc is required to compile the kernels")
    tmp = tmp_path_factory.mktemp("asm")
    runs = {}
    for src in SOURCES:
        out = str(tmp / (src + ".s"))
        runs[src] = out, subprocess.Popen(
            [HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "-Xclang", "-target-feature", "-Xclang",
             "-packed-fp32-ops", "-Wno-unused-command-line-argument", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
             "--cuda-device-only", "-S", os.path.join(CSRC, src), "-o", out],
            stdout=subprocess.DEVNULL, stderr=subprocess.PIPE, text=True)
    found = {}
    for src, (out, p) in runs.items():
        err = p.communicate(timeout=600)[1]
        assert p.returncode == 0, err[-4000:]
        text = open(out).read()
        bodies = re.findall(r"^(_Z\w+):\s*;?.*?$(.*?)^\.Lfunc_end", text, re.M | re.S)
        found[src] = [k for k in (Kernel(n, b.splitlines()) for n, b in bodies) if loads(k)]
    return found


@pytest.mark.parametrize("src", SOURCES)
def test_kernels_with_direct_loads(kernels, src):
    assert len(kernels[src]) == EXPECTED[src], [k.name for k in kernels[src]]


@pytest.mark.parametrize("src", SOURCES)
def test_wait_states_behind_vector_writes_of_a_load_s_scalars(kernels, src):
    bad = {k.name: h for k in kernels[src] if (h := vector_write_hazards(k))}
    assert not bad, {n: (len(h), h[0]) for n, h in bad.items()}


@pytest.mark.parametrize("src", SOURCES)
def test_wait_states_behind_writes_of_m0(kernels, src):
    bad = {k.name: h for k in kernels[src] if (h := m0_hazards(k))}
    assert not bad, {n: (len(h), h[0]) for n, h in bad.items()}


def test_the_scan_itself():
    """Planted: a lane read three states before a load, on a loop's way back to it, and one behind enough of them."""
    near = ["v_readfirstlane_b32 s46, v4", "s_mov_b32 m0, s5", "s_nop 0", "buffer_load_dwordx4 v1, s[44:47], 0 offen lds"]
    assert vector_write_hazards(Kernel("near", near)) and not m0_hazards(Kernel("near", near))
    far = ["v_readfirstlane_b32 s46, v4", "s_mov_b32 m0, s5", "s_nop 3", near[-1]]
    assert not vector_write_hazards(Kernel("far", far))
    assert vector_write_hazards(Kernel("offset", ["v_readlane_b32 s3, v9, 16", "s_nop 2",
                                                  "buffer_load_dwordx4 v1, s[44:47], s3 offen lds"]))
    assert m0_hazards(Kernel("m0", ["s_mov_b32 m0, s5", near[-1]]))
    loop = [".L1:", "s_nop 1", near[-1], "s_nop 7", "v_cmp_eq_u32_e64 s[46:47], v1, v2", "s_cbranch_scc1 .L1", "s_endpgm"]
    assert vector_write_hazards(Kernel("loop", loop))
    assert not vector_write_hazards(Kernel("other", ["v_readlane_b32 s48, v9, 16", near[-1]]))
