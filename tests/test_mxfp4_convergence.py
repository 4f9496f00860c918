"""Instructions that a whole warp has to issue together (PTX `.aligned`) stand
behind a point at which the warp has met again, in the MXFP4 kernels (CPU: by the
source, as leaving such a point out need not show on a GPU, and must not be tried).

Lanes of a warp may be apart behind a branch on the lane, on an output's place or on
a loop that some of them leave earlier.  So between such an instruction and the
nearest of __syncwarp, __syncthreads, a vote or another of these instructions before
it there may be no branch at all but those on values that are one per warp, which are
named here."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "w4a16_decode_paged_gb300", "csrc")

# conditions whose value is the same in every lane of a warp
UNIFORM = [r"clog > 0", r"csize > 1", r"csize == 1", r"round \+ 1 < rounds", r"warp == \d", r"!ok",
           r"p\.silu && !parts"]
UNROLLED = [r"for \(int h = 0; h < 64; h \+= 32\)", r"for \(int c = 0; c < 32; c \+= 8\)"]  # (one instruction a turn)
# (a vote behind a condition of its own does not count)
MEETS = r"__syncwarp\(\)|__syncthreads\(\)|(?<!\) ok = )__all_sync\([^;]*;|ALIGNED<[^>]*>"
BRANCH = r"\b(?:if|for|while)\s*\(|\?|&&|\|\|"


def _code(name):
    text = open(os.path.join(CSRC, name)).read()
    text = re.sub(r"//[^\n]*", "", text)
    # an asm statement is its name and whether it is aligned
    def asm(m):
        a = re.search(r"(?:barrier\.cluster|tcgen05)[\w.:]*aligned", m.group(0))
        return f"ALIGNED<{a.group(0)}>;" if a else "ASM;"
    return re.sub(r"asm volatile\(.*?\);", asm, text, flags=re.S)


def _inlined(code, helpers):
    for h in helpers:
        code = re.sub(rf"(?<!void ){h}\([^;{{]*\);", f"ALIGNED<{h}>;", code)
    return code


def _unmet(code):
    """The aligned instructions of a kernel that a branch may have left a warp apart at."""
    found = []
    for m in re.finditer(r"ALIGNED<([^>]*)>", code):
        before = code[:m.start()]
        last = [x.end() for x in re.finditer(MEETS, before)]
        gap = before[last[-1]:] if last else before
        for u in UNIFORM:
            gap = re.sub(rf"(?:else\s+)?if \({u}\)", "", gap)
        for u in UNROLLED:
            gap = re.sub(u, "", gap)
        if re.search(BRANCH, gap):
            found.append((m.group(1), gap.strip()[-120:]))
    return found


def _kernel(name, kernel, helpers=()):
    code = _inlined(_code(name), helpers)
    at = re.search(rf"\b{kernel}\(const __grid_constant__", code)
    start = code.index("{", at.end())
    depth = 0
    for i in range(start, len(code)):
        depth += {"{": 1, "}": -1}.get(code[i], 0)
        if depth == 0:
            return code[start:i]
    raise AssertionError("no end")


def test_the_check_itself():
    bad = "{ for (;;) { if (!live) break; } if (csize > 1) ALIGNED<x>; }"
    assert _unmet(bad)
    assert not _unmet(bad.replace("if (csize", "__syncwarp(); if (csize"))


def test_stream_kernel():
    code = _kernel("mxfp4_matvec.cu", "w4pg_mxfp4_matvec", ("cluster_arrive", "cluster_wait", "cluster_sync"))
    assert len(re.findall("ALIGNED", code)) == 4
    assert not _unmet(code), _unmet(code)


@pytest.mark.parametrize("name,helpers,n", [("mxfp4_a16", ("mx_tmem_ld8",), 8), ("mxfp4_a4", (), 5)])
def test_tensor_core_kernels(name, helpers, n):
    """Tensor memory allocated, written, read, waited for and freed."""
    code = _kernel(name + ".cu", "w4pg_" + name, helpers)
    assert len(re.findall("ALIGNED", code)) == n
    assert not _unmet(code), _unmet(code)
