"""Kernels that are set up while the kernel before them on the stream still runs (no GPU).

What such a kernel reads may be written during its own lifetime, before its cudaGridDependencySynchronize(): loads through
the read-only path (__ldg, or a const __restrict__ operand, of which the compiler makes the same) are promised for data that
nobody writes while the kernel lives, and the compiler may move them up past that call."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixture_experts_layer_expert_gb300", "csrc")
SOURCES = {os.path.basename(p): re.sub(r"//[^\n]*", "", open(p).read()) for p in glob.glob(os.path.join(CSRC, "*.cu*"))}


def body(text, at):
    """Parameter list and body of the function whose name is at `at`."""
    i, depth = text.index("{", at), 0
    for j in range(i, len(text)):
        depth += {"{": 1, "}": -1}.get(text[j], 0)
        if depth == 0:
            return text[at:j + 1]
    raise AssertionError("unbalanced braces")


def early():
    """(file, kernel) of every launch with the attribute of an early set-up."""
    found = set()
    for f, text in SOURCES.items():
        names = re.findall(r"launch_after\(\s*(?:\w+::)*(\w+)", text) + re.findall(r"FS_BALANCE\(\s*(?:\w+::)*(\w+)", text)
        if "ProgrammaticStreamSerialization" in text and f != "common.cuh":
            names += re.findall(r"cudaLaunchKernelEx\(&cfg, (?:\w+::)*(\w+)", text)
        found |= {(f, n) for n in names if n not in ("KERNEL", "void")}
    return sorted(found)


def defined(f, kernel):
    return [m.start(1) for m in re.finditer(r"__global__[^;{]*?\b(%s)\(" % kernel, SOURCES[f])]


def test_the_kernels_are_found():
    names = {n for _, n in early()}
    assert names >= {"piece_kernel", "finish_kernel", "backward_kernel", "dispatch_one_chunk_kernel", "quant_rows_mx4_kernel",
                     "dispatch_copy_mx4_kernel", "mx_gemm_kernel", "mx4_pair_kernel", "gemm_kernel", "norm_kernel",
                     "scale_rows_kernel", "scale_tall_kernel", "small_kernel", "tiny_kernel"}
    assert all(len(defined(f, n)) == 1 for f, n in early())


@pytest.mark.parametrize("f,kernel", early())
def test_no_read_only_loads(f, kernel):
    text = body(SOURCES[f], defined(f, kernel)[0])
    # with the functions of this file, and of its own header, that the kernel calls
    todo, seen = [text], {kernel}
    while todo:
        part = todo.pop()
        for name in set(re.findall(r"\b([a-z]\w+)(?:<[^<>;]*>)?\(", part)) - seen:
            for src in (f, "ortho.cuh", "gemm_mx.cuh", "mx.cuh"):
                for m in re.finditer(r"__device__ __forceinline__ [^;{}()]*?\b(%s)\(" % name, SOURCES[src]):
                    seen.add(name)
                    todo.append(body(SOURCES[src], m.start(1)))
        assert "__ldg" not in part and "ld.global.nc" not in part, part[:60]
        assert not re.search(r"const [\w ]+\*\s*__restrict__", part), part[:60]
    assert "cudaGridDependencySynchronize()" in text
