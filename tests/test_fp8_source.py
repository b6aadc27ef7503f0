"""The kernels of the 8-bit product and of the expert layer are launched before the kernel ahead of them ends, so what that
one writes is written in their lifetime: none of their loads may be of the non-coherent kind, nor one that the compiler may
move past the wait, and none may come before it."""
from __future__ import annotations

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "linear_attention_ssm_gb300", "csrc")
FILES = ["fp8_quantize.cu", "fp8_matmul.cu", "moe.cu"]


def code(name):
    """The file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


@pytest.mark.parametrize("name", FILES)
def test_loads_are_coherent_and_stay_behind_the_wait(name):
    text = code(name)
    assert not re.findall(r"__ldg\b|\bld\.global\.nc\b|__ldc[agsv]\b|__ldlu\b|__restrict__", text)
    for asm in re.findall(r'asm\b(?! volatile)\s*\([^;]*', text):  # an asm that may be moved reads no memory
        assert not re.search(r'"[^"]*\bld\.', asm), asm


def test_every_kernel_waits_first():
    kernels = {}
    for name in FILES:
        text = code(name)
        for m in re.finditer(r"__global__ void[^;{]*?(\w+)\(const (?:__grid_constant__ )?\w+ p[^)]*\) \{", text):
            body = text[m.end():]
            wait = body.index("await_grid();")
            kernels[m.group(1)] = re.search(
                r"\bp\.(x|w|x_scale|w_scale|out|codes|scales|err|c\.\w+|m\.\w+\[|counters|logits|ids|weights|hidden|y)\b[\[ +]*[\[+]",
                body[:wait])
    assert {"quantize_rows_kernel", "quantize_blocks_kernel", "few_kernel", "tile_kernel", "prepare_kernel", "choose_kernel",
            "experts_kernel"} <= set(kernels)
    assert not any(kernels.values()), kernels


def test_a_wait_that_ran_out_passes_every_barrier_of_the_tile():
    """The warps of the sums count their polls apart, so one may give up where the others do not: none may leave between
    its sums and the last barrier that the others wait at."""
    text = code("fp8_matmul.cu")
    body = text[text.index("tile_kernel("):text.index("cudaError_t launch_tiles")]
    sums, last = body.index("++group;\n      asm volatile(\"cp.async.wait_group 0"), body.rindex("bar.sync")
    assert sums < last and not re.search(r"!ok|\breturn\b", body[sums:last])


def test_blocks_of_the_longest_rows():
    """k is at most 2^31 - 1: the number of its blocks is formed without a sum that leaves 31 bits."""
    text = code("fp8_matmul.cu")
    for k in (1, 127, 128, 129, 2 ** 31 - 128, 2 ** 31 - 127, 2 ** 31 - 1):
        expr = re.search(r"p\.blocks = ([^;]*);", text).group(1).replace("m.k", str(k)).replace("kBlockK", "128")
        steps = re.findall(r"\(([^()]*)\)", expr)
        assert all(abs(eval(s)) < 2 ** 31 for s in steps), expr
        assert eval(expr.replace("/", "//")) == -(-k // 128)


def test_columns_of_the_longest_rows():
    """Columns are numbered in 31 bits, up to 2^31 - 2: whether sixteen values from one on are all there is asked without a
    sum beyond that (their codes would go behind the row's end)."""
    text = code("fp8_quantize.cu")
    asked = re.search(r"if \(([^()]*)\) \{\s*\*reinterpret_cast<uint4\*>\(row \+ c\)", text).group(1)
    sides = asked.split("<=")
    for cols in (1, 15, 16, 17, 300, 2 ** 31 - 17, 2 ** 31 - 16, 2 ** 31 - 1):
        for c in range(0, cols, 16) if cols < 1000 else range(cols // 128 * 128, cols, 16):
            left, right = (eval(s.replace("p.cols", str(cols)), {"c": c}) for s in sides)
            assert abs(left) < 2 ** 31 and abs(right) < 2 ** 31 and (left <= right) == (c + 16 <= cols)


def test_a_warp_leaves_a_wait_as_a_whole():
    """What another warp writes while this one reads it is one answer for all lanes: the votes of the next wait name them all."""
    text = code("moe.cu")
    reads = [m.start() for m in re.finditer(r"\*\(volatile int\*\)&team\.failed(?! = 1)", text)]
    assert reads and all(re.search(r"__any_sync\(~0u, $", text[:at]) for at in reads)
