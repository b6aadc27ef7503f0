"""The attention kernels are launched before the kernel ahead of them ends, so what that one writes is written in their
lifetime: none of their loads may be of the non-coherent kind, nor one that the compiler may move past the wait."""
from __future__ import annotations

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "linear_attention_ssm_gb300", "csrc")
FILES = sorted(glob.glob(os.path.join(CSRC, "attn*.cu*")))


def code(path):
    """The file without its comments."""
    with open(path) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


@pytest.mark.parametrize("path", FILES, ids=[os.path.basename(f) for f in FILES])
def test_loads_are_coherent_and_stay_behind_the_wait(path):
    text = code(path)
    assert not re.findall(r"__ldg\b|\bld\.global\.nc\b|__ldc[agsv]\b|__ldlu\b|__restrict__", text)
    for asm in re.findall(r'asm\b(?! volatile)\s*\([^;]*', text):  # an asm that may be moved reads no memory
        assert not re.search(r'"[^"]*\bld\.', asm), asm


def test_every_kernel_launched_early_waits_first():
    kernels = {}
    for path in FILES:
        for m in re.finditer(r"__global__ void[^;{]*?(\w+)\(const __grid_constant__ (\w+) p[^)]*\) \{", code(path)):
            body = code(path)[m.end():]
            wait = body.index("await_grid();")
            touched = re.search(r"\bp\.(desc|cu|kv_lens|ml|part|out|q_out|cache\.\w+|z\.p|starts|rope\.freqs)\b", body[:wait])
            kernels[m.group(1)] = touched
    assert {"attn_kernel", "attn_join_kernel", "attn_decode_kernel", "prepare_kernel", "cache_read_kernel"} <= set(kernels)
    assert not any(kernels.values()), kernels
