"""Quantising at its edges: zeros' signs, the borders of a launch, rows as long as they may be."""
from __future__ import annotations

import pytest
import torch

from tests.fp8_reference import DEV, quantise
from tests.gpu_common import lib

pytestmark = pytest.mark.gpu


def bits(codes):
    return codes.contiguous().view(torch.uint8)


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("scale", [1.0, 1e-20, 2.0 ** -126, 5e37])
def test_zeros_keep_their_signs(block_rows, scale):
    """-0 beside values of every size in one block: the codes are those of x / s to the bit, 0x80 for -0 and for what is
    too small and negative."""
    g = lib()
    gen = torch.Generator(device=DEV).manual_seed(31)
    x = torch.randn(130, 300, generator=gen, device=DEV) * scale
    x[:, 1::3] = -0.0
    x[:, 2::7] = 0.0
    x[:, 5::11] *= 2.0 ** -12
    x = x.bfloat16()
    codes, scales = g.gdn_fp8_quantize(x, block_rows)
    want, ws = quantise(x, block_rows)
    assert torch.equal(scales, ws) and torch.equal(bits(codes), bits(want))
    assert bool((bits(codes)[:, 1] == 0x80).all())
