"""Quantising at its edges: zeros' signs, the borders of a launch."""
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


def reference(x, block_rows):
    """tests.fp8_reference.quantise of 16 columns or fewer, all blocks at once."""
    rows, cols = x.shape
    f = torch.zeros(-(-rows // block_rows) * block_rows, cols, device=x.device)
    f[:rows] = x.float()
    f = f.view(-1, block_rows, cols)
    top = f.abs().amax((1, 2))
    s = torch.maximum(top / torch.full_like(top, 448), torch.full_like(top, 2.0 ** -126))
    c = (f / s[:, None, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return c.view(torch.uint8).view(-1, cols)[:rows], s[:, None]


@pytest.mark.parametrize("stride", [16, 17])
def test_more_row_blocks_than_a_launch_holds(stride):
    """65,535 rows of blocks are one launch: codes and scales on both sides of its border, rows of any alignment, nothing
    between the rows' ends and their strides."""
    g = lib()
    rows, cols = 65535 * 128 + 130, 16
    gen = torch.Generator(device=DEV).manual_seed(32)
    x = torch.randn(rows, stride, generator=gen, device=DEV, dtype=torch.bfloat16)
    x *= torch.exp(torch.randn(rows, 1, generator=gen, device=DEV)).bfloat16()
    x = x[:, :cols]
    room = torch.full((rows, 32), 0xAB, dtype=torch.uint8, device=DEV)
    codes, scales = g.gdn_fp8_quantize(x, 128, codes=room.view(torch.float8_e4m3fn)[:, :cols])
    want, ws = reference(x, 128)
    assert torch.equal(scales, ws) and torch.equal(room[:, :cols], want) and bool((room[:, cols:] == 0xAB).all())
    g.gdn_check_device_errors()
