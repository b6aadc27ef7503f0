"""What an expert layer keeps of its values: h = silu(gate) * up between the two products."""
from __future__ import annotations

import math

import pytest
import torch

from tests.fp8_reference import DEV, HALF_BF16, TINY, ULP, assert_within, experts
from tests.gpu_common import lib

pytestmark = pytest.mark.gpu


def weights_of(matrix, e4m3):
    """(matrix, scales of one) in a type that holds its values."""
    m = matrix.to(torch.float8_e4m3fn if e4m3 else torch.bfloat16)
    assert torch.equal(m.float(), matrix)
    return m, torch.ones(*matrix.shape[:-2], 1, 1, device=DEV) if e4m3 else None


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("e4m3", [True, False], ids=["e4m3", "bf16"])
@pytest.mark.parametrize("T", [1, 3, 64])
def test_h_keeps_what_32_bits_hold(T, e4m3, shared):
    """An h of 23 bits, exact in fp32, less two others that come near it: what is left is its last bits.

    Gate values are 64 at least, whose silu is the value itself in fp32, and every gate, up and h is exact there.  The first
    h may be held in two parts of 11 bits (off by 2^-22 of it), and three values are added up in parts: 3 additions in all,
    one more for the sum over experts, each off by at most 2^-23 of the sum of magnitudes."""
    g = lib()
    H, I = 32, 16
    gen = torch.Generator(device=DEV).manual_seed(21)
    x = torch.zeros(T, H, dtype=torch.float64, device=DEV)
    a, b, c = (1 + torch.rand(3, T, generator=gen, device=DEV)).bfloat16().double()
    h = (64 * a + c / 2) * b
    near = (h / 64).bfloat16().double()
    rest = ((h - 64 * near) / 64).bfloat16().double()
    for j, v in enumerate((64 * a, b, torch.full_like(a, 64), near, rest, 64 * c)):
        x[:, j] = v
    gate_up = torch.zeros(2, I, H, device=DEV)
    gate_up[0, 0, 0], gate_up[0, 0, 5], gate_up[0, 1:3, 2] = 1, 2.0 ** -7, 1
    gate_up[1, 0, 1], gate_up[1, 1, 3], gate_up[1, 2, 4] = 1, 1, 1
    down = torch.zeros(H, I, device=DEV)
    down[:, 0], down[:, 1:3] = 1, -1
    (gu, gus), (dn, dns) = weights_of(gate_up, e4m3), weights_of(down, e4m3)
    none = torch.zeros_like(gu)[None], torch.zeros_like(dn)[None]  # an expert that gives nothing
    one = (lambda s: None if s is None else s[None])
    if shared:
        ex = g.Experts(*none, one(gus), one(dns), shared_gate_up=gu, shared_down=dn, shared_gate_up_scale=gus,
                       shared_down_scale=dns)
    else:
        ex = g.Experts(gu[None], dn[None], one(gus), one(dns))
    ids, w = torch.zeros(T, 1, dtype=torch.int32, device=DEV), torch.ones(T, 1, device=DEV)
    out = g.gdn_moe_step_routed(x.bfloat16(), ex, ids, w)
    g.gdn_check_device_errors()
    assert torch.equal(x.bfloat16().double(), x) and torch.equal(h.float().double(), h)
    want = h - 64 * near - 64 * rest
    size = h + 64 * near + 64 * rest.abs()
    tol = size * (2.0 ** -22 + 4 * ULP) + TINY
    assert_within(out, want[:, None].expand(T, H), (tol + HALF_BF16 * (want.abs() + tol))[:, None].expand(T, H), "h")


@pytest.mark.parametrize("largest", [64.0, 65.0, 127.5, -64.0])
def test_small_values_beside_a_large_one(largest):
    """e4m3 weights that single out one small value of a token: exact down to 2^-32 of the token's largest value, off by at
    most 2^-40 of it below.  The gate is the largest value's magnitude, whose silu is the value itself in fp32, and the
    token's one h is a power of two times 16 bits; with 64 as the largest value the row's 8 bits are the small value's own."""
    g = lib()
    H, I, T = 32, 16, 64
    j = torch.arange(T, device=DEV)
    small = (1 + (37 * j % 128) / 128.0) * 2.0 ** -(8 + j * 0.5).floor() * 32
    small[40] = abs(largest) * 2.0 ** -32 * (1 + 2.0 ** -7)
    x = torch.zeros(T, H, device=DEV)
    x[:, 0], x[:, 1] = largest, small
    x = x.bfloat16()
    gate_up = torch.zeros(2, I, H, device=DEV)
    gate_up[0, 0, 0], gate_up[1, 0, 1] = (1 if largest > 0 else -1), 1
    down = torch.zeros(H, I, device=DEV)
    down[:, 0] = 1
    (gu, gus), (dn, dns) = weights_of(gate_up, True), weights_of(down, True)
    ex = g.Experts(gu[None], dn[None], gus[None], dns[None])
    ids, w = torch.zeros(T, 1, dtype=torch.int32, device=DEV), torch.ones(T, 1, device=DEV)
    out = g.gdn_moe_step_routed(x, ex, ids, w)
    g.gdn_check_device_errors()
    top, v = x[:, 0].double().abs(), x[:, 1].double()
    want = top * v
    exact = v >= top * 2.0 ** -32
    assert bool(exact[40]) and 5 < int(exact.sum()) < T - 5
    room = top * torch.where(exact, 0.0, top * 2.0 ** -40)
    room = room + want.abs() * (2.0 ** -23 + 4 * ULP)  # h in two parts, sums as above
    if abs(largest) == 64:
        assert torch.equal(out[exact], want[exact].bfloat16()[:, None].expand(-1, H))
    assert_within(out, want[:, None].expand(T, H), (room + HALF_BF16 * (want.abs() + room))[:, None].expand(T, H), "small values")


@pytest.mark.parametrize("shared", [0, 32])
@pytest.mark.parametrize("e4m3", [True, False], ids=["e4m3", "bf16"])
def test_weights_that_are_not_finite_reach_the_tokens_that_pass_them(e4m3, shared):
    """One NaN (or infinity) among an expert's weights or scales: the rows of its tokens are not finite where the definition's
    are not, every other row is as it was."""
    g = lib()
    gen = torch.Generator(device=DEV).manual_seed(22)
    T, E, H, I = 40, 6, 272, 144
    clean = experts(g, gen, E, H, I, shared, e4m3)
    x = (torch.randn(T, H, generator=gen, device=DEV)).bfloat16()
    ids = torch.randint(0, E, (T, 2), generator=gen, device=DEV).int()
    ids[:, 1] = (ids[:, 0] + 1 + ids[:, 1] % (E - 1)) % E
    w = torch.rand(T, 2, generator=gen, device=DEV) + 0.1
    want = g.gdn_moe_step_routed(x, clean, ids, w)
    parts = ["gate_up", "down"] + (["gate_up_scale", "down_scale"] if e4m3 else [])
    for name in parts:
        for value in [math.nan] + ([] if e4m3 and "scale" not in name else [math.inf]):
            t = getattr(clean, name)
            kept = t.clone()
            row = t.view(E, -1).shape[1] // 2 + 3
            t.view(E, -1)[2, row if "scale" not in name else 1] = value
            out = g.gdn_moe_step_routed(x, clean, ids, w)
            g.gdn_check_device_errors()
            hit = (ids == 2).any(1)
            assert bool(hit.any()) and torch.equal(out[~hit], want[~hit]), name
            bad = ~out[hit].isfinite()
            assert bool(bad.any(1).all()), (name, value)
            if name.startswith("gate_up"):  # an h that is not finite reaches every column
                assert bool(bad.all()), (name, value)
            t.copy_(kept)
    assert torch.equal(g.gdn_moe_step_routed(x, clean, ids, w), want)
