"""The expert layer for a few tokens against its definition in 64 bits."""
from __future__ import annotations

import math

import pytest
import torch

from tests.fp8_reference import DEV, assert_choice, assert_layer, experts
from tests.gpu_common import Guarded, lib

pytestmark = pytest.mark.gpu


def gen_of(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def rows(gen, T, H, scale=1.0):
    return (torch.randn(T, H, generator=gen, device=DEV) * scale).bfloat16()


def run(g, x, ex, top_k, scoring="softmax", renormalise=True, scale=1.0):
    """out, ids, weights of a call into guarded memory, with a workspace full of ones' bits."""
    T, H = x.shape
    out = Guarded((T, H), torch.bfloat16)
    ids, w = Guarded((T, top_k), torch.int32), Guarded((T, top_k), torch.float32)
    ws = Guarded((g.gdn_moe_workspace_size(ex, T, top_k) + 256,), torch.uint8)
    at = -ws.t.data_ptr() % 256
    ws.t.fill_(255)
    work = ws.t[at:at + g.gdn_moe_workspace_size(ex, T, top_k)]
    g.gdn_moe_step(x, ex, top_k, scoring, renormalise, scale, out=out.t, ids=ids.t, weights=w.t, workspace=work)
    g.gdn_check_device_errors()
    for b, n in ((out, "out"), (ids, "ids"), (w, "weights"), (ws, "workspace")):
        b.check(n)
    assert bool((ws.t[:at] == 255).all()) and bool((ws.t[at + work.numel():] == 255).all())
    return out.t, ids.t, w.t


CASES = [  # T, E, top_k, H, I, Is
    (1, 1, 1, 16, 16, 0), (1, 8, 2, 128, 128, 0), (1, 64, 8, 2048, 256, 0), (2, 7, 7, 144, 48, 16), (5, 40, 6, 272, 208, 160),
    (8, 128, 10, 512, 128, 128), (9, 3, 2, 256, 400, 0), (16, 16, 1, 1040, 96, 32), (17, 32, 4, 384, 352, 0),
    (33, 60, 4, 256, 176, 704), (64, 288, 8, 256, 64, 64), (64, 8, 8, 512, 256, 0), (64, 5, 2, 4096, 32, 0), (3, 1024, 16, 64, 32, 0),
    # more blocks of k than scales are kept at hand; shared experts of every number of tokens; units of one stage by the thousand
    (2, 3, 2, 4240, 48, 0), (20, 3, 2, 144, 4368, 0), (4, 6, 3, 4112, 4112, 0), (6, 20, 3, 400, 80, 272), (17, 5, 2, 96, 112, 1040),
    (64, 1000, 16, 128, 16, 16), (64, 40, 3, 2048, 96, 0),
    # the widest
    (3, 3, 2, 16384, 2064, 0), (2, 2, 2, 1040, 16384, 16)]


@pytest.mark.parametrize("e4m3", [True, False], ids=["e4m3", "bf16"])
@pytest.mark.parametrize("T,E,k,H,I,Is", CASES)
def test_layer(T, E, k, H, I, Is, e4m3):
    g = lib()
    gen = gen_of(T * 31 + E + H)
    scoring, bias = ("sigmoid", True) if (T + E) % 2 else ("softmax", False)
    ex = experts(g, gen, E, H, I, Is, e4m3, bias, gate=T % 2 == 1)
    x = rows(gen, T, H)
    out, ids, w = run(g, x, ex, k, scoring, True, 1.5)
    assert_choice(ids, w, x, ex, k, scoring, True, 1.5)
    assert_layer(out, x, ex, ids, w)
    again = g.gdn_moe_step(x, ex, k, scoring, True, 1.5)
    assert torch.equal(out, again), "two calls, the same bits"
    given = g.gdn_moe_step_routed(x, ex, ids, w)
    assert torch.equal(out, given), "the routing given"


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [False, True])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("spread", [0.5, 20.0, 300.0])
def test_routing(scoring, renormalise, bias, spread):
    """Every way of scoring, with logits from close together to where scores underflow."""
    g = lib()
    gen = gen_of(5)
    ex = experts(g, gen, 50, 256, 16, 0, True, bias, spread_logits=spread)
    x = rows(gen, 20, 256)
    out, ids, w = run(g, x, ex, 5, scoring, renormalise, 0.75)
    assert bool(w.isfinite().all())
    assert_choice(ids, w, x, ex, 5, scoring, renormalise, 0.75)
    assert_layer(out, x, ex, ids, w)


def test_ties_go_to_the_lowest_index():
    g = lib()
    gen = gen_of(6)
    ex = experts(g, gen, 70, 128, 16, 0, True)
    ex.router.copy_(ex.router[:7].repeat(10, 1))  # experts 7 apart are alike
    x = rows(gen, 9, 128)
    _, ids, w = run(g, x, ex, 12)
    s = x.double() @ ex.router.double().T
    want = s.round(decimals=9).sort(dim=1, descending=True, stable=True).indices[:, :12]
    assert torch.equal(ids.long(), want)
    zero = torch.zeros_like(x)
    out, ids, w = run(g, zero, ex, 4)
    assert torch.equal(ids, torch.arange(4, dtype=torch.int32, device=DEV).expand(9, 4)) and bool((out == 0).all())
    assert_choice(ids, w, zero, ex, 4, "softmax", True, 1.0)


@pytest.mark.parametrize("e4m3", [True, False], ids=["e4m3", "bf16"])
@pytest.mark.parametrize("T", [1, 7, 8, 16, 24, 40, 64])
def test_all_tokens_to_one_expert(T, e4m3):
    g = lib()
    gen = gen_of(7)
    ex = experts(g, gen, 9, 272, 144, 48, e4m3)
    x = rows(gen, T, 272)
    ids = torch.full((T, 2), 4, dtype=torch.int32, device=DEV)
    ids[:, 1] = 8
    w = torch.rand(T, 2, generator=gen, device=DEV)
    out = g.gdn_moe_step_routed(x, ex, ids, w)
    g.gdn_check_device_errors()
    assert_layer(out, x, ex, ids, w)


@pytest.mark.parametrize("shared", [0, 48])
def test_given_routing_with_gaps_and_repeats(shared):
    """No expert at all, some, the same one several times, weights of zero and below."""
    g = lib()
    gen = gen_of(8)
    ex = experts(g, gen, 6, 144, 80, shared)
    x = rows(gen, 8, 144)
    ids = torch.tensor([[-1, -1, -1, -1], [0, -1, 5, -1], [2, 2, 2, 2], [1, 3, 1, 3], [-7, 4, -1, 4], [5, 4, 3, 2],
                        [0, 0, 1, 1], [-1, -1, -1, 0]], dtype=torch.int32, device=DEV)
    w = torch.randn(8, 4, generator=gen, device=DEV)
    w[5, 1] = 0
    out = g.gdn_moe_step_routed(x, ex, ids, w)
    g.gdn_check_device_errors()
    assert_layer(out, x, ex, ids, w)
    if not shared:
        assert bool((out[0] == 0).all())
    none = torch.full((8, 4), -1, dtype=torch.int32, device=DEV)
    out = g.gdn_moe_step_routed(x, ex, none, w, out=torch.full_like(x, 3.0))
    assert_layer(out, x, ex, none, w)
    ids[3, 2] = 6  # there are six
    out = g.gdn_moe_step_routed(x, ex, ids, w)
    with pytest.raises(g.GdnError) as e:
        g.gdn_check_device_errors()
    assert e.value.name == "GDN_ERR_DEVICE_ARGUMENT"
    assert_layer(out, x, ex, ids, w)
    g.gdn_check_device_errors()


@pytest.mark.parametrize("e4m3", [True, False], ids=["e4m3", "bf16"])
def test_tokens_that_are_not_finite_stay_alone(e4m3):
    g = lib()
    gen = gen_of(9)
    ex = experts(g, gen, 10, 256, 64, 32, e4m3, bias=True)
    x = rows(gen, 12, 256)
    clean, ids, w = run(g, x, ex, 3, "sigmoid")
    x[2, 5], x[7, 200], x[9, 0] = math.nan, math.inf, -math.inf
    out, bad_ids, _ = run(g, x, ex, 3, "sigmoid")
    assert bool(((bad_ids >= 0) & (bad_ids < 10)).all())
    bad = torch.tensor([2, 7, 9], device=DEV)
    keep = torch.tensor([i for i in range(12) if i not in (2, 7, 9)], device=DEV)
    assert not bool(out[bad].isfinite().all(1).any())
    assert torch.equal(bad_ids[keep], ids[keep])
    assert_layer(out[keep], x[keep], ex, ids[keep], w[keep])


@pytest.mark.parametrize("e4m3", [True, False], ids=["e4m3", "bf16"])
def test_large_and_small_activations(e4m3):
    """Hidden values far beyond binary16's range, and far below one."""
    g = lib()
    gen = gen_of(10)
    ex = experts(g, gen, 4, 256, 128, 0, e4m3)
    ids = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device=DEV).repeat(3, 1)
    w = torch.rand(6, 2, generator=gen, device=DEV)
    x = rows(gen, 6, 256) * torch.tensor([1e9, 1e-9, 3e4, 1e-20, 2.0 ** -100, 1e15], device=DEV)[:, None].bfloat16()
    out = g.gdn_moe_step_routed(x, ex, ids, w)
    for t in range(6):  # each against its own magnitudes
        assert_layer(out[t:t + 1], x[t:t + 1], ex, ids[t:t + 1], w[t:t + 1], f"token {t}")


def test_every_code_is_exact():
    """A token that picks out single weights: every finite e4m3 code comes through as its value."""
    g = lib()
    H = I = 256
    codes = torch.arange(256, dtype=torch.uint8, device=DEV)
    codes[[0x7F, 0xFF]] = 0
    gu = torch.zeros(1, 2, I, H, dtype=torch.uint8, device=DEV)
    gu[0, 0, 0, 0] = 0x7E       # the gate: silu(448 * 1) = 448
    gu[0, 1, 0] = codes         # one up row holds every code
    gu[0, 0, 0, 1:] = 0
    dn = torch.zeros(1, H, I, dtype=torch.uint8, device=DEV)
    dn[0, :, 0] = codes
    one = torch.ones(1, 2, 2, 2, device=DEV)
    ex = g.Experts(gu.view(torch.float8_e4m3fn), dn.view(torch.float8_e4m3fn), one, one[:, 0])
    ids, w = torch.zeros(64, 1, dtype=torch.int32, device=DEV), torch.ones(64, 1, device=DEV)
    for lo in range(0, 256, 64):
        x = torch.zeros(64, H, dtype=torch.bfloat16, device=DEV)
        x[torch.arange(64), torch.arange(lo, lo + 64)] = 1
        x[:, 0] = 1
        out = g.gdn_moe_step_routed(x, ex, ids, w)
        assert_layer(out, x, ex, ids, w, f"codes from {lo}")


def test_strided_rows_and_no_rows():
    g = lib()
    gen = gen_of(11)
    ex = experts(g, gen, 8, 128, 32, 16)
    wide = rows(gen, 6, 400)
    x = wide[:, 40:168]
    assert torch.equal(g.gdn_moe_step(x, ex, 2), g.gdn_moe_step(x.contiguous(), ex, 2))
    assert torch.equal(g.gdn_moe_step(x[::2], ex, 2), g.gdn_moe_step(x[::2].contiguous(), ex, 2))
    assert g.gdn_moe_step(x[:0], ex, 2).shape == (0, 128)
    with pytest.raises(g.GdnError):
        g.gdn_moe_step(wide[:, 1:129], ex, 2)
    with pytest.raises(g.GdnError):
        g.gdn_moe_step(rows(gen, 65, 128), ex, 2)
    with pytest.raises(ValueError):
        g.gdn_moe_step(rows(gen, 4, 144), ex, 2)
    with pytest.raises(ValueError):
        g.gdn_moe_step(x, ex, 2, scoring="other")
    with pytest.raises(ValueError):
        g.Experts(ex.gate_up, ex.down, ex.gate_up_scale)
    with pytest.raises(ValueError):
        g.Experts(ex.gate_up, ex.down[:, :, :16], ex.gate_up_scale, ex.down_scale)


def test_two_streams_and_graphs_at_once():
    """Calls that overlap, each with its own workspace; captured ones replayed on new tokens."""
    g = lib()
    gen = gen_of(12)
    ex = experts(g, gen, 64, 1024, 512, 128, bias=True)
    xs = [rows(gen, T, 1024) for T in (1, 8, 30, 64)]
    want = [g.gdn_moe_step(x, ex, 6, "sigmoid") for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    outs = [[] for _ in xs]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(g.gdn_moe_step(xs[i], ex, 6, "sigmoid"))
    torch.cuda.synchronize()
    for o, y in zip(outs, want):
        assert all(torch.equal(a, y) for a in o)
    graphs, held = [], [torch.empty_like(x) for x in xs]
    for x, y in zip(xs, held):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            for _ in range(3):
                g.gdn_moe_step(x, ex, 6, "sigmoid", out=y)
        graphs.append(gr)
    for x in xs:
        x.copy_(x.roll(17, 1))
    want = [g.gdn_moe_step(x, ex, 6, "sigmoid") for x in xs]
    torch.cuda.synchronize()
    for _ in range(5):
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    g.gdn_check_device_errors()
    for a, b in zip(held, want):
        assert torch.equal(a, b)


def test_far_offsets():
    """Experts beyond 2^31 weights."""
    g = lib()
    E, H, I = 300, 2048, 2048
    gu = torch.zeros(E, 2, I, H, dtype=torch.uint8, device=DEV)
    dn = torch.zeros(E, H, I, dtype=torch.uint8, device=DEV)
    gen = gen_of(13)
    small = experts(g, gen, 2, H, I)
    sg, sd = torch.ones(E, 2, 16, 16, device=DEV), torch.ones(E, 16, 16, device=DEV)
    for a, b in ((0, 0), (E - 1, 1)):
        gu[a], dn[a] = small.gate_up[b].view(torch.uint8), small.down[b].view(torch.uint8)
        sg[a], sd[a] = small.gate_up_scale[b], small.down_scale[b]
    ex = g.Experts(gu.view(torch.float8_e4m3fn), dn.view(torch.float8_e4m3fn), sg, sd)
    x = rows(gen, 3, H)
    w = torch.rand(3, 2, generator=gen, device=DEV)
    far = torch.tensor([[0, E - 1]], dtype=torch.int32, device=DEV).repeat(3, 1)
    near = torch.tensor([[0, 1]], dtype=torch.int32, device=DEV).repeat(3, 1)
    assert torch.equal(g.gdn_moe_step_routed(x, ex, far, w), g.gdn_moe_step_routed(x, small, near, w))


def test_a_hybrid_block_in_8_bits():
    """Input projection, the gated delta rule, output projection and an expert layer, as a model runs them."""
    g = lib()
    from linear_attention_ssm_gb300.synth import Geometry
    gen = gen_of(14)
    geo = Geometry(num_k_heads=2, num_v_heads=4)
    T, H, C, V = 40, 256, geo.conv_dim, 4 * 128

    def weight(n, k):
        return g.gdn_fp8_quantize((torch.randn(n, k, generator=gen, device=DEV) * k ** -0.5).bfloat16(), 128)
    w_in, w_out = weight(C + V, H), weight(H, V)
    ex = experts(g, gen, 12, H, 96, 64, bias=True)
    x = rows(gen, T, H)
    xc, xs = g.gdn_fp8_quantize(x)
    proj = g.gdn_fp8_matmul(xc, xs, *w_in)
    cu = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    conv_w = (0.5 * torch.randn(C, 4, generator=gen, device=DEV)).bfloat16()
    gl, beta = -torch.rand(T, 4, generator=gen, device=DEV), torch.rand(T, 4, generator=gen, device=DEV)
    y = g.gdn_prefill(proj[:, :C].contiguous(), conv_w, cu, gl, beta, proj[:, C:].contiguous().view(T, 4, 128),
                      torch.ones(128, dtype=torch.bfloat16, device=DEV), 128 ** -0.5, geometry=geo)
    yc, ys = g.gdn_fp8_quantize(y.view(T, V))
    mid = x + g.gdn_fp8_matmul(yc, ys, *w_out)
    ids, w = torch.empty(T, 3, dtype=torch.int32, device=DEV), torch.empty(T, 3, device=DEV)
    out = g.gdn_moe_step(mid, ex, 3, "sigmoid", ids=ids, weights=w)
    g.gdn_check_device_errors()
    from tests.fp8_reference import assert_within, product
    want, tol = product(xc, xs, *w_in, torch.bfloat16)
    assert_within(proj, want, tol, "input projection")
    want, tol = product(yc, ys, *w_out, torch.bfloat16)
    assert_within(g.gdn_fp8_matmul(yc, ys, *w_out), want, tol, "output projection")
    assert_choice(ids, w, mid, ex, 3, "sigmoid", True, 1.0)
    assert_layer(out, mid, ex, ids, w)
