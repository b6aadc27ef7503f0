"""8-bit products and expert layers without a GPU: refusals before any launch, and the bindings' own checks."""
from __future__ import annotations

import ctypes
import math
import os

import pytest
import torch

from linear_attention_ssm_gb300 import binding


def at(x):
    return ctypes.c_void_p(x)


X, XS, W, WS, OUT, ODD = (at(v) for v in (0x10000000, 0x20000000, 0x30000000, 0x40000000, 0x50000000, 0x18000002))


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        from linear_attention_ssm_gb300 import build
        build.build()
    return binding.load_library()


def quantize(lib, x=X, xs=300, rows=5, cols=300, br=1, codes=W, cs=304, scales=WS):
    return lib.gdn_fp8_quantize(x, xs, rows, cols, br, codes, cs, scales, None)


def test_quantize_refuses(lib):
    for kw in (dict(rows=-1), dict(cols=0), dict(cols=-5), dict(br=0), dict(br=64), dict(x=None), dict(codes=None),
               dict(scales=None), dict(xs=299), dict(cs=288), dict(xs=-300), dict(xs=1 << 40), dict(cs=1 << 40)):
        assert quantize(lib, **kw) == 1, kw
    for kw in (dict(x=ODD), dict(codes=at(0x30000008)), dict(scales=ODD), dict(cs=305), dict(cs=312)):
        assert quantize(lib, **kw) == 3, kw
    assert quantize(lib, rows=0) == 0 and quantize(lib, rows=0, x=None, codes=None, scales=None) == 0
    nx, nc, ns = (4 * 300 + 300) * 2, 4 * 304 + 300, 5 * 3 * 4
    for codes in (0x10000000, 0x10000000 + nx - 8 & ~15, 0x10000000 - nc + 15 & ~15):
        assert quantize(lib, codes=at(codes)) == 1, hex(codes)
    assert quantize(lib, scales=at(0x10000000 + 16)) == 1 and quantize(lib, scales=at(0x30000000 + 16)) == 1
    assert quantize(lib, scales=at(0x30000000 - 48)) == 1  # its last 12 bytes are codes


def matmul(lib, x=X, xs=1008, xsc=XS, w=W, ws=1008, wsc=WS, t=5, n=70, k=1000, kind=0, out=OUT, os_=70):
    return lib.gdn_fp8_matmul(x, xs, xsc, w, ws, wsc, t, n, k, kind, out, os_, None)


def test_matmul_refuses(lib):
    for kw in (dict(t=-1), dict(n=-1), dict(k=0), dict(k=-4), dict(kind=2), dict(kind=-1), dict(x=None), dict(w=None),
               dict(xsc=None), dict(wsc=None), dict(out=None), dict(xs=992), dict(ws=992), dict(os_=69), dict(xs=-1008),
               dict(xs=1 << 40), dict(ws=1 << 40), dict(os_=1 << 40)):
        assert matmul(lib, **kw) == 1, kw
    for kw in (dict(x=ODD), dict(w=at(0x30000008)), dict(xsc=ODD), dict(wsc=ODD), dict(out=ODD), dict(xs=1004), dict(ws=1001)):
        assert matmul(lib, **kw) == 3, kw
    assert matmul(lib, t=0) == 0 and matmul(lib, n=0, os_=0) == 0 and matmul(lib, t=0, x=None, out=None) == 0
    for kw in (dict(out=X), dict(out=W), dict(out=XS), dict(out=WS), dict(out=at(0x30000000 + 69 * 1008 + 992)),
               dict(out=at(0x30000000 - 5 * 70 * 2 + 12 & ~15))):
        assert matmul(lib, **kw) == 1, kw


SIZES = dict(hidden=64, inter=48, num_experts=6, shared_inter=32)


def moe_geo(**kw):
    return binding._MoeGeo(*{**SIZES, **kw}.values())


PARTS = ["router", "router_bias", "gate_up", "down", "gate_up_scale", "down_scale", "shared_gate_up", "shared_down",
         "shared_gate_up_scale", "shared_down_scale", "shared_gate"]


def moe_weights(kind=1, **kw):
    base = {n: 0x100000000 + 0x1000000 * i for i, n in enumerate(PARTS)}
    return binding._MoeWeights(kind, *{**base, **kw}.values())


IDS, WTS, WORK = at(0x60000000), at(0x70000000), at(0x80000000)


def step(lib, geo=None, w=None, top_k=3, scoring=0, scale=1.0, x=X, xs=64, t=4, ids=IDS, wts=WTS, out=OUT, ws=WORK,
         wsb=1 << 40, routed=False, routing=True):
    geo, w = geo or moe_geo(), w or moe_weights()
    if routed:
        return lib.gdn_moe_step_routed(geo, w, ids, wts, top_k, x, xs, t, out, ws, wsb, None)
    r = binding._MoeRouting(top_k, scoring, 1, scale) if routing else None
    return lib.gdn_moe_step(geo, w, r, x, xs, t, ids, wts, out, ws, wsb, None)


@pytest.mark.parametrize("routed", [False, True])
def test_moe_refuses(lib, routed):
    def call(**kw):
        return step(lib, routed=routed, **kw)
    for kw in (dict(hidden=0), dict(hidden=24), dict(inter=0), dict(inter=40), dict(shared_inter=-16), dict(shared_inter=8),
               dict(hidden=16400), dict(inter=1 << 20), dict(num_experts=0), dict(num_experts=1025)):
        assert call(geo=moe_geo(**kw)) == 2, kw
        assert lib.gdn_moe_workspace_size(moe_geo(**kw), 4, 3) == 0
    for kw in (dict(t=-1), dict(t=65), dict(top_k=0), dict(top_k=17), dict(x=None), dict(out=None), dict(xs=56),
               dict(xs=-64), dict(w=moe_weights(2)), dict(w=moe_weights(-1))):
        assert call(**kw) == 1, kw
    for kw in (dict(xs=68), dict(x=ODD), dict(out=ODD), dict(ids=ODD), dict(wts=ODD), dict(ws=at(0x80000010))):
        assert call(**kw) == 3, kw
    for name in PARTS:
        optional = name in ("router_bias", "shared_gate") or (routed and name == "router")
        if not optional:
            assert call(w=moe_weights(**{name: None})) == 1, name
        if not (routed and name.startswith("router")):
            assert call(w=moe_weights(**{name: 0x100000008})) == 3, name
            assert call(out=at(getattr(moe_weights(), name))) == 1, name
    need = lib.gdn_moe_workspace_size(moe_geo(), 4, 3)
    assert need > 0 and need % 256 == 0
    assert call(ws=None) == 7 and call(wsb=need - 1) == 7
    assert call(out=X) == 1 and call(out=IDS) == 1 and call(out=WTS) == 1
    for kw in (dict(ws=X), dict(ws=OUT), dict(ws=IDS), dict(ws=at(0x102000000))):
        assert call(**kw) == 1, kw
    assert call(t=0) == 0 and call(t=0, x=None, out=None, ws=None) == 0
    # what is not read may be anything: scales beside bf16 weights, a shared expert's parts without one; the call
    # goes on to the refusal of its workspace
    assert call(w=moe_weights(0, **{n: 0x100000008 for n in PARTS if n.endswith("scale")}), ws=None) == 7
    assert call(geo=moe_geo(shared_inter=0), w=moe_weights(**{n: None for n in PARTS if n.startswith("shared")}), ws=None) == 7
    assert call(xs=0, t=1, ws=None) == 7  # a single row's stride is of no account


def test_moe_step_refuses_its_routing(lib):
    assert step(lib, routing=False) == 1 and step(lib, top_k=7) == 1
    assert step(lib, scoring=2) == 1
    for scale in (math.inf, math.nan):
        assert step(lib, scale=scale) == 1
    assert step(lib, ids=WTS) == 1 and step(lib, ids=None, wts=None, ws=None) == 7
    assert step(lib, routed=True, ids=None) == 1 and step(lib, routed=True, wts=None) == 1
    assert step(lib, routed=True, top_k=7, ws=None) == 7  # more places than experts: some name none


def test_bindings_refuse_before_the_library():
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    c = torch.zeros(4, 128, dtype=torch.float8_e4m3fn)
    s = torch.zeros(4, 1)
    for call in (lambda: binding.gdn_fp8_quantize(x), lambda: binding.gdn_fp8_matmul(c, s, c, s),
                 lambda: binding.Experts(torch.zeros(2, 2, 16, 16, dtype=torch.bfloat16), x),
                 lambda: binding.gdn_fp8_quantize(None)):
        with pytest.raises(TypeError):
            call()
