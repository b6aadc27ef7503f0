"""The paged-cache attention layer without a GPU: refusals before any launch, the host function of
the rotation's frequencies, and the 64-bit reference's quantiser against torch's e4m3."""
from __future__ import annotations

import ctypes
import math

import pytest
import torch

from linear_attention_ssm_gb300 import binding

FAKE, OTHER, ODD = (ctypes.c_void_p(x) for x in (0x10000, 0x4000000, 0x10002))  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(binding.LIB_PATH):
        from linear_attention_ssm_gb300 import build
        build.build()
    return binding.load_library()


def geo(hq=16, hkv=2, d=256):
    return ctypes.byref(binding._AttnGeo(hq, hkv, d))


def cache(kind=0, page=64, pages=4, k=0x10000, v=0x20000, ks=0x30000, vs=0x40000):
    return ctypes.byref(binding._Cache(kind, page, pages, k, v, ks, vs))


def prepare(lib, g=None, c=None, q=FAKE, qs=(5120, 256), k=FAKE, ks=(5120, 256), v=FAKE, vs=(5120, 256), qw=None, kw=None,
            eps=1e-6, rope=None, table=FAKE, mp=8, kv=FAKE, cu=FAKE, n=2, t=6, out=OTHER):
    return lib.gdn_attn_prepare(g or geo(), q, *qs, k, *ks, v, *vs, qw, kw, eps, rope, c or cache(), table, mp, kv, cu,
                                n, t, out, None)


def attend(lib, g=None, c=None, q=FAKE, table=FAKE, mp=8, kv=FAKE, cu=FAKE, n=2, t=6, scale=0.1, z=None, zs=(256, 256),
           out=OTHER, ws=FAKE, wsb=1 << 40, one=False):
    if one:
        return lib.gdn_attn_decode_step(g or geo(), q, c or cache(), table, mp, kv, t, scale, z, *zs, out, ws, wsb, None)
    return lib.gdn_attn_prefill(g or geo(), q, c or cache(), table, mp, kv, cu, n, t, scale, z, *zs, out, ws, wsb, None)


def read(lib, g=None, c=None, table=FAKE, mp=8, starts=None, cu=FAKE, n=2, t=6, k=FAKE, v=OTHER):
    return lib.gdn_attn_cache_read(g or geo(), c or cache(), table, mp, starts, cu, n, t, k, v, None)


@pytest.mark.parametrize("call", [prepare, attend, read])
def test_geometry_cache_and_batch_are_checked(lib, call):
    for bad in (geo(d=64), geo(hq=3, hkv=2), geo(hkv=0), geo(hq=130, hkv=2), geo(hq=512, hkv=256)):
        assert call(lib, g=bad) == 2
    assert call(lib, c=cache(page=48)) == 2 and call(lib, c=cache(page=8)) == 2
    assert call(lib, c=cache(kind=2)) == 1
    assert call(lib, c=cache(pages=0)) == 1 and call(lib, mp=0) == 1
    assert call(lib, c=cache(k=None)) == 1 and call(lib, c=cache(v=0x20008)) == 3
    assert call(lib, c=cache(kind=1, ks=None)) == 1 and call(lib, c=cache(kind=1, vs=None)) == 1
    assert call(lib, table=None) == 1 and call(lib, table=ODD) == 3
    assert call(lib, cu=ODD) == 3
    assert call(lib, n=-1) == 1 and call(lib, t=-1) == 1 and call(lib, n=0) == 1
    assert call(lib, n=0, t=0) == 0 and call(lib, t=0) == 0


def test_prepare_refuses(lib):
    assert prepare(lib, cu=None) == 1                       # 2 sequences, 6 tokens, one token each
    assert prepare(lib, kv=None) == 1 and prepare(lib, kv=ODD) == 3
    assert prepare(lib, k=None) == 1 and prepare(lib, v=ODD) == 3 and prepare(lib, out=None) == 1
    assert prepare(lib, ks=(5120, 257)) == 3 and prepare(lib, qs=(5124, 256)) == 3
    assert prepare(lib, qw=ODD) == 3 and prepare(lib, kw=ODD) == 3
    assert prepare(lib, eps=-1.0) == 1 and prepare(lib, eps=math.nan) == 1
    assert prepare(lib, out=FAKE) == 1                      # at q's place with other strides
    assert prepare(lib, out=ctypes.c_void_p(0x10000 + 512)) == 1

    def rope(rot, f=0x10000):
        return ctypes.byref(binding._Rope(rot, 0, 1.0, f))
    for bad in (8, 24, 272, -16):
        assert prepare(lib, rope=rope(bad)) == 2
    assert prepare(lib, rope=rope(64, None)) == 1 and prepare(lib, rope=rope(64, 0x10004)) == 3


@pytest.mark.parametrize("one", [False, True])
def test_attention_refuses(lib, one):
    need = lib.gdn_attn_workspace_size(geo())
    assert need > 0 and need % 256 == 0 and lib.gdn_attn_workspace_size(geo(d=64)) == 0
    kw = dict(one=one)
    assert attend(lib, kv=None, **kw) == 1 and attend(lib, q=None, **kw) == 1 and attend(lib, out=ODD, **kw) == 3
    assert attend(lib, out=FAKE, **kw) == 1
    for scale in (0.0, -1.0, math.inf, math.nan):
        assert attend(lib, scale=scale, **kw) == 1
    assert attend(lib, z=ODD, **kw) == 3 and attend(lib, z=FAKE, zs=(256, 4), **kw) == 3
    assert attend(lib, ws=None, **kw) == 7 and attend(lib, wsb=need - 1, **kw) == 7
    assert attend(lib, ws=ctypes.c_void_p(0x10010), **kw) == 3
    if not one:
        assert attend(lib, cu=None) == 1


def test_frequencies():
    f, m = binding.gdn_attn_rope_frequencies(64, 1e6)
    plain = 1e6 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)
    assert m == 1.0 and torch.allclose(f, plain, rtol=1e-14, atol=0)
    f, m = binding.gdn_attn_rope_frequencies(64, 1e6, "linear", factor=4)
    assert m == 1.0 and torch.allclose(f, plain / 4, rtol=1e-14, atol=0)
    f, _ = binding.gdn_attn_rope_frequencies(64, 1e4, "base", factor=8)
    one = 1e4 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)
    assert f[0] == 1.0 and math.isclose(f[-1], one[-1] / 8, rel_tol=1e-12)
    f, m = binding.gdn_attn_rope_frequencies(64, 1e4, "ramp", factor=8, original_positions=4096, low=1, high=32)
    turns = 4096 * one / (2 * math.pi)
    assert math.isclose(m, 0.1 * math.log(8) + 1)
    assert torch.allclose(f[turns >= 32], one[turns >= 32]) and torch.allclose(f[turns <= 1], one[turns <= 1] / 8)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and bool(((f < one) & (f > one / 8))[mid].all())
    for bad in (dict(rot_dim=63), dict(rot_dim=0), dict(rot_dim=-2), dict(base=0.0), dict(base=math.inf),
                dict(scaling="linear", factor=0.0), dict(scaling="base", rot_dim=2, factor=2.0),
                dict(scaling="ramp", factor=2.0, original_positions=0.0),
                dict(scaling="ramp", factor=2.0, original_positions=10.0, low=3.0, high=3.0)):
        with pytest.raises(binding.GdnError):
            binding.gdn_attn_rope_frequencies(**{"rot_dim": 64, "base": 1e4, **bad})
    with pytest.raises(ValueError):
        binding.gdn_attn_rope_frequencies(64, 1e4, "other")


def test_binding_refuses_before_the_library():
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    c = binding.KVCache(torch.zeros(2, 2, 16, 128, dtype=torch.bfloat16), torch.zeros(2, 2, 16, 128, dtype=torch.bfloat16))
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(TypeError):
        binding.gdn_attn_prepare(x, x, x, c, i[:, None], i)
    with pytest.raises(TypeError):
        binding.gdn_attn_decode_step(x, c, i[:, None], i, 0.1)
    with pytest.raises(TypeError):
        binding.gdn_attn_prefill(x, c, i[:, None], i, None, 0.1)


def test_reference_quantiser_is_the_nearest_code():
    """Against torch's conversion, and (the power of two) against its definition."""
    from tests.attn_reference import quantise, two as power
    gen = torch.Generator().manual_seed(0)
    x = (torch.randn(4000, 16, generator=gen) * torch.exp2(torch.randint(-130, 126, (4000, 1), generator=gen))).bfloat16().double()
    codes, byte = quantise(x)
    two = power(byte.long() - 127)
    top = x.abs().amax(-1)
    assert bool((top <= 448 * two).all()) and bool(((top > 224 * two) | (byte == 10)).all())
    assert torch.equal(codes, (x / two[:, None]).float().to(torch.float8_e4m3fn).double())


def test_outputs_that_overlap_what_is_read(lib):
    def at(x):
        return ctypes.c_void_p(x)
    assert attend(lib, z=OTHER) == 1                                   # out is z
    assert attend(lib, z=at(0x4000000 - 512), zs=(4096, 256)) == 1     # z's last rows reach into out
    assert attend(lib, z=at(0x4000000 + 6 * 8192), zs=(-4096, 256)) == 1  # and its first ones, from behind
    assert attend(lib, scale=2e38) == 1 and attend(lib, scale=float("inf")) == 1 and attend(lib, scale=float("nan")) == 1
    assert prepare(lib, k=at(0x4000000 + 512)) == 1 and prepare(lib, v=OTHER) == 1
    assert prepare(lib, k=at(0x4000000 - 52208)) == 1  # k spans (5 * 5120 + 256 + 256) * 2 = 52224 bytes
