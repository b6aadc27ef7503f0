"""The paged-cache attention layer's outputs over the cache or one another are refused, without a GPU."""
from __future__ import annotations

import ctypes

import pytest

from linear_attention_ssm_gb300 import binding
from tests.test_attn_abi import OTHER, attend, cache, geo, lib, prepare, read  # noqa: F401

POOL, SCALES = 4 * 2 * 64 * 256, 4 * 2 * 64  # values and rows of the four pages of two heads
K, V, KS, VS = 0x10000000, 0x20000000, 0x30000000, 0x40000000


def at(x):
    return ctypes.c_void_p(x)


@pytest.mark.parametrize("kind", [0, 1])
def test_outputs_over_the_cache(lib, kind):  # noqa: F811
    def pool():
        return cache(kind, k=K, v=V, ks=KS, vs=VS)
    size = POOL * (2 - kind)
    out = 6 * 16 * 256 * 2  # bytes of an output of the queries
    places = [K, K + size - 16, V, V + size - 16] + ([KS, VS + SCALES - 16] if kind else [])
    for place in places + [V - 16]:  # from before the values into them
        assert attend(lib, c=pool(), out=at(place)) == 1, hex(place)
        assert attend(lib, c=pool(), out=at(place), one=True) == 1
        assert prepare(lib, c=pool(), out=at(place)) == 1
        assert read(lib, c=pool(), k=at(place)) == 1 and read(lib, c=pool(), k=OTHER, v=at(place)) == 1
    # beside it the call goes on, to a refusal of another kind
    bad_rope = ctypes.byref(binding._Rope(24, 0, 1.0, 0x10000))
    for place in [K + size, V - out] + ([] if kind else [KS, VS]):
        assert attend(lib, c=pool(), out=at(place), ws=None) == 7, hex(place)
        assert prepare(lib, c=pool(), out=at(place), rope=bad_rope) == 2
    assert prepare(lib, c=pool(), q=None, out=at(K), rope=bad_rope) == 2  # not an output of that call


def test_read_into_one_place(lib):  # noqa: F811
    pool = cache(0, k=K, v=V)
    kv = 6 * 2 * 256 * 2
    assert read(lib, c=pool, k=OTHER, v=OTHER) == 1
    assert read(lib, c=pool, k=OTHER, v=at(OTHER.value + kv - 16)) == 1
    assert read(lib, c=pool, k=at(OTHER.value + 16), v=OTHER) == 1


def test_queries_in_place(lib):  # noqa: F811
    """q_out is q where every row lies at its own place: a stride that no row uses does not matter."""
    pool, bad_rope = cache(0, k=K, v=V), ctypes.byref(binding._Rope(24, 0, 1.0, 0x10000))

    def call(**kw):
        return prepare(lib, c=pool, q=OTHER, out=OTHER, rope=bad_rope, **kw)
    assert call(qs=(4096, 256)) == 2 and call(qs=(5120, 256)) == 1 and call(qs=(4096, 264)) == 1
    assert call(qs=(5120, 256), n=1, t=1) == 2 and call(qs=(5120, 264), n=1, t=1) == 1
    assert call(g=geo(1, 1), qs=(256, 5120)) == 2 and call(g=geo(1, 1), qs=(512, 256)) == 1
