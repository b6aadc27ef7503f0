"""The paged-cache attention layer at values where its forms differ: rows of zeros and of tiny values."""
from __future__ import annotations

import pytest
import torch

from tests.attn_reference import DEV, assert_within, attention
from tests.gpu_common import lib
from tests.test_gpu_attn import cu_of, ints, make_cache
from tests.test_gpu_attn_edges import call, randn

pytestmark = pytest.mark.gpu

# the kernel's forms: one and two tiles of 128 rows at D = 128 (by tokens and group), one at D = 256
FORMS = [([30], [30], 8, 2, 128), ([200], [200], 8, 2, 128), ([40, 3, 17], [300, 3, 130], 8, 2, 128), ([150], [900], 8, 1, 256),
         ([5, 70], [129, 70], 12, 1, 256), ([300], [5000], 8, 2, 128)]


def written(g, k, v, q_lens, kv_lens, page, e4m3):
    """A cache that holds k and v [positions of all sequences, Hkv, D], and its block table."""
    gen = torch.Generator(device=DEV).manual_seed(0)
    cache, table = make_cache(g, gen, q_lens, kv_lens, k.shape[1], page, k.shape[2], e4m3, fill=False)
    g.gdn_attn_prepare(None, k, v, cache, table, ints(kv_lens), cu_of(kv_lens))
    g.gdn_check_device_errors()
    return cache, table


# ------------------------------------------------------------------------------------ zero and tiny rows

@pytest.mark.parametrize("q_size,k_size", [(0.0, 0.0), (0.0, 1.0), (0.0, 2.0 ** -40), (1.0, 0.0), (2.0 ** -100, 2.0 ** -100), (2.0 ** -126, 0.0)])
@pytest.mark.parametrize("q_lens,kv_lens,hq,hkv,D", FORMS)
@pytest.mark.parametrize("e4m3", [False, True])
def test_zero_and_tiny_queries_and_keys(q_lens, kv_lens, hq, hkv, D, e4m3, q_size, k_size):
    """A warm-up pass over zeros, padding tokens: every weight is the same, the result the mean of the values seen."""
    g = lib()
    gen = torch.Generator(device=DEV).manual_seed(20)
    k, v = randn(gen, sum(kv_lens), hkv, D) * k_size, randn(gen, sum(kv_lens), hkv, D)
    cache, table = written(g, k, v, q_lens, kv_lens, 32, e4m3)
    q = randn(gen, sum(q_lens), hq, D) * q_size
    out = call(g, q, cache, table, q_lens, kv_lens, D ** -0.5)
    one = g.gdn_attn_decode_step(q[cu_of(q_lens)[1:].long() - 1].contiguous(), cache, table, ints(kv_lens), D ** -0.5)
    g.gdn_check_device_errors()
    want, tol = attention(q, cache, table, q_lens, kv_lens, D ** -0.5)
    assert_within(out, want, tol, "attention")
    last = cu_of(q_lens)[1:].long() - 1
    assert_within(one, want[last], tol[last], "one token")


@pytest.mark.parametrize("q_lens,kv_lens,hq,hkv,D", FORMS)
def test_single_rows_of_zeros_among_others(q_lens, kv_lens, hq, hkv, D):
    g = lib()
    gen = torch.Generator(device=DEV).manual_seed(21)
    k, v = randn(gen, sum(kv_lens), hkv, D), randn(gen, sum(kv_lens), hkv, D)
    k[::3] = 0
    k[-140:] = 0
    cache, table = written(g, k, v, q_lens, kv_lens, 16, True)
    q = randn(gen, sum(q_lens), hq, D)
    q[::2] = 0
    q[1::4, ::2] *= 2.0 ** -90
    out = call(g, q, cache, table, q_lens, kv_lens, D ** -0.5)
    g.gdn_check_device_errors()
    want, tol = attention(q, cache, table, q_lens, kv_lens, D ** -0.5)
    assert_within(out, want, tol, "attention")
