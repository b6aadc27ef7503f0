"""The paged-cache attention layer at values where its forms differ: rows of zeros and of tiny values,
values that are not finite behind a token's own position, rows of very different sizes in one block,
tokens whose page does not exist, nine to sixteen query heads to a key head in the single-token form."""
from __future__ import annotations

import math

import pytest
import torch

from tests.attn_reference import DEV, assert_within, attention, dense_rows
from tests.gpu_common import lib
from tests.test_gpu_attn import cu_of, ints, make_cache, run_attention
from tests.test_gpu_attn_edges import call, poison, randn

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


# ------------------------------------------------------------------------------------ behind a token's own position

def seen_marks(bad, q_lens, kv_lens, hq):
    """Whether a row sees a marked value: bad (a list, for each sequence [Hkv, positions, D] bool) -> [T, Hq, D]."""
    rows = []
    for b, ql, kv in zip(bad, q_lens, kv_lens):
        upto = b.long().cumsum(1)  # marked values among the first positions
        pos = torch.arange(kv - ql, kv, device=DEV)
        n = torch.where((pos >= 0)[None, :, None], upto[:, pos.clamp(min=0)], torch.zeros((), dtype=torch.long, device=DEV))
        rows.append((n > 0).repeat_interleave(hq // b.shape[0], 0).transpose(0, 1))
    return torch.cat(rows)


@pytest.mark.parametrize("q_lens,kv_lens,hq,hkv,D", FORMS + [([9, 260], [4, 257], 6, 2, 128), ([100], [2500], 64, 1, 128)])
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("e4m3", [False, True])
def test_values_that_are_not_finite_reach_the_rows_that_see_them(q_lens, kv_lens, hq, hkv, D, page, e4m3):
    """Infinities and NaN in value rows of new tokens: the tokens before them stay as they are, the others have them."""
    g = lib()
    gen = torch.Generator(device=DEV).manual_seed(22)
    cache, table = make_cache(g, gen, q_lens, kv_lens, hkv, page, D, e4m3)
    clean = g.KVCache(cache.k, cache.v.clone(), cache.k_scale, cache.v_scale)
    marks = []  # of NaN, of +inf, of -inf (an e4m3 code has NaN alone)
    for n, (ql, kv) in enumerate(zip(q_lens, kv_lens)):
        m = torch.zeros(3, hkv, kv, D, dtype=torch.bool, device=DEV)
        lo = max(kv - ql, 0)
        for i, p in enumerate(sorted({lo, lo + 1, lo + (kv - lo) // 3, lo + (kv - lo) // 2, lo + 2 * (kv - lo) // 3, kv - 2, kv - 1} - {-1})):
            m[0 if e4m3 else i % 3, i % hkv, min(p, kv - 1), 7 * i + 1::D // 2] = True
        m[0, 0, kv - 1, 100] = True
        if kv - ql > 200:
            m[0, 0, 50, 5] = True  # before every new token
        marks.append(m)
        for p in m.any(0).any(0).any(-1).nonzero().flatten().tolist():
            row = cache.v[int(table[n, p // page]), :, p % page]
            row, at = (row.view(torch.uint8), m[:, :, p]) if e4m3 else (row, m[:, :, p])
            for value, w in zip((0x7F,) if e4m3 else (math.nan, math.inf, -math.inf), at):
                row[w] = value
    q = randn(gen, sum(q_lens), hq, D) * 0.3
    out = call(g, q, cache, table, q_lens, kv_lens, D ** -0.5).double()
    g.gdn_check_device_errors()
    nan, up, down = (seen_marks([m[i] for m in marks], q_lens, kv_lens, hq) for i in range(3))
    nan = nan | (up & down)
    assert torch.equal(torch.isnan(out), nan)
    assert torch.equal(torch.isposinf(out), up & ~nan) and torch.equal(torch.isneginf(out), down & ~nan)
    # the rest: as if those values were not there (their rows' other values and weights are)
    for n, m in enumerate(marks):
        for p in m.any(0).any(0).any(-1).nonzero().flatten().tolist():
            row = clean.v[int(table[n, p // page]), :, p % page]
            (row.view(torch.uint8) if e4m3 else row)[m[:, :, p].any(0)] = 0
    want, tol = attention(q, clean, table, q_lens, kv_lens, D ** -0.5)
    fine = torch.isfinite(out)
    assert bool(((out - want).abs() <= tol)[fine].all())


@pytest.mark.parametrize("e4m3", [False, True])
def test_a_gated_row_beside_values_that_are_not_finite(e4m3):
    """With a gate, and rows cut into parts: only the last token has the NaN."""
    g = lib()
    gen = torch.Generator(device=DEV).manual_seed(23)
    for q_lens, kv_lens, hq, hkv, D in (([20], [6000], 16, 2, 256), ([90], [9000], 8, 2, 128)):
        cache, table = make_cache(g, gen, q_lens, kv_lens, hkv, 64, D, e4m3)
        q, z = randn(gen, q_lens[0], hq, D), randn(gen, q_lens[0], hq, D)
        want, tol = attention(q, cache, table, q_lens, kv_lens, D ** -0.5, z)
        p = kv_lens[0] - 1
        row = cache.v[int(table[0, p // 64]), :, p % 64]
        row.copy_(torch.full(row.shape, math.nan, device=DEV).to(row.dtype))
        out = g.gdn_attn_prefill(q, cache, table, ints(kv_lens), cu_of(q_lens), D ** -0.5, z=z)
        g.gdn_check_device_errors()
        assert bool(torch.isnan(out[-1]).all())
        assert_within(out[:-1], want[:-1], tol[:-1], "attention")


def test_values_that_are_not_finite_under_bad_cu_seqlens():
    """Sequences that overlap and decrease: reported, whatever the values are."""
    g = lib()
    gen = torch.Generator(device=DEV).manual_seed(27)
    cache, table = make_cache(g, gen, [4, 4, 4], [40, 40, 40], 2, 16, 128, False)
    cache.v[:] = math.nan
    q = randn(gen, 12, 8, 128)
    for cu in ([0, 8, 3, 12], [0, 12, 2, 5], [0, -4, 6, 12], [5, 4, 12, 3]):
        g.gdn_attn_prefill(q, cache, table, ints([40, 40, 40]), ints(cu), 0.1)
        with pytest.raises(g.GdnError) as e:
            g.gdn_check_device_errors()
        assert e.value.status == 6


# ------------------------------------------------------------------------------------ rows of very different sizes

@pytest.mark.parametrize("apart", [10, 20, 24, 28])
@pytest.mark.parametrize("hq,hkv,D,q_len", [(8, 2, 128, 120), (2, 2, 128, 120), (4, 1, 256, 120)])
@pytest.mark.parametrize("e4m3", [False, True])
def test_rows_do_not_go_by_the_size_of_later_ones(hq, hkv, D, q_len, e4m3, apart):
    """Keys and values of the first 60 positions 2^-apart of those behind them in the same block: the first rows come
    out as they would alone (the error counted from what they see)."""
    g = lib()
    gen = torch.Generator(device=DEV).manual_seed(24)
    k, v, q = randn(gen, q_len, hkv, D), randn(gen, q_len, hkv, D), randn(gen, q_len, hq, D)
    half = 2.0 ** (apart // 2)
    k[:60] /= half
    v[:60] /= half
    k[60:] *= half
    v[60:] *= half
    q[:60] *= half
    q[60:] /= half
    cache, table = written(g, k, v, [q_len], [q_len], 32, e4m3)
    out = g.gdn_attn_prefill(q, cache, table, ints([q_len]), ints([0, q_len]), D ** -0.5)
    g.gdn_check_device_errors()
    want, tol = attention(q[:60], cache, table, [60], [60], D ** -0.5)
    if e4m3 and apart > 20:
        # Widened codes carry 2^7 and their row's power of two relative to the block's largest.  The largest row's top
        # code is 224 or more, 2^14.8 with the factor; rows more than 2^22 below round in steps of 2^-24, by 2^-25 at most:
        # less than 2^-39 of the block's largest value, and as much of its largest key in every term of a score (a
        # relative change of a weight, in numerator and denominator), then the rounding of the result.
        kd, vd = dense_rows(cache, table[0], q_len)
        rel = 2.0 ** -39 * D ** -0.5 * kd.abs().max() * q[:60].double().abs().sum(-1, keepdim=True)
        tol = tol + (1 + 2.0 ** -8) * (2.0 ** -39 * vd.abs().max() + 2 * rel * vd[:, :60].abs().max())
    assert_within(out[:60], want, tol, "first rows")
    want, tol = attention(q, cache, table, [q_len], [q_len], D ** -0.5)
    assert_within(out[60:], want[60:], tol[60:], "last rows")


# ------------------------------------------------------------------------------------ faults

@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("e4m3", [False, True])
def test_nothing_is_written_for_a_token_without_a_page(e4m3, in_place):
    """A page outside the pool, a length beyond the table: the queries of those tokens are left as well."""
    g = lib()
    gen = torch.Generator(device=DEV).manual_seed(26)
    cache, table = make_cache(g, gen, [1] * 4, [40] * 4, 2, 16, 128, e4m3)
    q, k, v = randn(gen, 4, 4, 128), randn(gen, 4, 2, 128), randn(gen, 4, 2, 128)
    w = torch.full((128,), 2.0, dtype=torch.bfloat16, device=DEV)
    good = g.gdn_attn_prepare(q, k, v, cache, table, ints([40] * 4), q_norm_w=w)
    g.gdn_check_device_errors()
    table[1, 2], table[2, 2] = -1, cache.k.shape[0]
    q_out = q.clone() if in_place else torch.full_like(q, 7.0)
    before = q_out.clone()
    g.gdn_attn_prepare(q_out if in_place else q, k, v, cache, table, ints([40, 40, 40, 16 * table.shape[1] + 1]), q_norm_w=w, q_out=q_out)
    with pytest.raises(g.GdnError) as e:
        g.gdn_check_device_errors()
    assert e.value.status == 6
    assert torch.equal(q_out[0], good[0]) and torch.equal(q_out[1:], before[1:])


def test_rows_before_the_first_sequence_are_reported():
    """cu_seqlens that does not begin at 0: an error in every call, the sequences themselves as ever."""
    g = lib()
    gen = torch.Generator(device=DEV).manual_seed(28)
    cache, table = make_cache(g, gen, [3, 4], [40, 50], 2, 16, 128, False)
    q, kv = randn(gen, 9, 4, 128), randn(gen, 9, 2, 128)
    lens, cu = ints([40, 50]), ints([2, 5, 9])
    out = torch.full_like(q, 7.0)
    g.gdn_attn_prefill(q, cache, table, lens, cu, 0.1, out=out)
    with pytest.raises(g.GdnError) as e:
        g.gdn_check_device_errors()
    assert e.value.status == 6 and bool((out[:2] == 7.0).all())
    want, tol = attention(q[2:], cache, table, [3, 4], [40, 50], 0.1)
    assert_within(out[2:], want, tol, "attention")
    for call_it in (lambda: g.gdn_attn_prepare(q, kv, kv, cache, table, lens, cu),
                    lambda: g.gdn_attn_cache_read(cache, table, cu, kv, kv.clone())):
        call_it()
        with pytest.raises(g.GdnError):
            g.gdn_check_device_errors()


@pytest.mark.parametrize("D,e4m3", [(128, False), (256, True)])
def test_more_positions_than_31_bits_hold_blocks_of(D, e4m3):
    """A table of 2^24 pages of 128 rows (all the same one): the last 255 of its lengths are refused by every call."""
    g = lib()
    gen = torch.Generator(device=DEV).manual_seed(29)
    cache, _ = make_cache(g, gen, [1], [100], 2, 128, D, e4m3)
    table = torch.zeros(1, 2 ** 24, dtype=torch.int32, device=DEV)
    q, kv = randn(gen, 3, 8, D), randn(gen, 3, 2, D)
    for length in (2 ** 31 - 255, 2 ** 31 - 1):
        lens, cu = ints([length]), ints([0, 3])
        for call_it in (lambda: g.gdn_attn_prefill(q, cache, table, lens, cu, 0.1), lambda: g.gdn_attn_prepare(q, kv, kv, cache, table, lens, cu),
                        lambda: g.gdn_attn_decode_step(q[:1].clone(), cache, table, lens, 0.1),
                        lambda: g.gdn_attn_cache_read(cache, table, cu, kv, kv.clone(), starts=ints([length]))):
            call_it()
            with pytest.raises(g.GdnError) as e:
                g.gdn_check_device_errors()
            assert e.value.status == 6
    g.gdn_attn_prepare(q, kv, kv, cache, table, ints([2 ** 31 - 256]), ints([0, 3]))  # the last that has a place
    g.gdn_check_device_errors()


# ------------------------------------------------------------------------------------ nine to sixteen heads to a key head

@pytest.mark.parametrize("kv_lens", [[1], [0, 1, 127, 128, 129, 5000], [20000, 3], [700] * 33])
@pytest.mark.parametrize("page,gate", [(16, True), (64, False), (128, True)])
@pytest.mark.parametrize("hq,hkv,D", [(9, 1, 128), (24, 2, 128), (16, 1, 128), (15, 1, 128), (64, 4, 128), (17, 1, 128), (9, 1, 256), (32, 2, 256)])
@pytest.mark.parametrize("e4m3", [False, True])
def test_decode_step_with_more_heads_to_a_key_head(kv_lens, page, gate, hq, hkv, D, e4m3):
    """The single-token kernel's form of two columns of eight rows (D = 128, 9 to 16 heads), and both sides of the
    borders where larger groups go to tiles."""
    run_attention(lib(), [1] * len(kv_lens), kv_lens, hq, hkv, D, page, e4m3, gate, decode=True, seed=hq)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("hq", [9, 12, 16])
def test_decode_step_with_more_heads_behind_the_last_key(hq, e4m3):
    g = lib()
    gen = torch.Generator(device=DEV).manual_seed(25)
    kv_lens = [130, 1, 64, 33, 3000]
    cache, table = make_cache(g, gen, [1] * 5, kv_lens, 1, 32, 128, e4m3)
    poison(cache, table, kv_lens, 32)
    q = randn(gen, 5, hq, 128) * 6
    out = g.gdn_attn_decode_step(q, cache, table, ints(kv_lens), 0.09)
    again = g.gdn_attn_decode_step(q, cache, table, ints(kv_lens), 0.09)
    g.gdn_check_device_errors()
    want, tol = attention(q, cache, table, [1] * 5, kv_lens, 0.09)
    assert_within(out, want, tol, "attention")
    assert torch.equal(out, again)
