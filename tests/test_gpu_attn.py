"""The paged-cache attention layer on the GPU against its definition in 64 bits."""
from __future__ import annotations

import math

import pytest
import torch

from tests.attn_reference import DEV, assert_within, attention, norm_rotate, positions, quantise, two
from tests.gpu_common import Guarded, lib

pytestmark = pytest.mark.gpu
EPS = 1e-6


def make_cache(g, gen, q_lens, kv_lens, hkv, page, D, e4m3, fill=True, spare=3, wide=2):
    """A cache whose sequences' pages are scattered over the pool, and the block table (entries that
    no position needs are -1)."""
    need = [-(-x // page) for x in kv_lens]
    pool = sum(need) + spare
    order = torch.randperm(pool, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((len(kv_lens), max(need + [1]) + wide), -1, dtype=torch.int32, device=DEV)
    at = 0
    for n, c in enumerate(need):
        table[n, :c] = order[at:at + c]
        at += c
    cache = g.KVCache.allocate(pool, hkv, page, D, torch.float8_e4m3fn if e4m3 else torch.bfloat16)
    if fill:
        k, v = (torch.randn(pool, hkv, page, D, generator=gen, device=DEV).bfloat16() for _ in range(2))
        k = k * torch.exp2(torch.randint(-6, 2, (pool, hkv, page, 1), generator=gen, device=DEV)).bfloat16()
        v = v * torch.exp2(torch.randint(-9, 9, (pool, hkv, page, 1), generator=gen, device=DEV)).bfloat16()
        if e4m3:
            for x, codes, scale in ((k, cache.k, cache.k_scale), (v, cache.v, cache.v_scale)):
                c, b = quantise(x.double())
                codes.copy_(c.to(torch.float32).to(torch.float8_e4m3fn))
                scale.copy_(b)
        else:
            cache.k.copy_(k)
            cache.v.copy_(v)
    return cache, table


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def cu_of(q_lens):
    return ints([sum(q_lens[:i]) for i in range(len(q_lens) + 1)])


def run_attention(g, q_lens, kv_lens, hq, hkv, D, page, e4m3, gate, seed=0, decode=False, q_std=1.0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    T = sum(q_lens)
    cache, table = make_cache(g, gen, q_lens, kv_lens, hkv, page, D, e4m3)
    q = (torch.randn(T, hq, D, generator=gen, device=DEV) * q_std).bfloat16()
    both = torch.randn(T, hq, 2 * D, generator=gen, device=DEV).bfloat16()
    z = both[..., D:] if gate else None  # a strided view, as a joint projection gives it
    out = Guarded((T, hq, D), torch.bfloat16)
    scale = 1 / math.sqrt(D)
    if decode:
        g.gdn_attn_decode_step(q, cache, table, ints(kv_lens), scale, z=z, out=out.t)
    else:
        g.gdn_attn_prefill(q, cache, table, ints(kv_lens), cu_of(q_lens), scale, z=z, out=out.t)
    g.gdn_check_device_errors()
    out.check("out")
    want, tol = attention(q, cache, table, q_lens, kv_lens, scale, z)
    assert_within(out.t, want, tol, "attention")
    return out.t


CHUNKS = [
    ([1], [1]),                                   # one token, nothing before it
    ([5], [5]),
    ([128], [128]),
    ([129], [257]),                               # one row past a tile, one key past a block
    ([17, 0, 300, 1], [1017, 40, 300, 700]),      # a sequence without new tokens
    ([7, 3, 4], [3, 3, 0]),                       # rows before the first position, an unused slot
    ([64, 200, 33], [4096, 640, 1933]),
]


@pytest.mark.parametrize("q_lens,kv_lens", CHUNKS)
@pytest.mark.parametrize("hq,hkv,D,page,e4m3,gate", [
    (4, 4, 128, 16, False, False), (6, 2, 128, 32, True, True), (16, 2, 256, 64, False, True),
    (5, 1, 256, 16, True, False), (64, 1, 128, 128, False, False), (24, 3, 256, 128, True, True)])
def test_prefill_against_the_definition(q_lens, kv_lens, hq, hkv, D, page, e4m3, gate):
    run_attention(lib(), q_lens, kv_lens, hq, hkv, D, page, e4m3, gate)


@pytest.mark.parametrize("kv_lens", [[1], [700], [0, 1, 127, 128, 129, 5000], [300] * 40, [20000, 3]])
@pytest.mark.parametrize("hq,hkv,D,page,e4m3,gate", [
    (4, 4, 128, 16, False, False), (48, 16, 128, 64, True, True), (16, 2, 256, 64, False, True),
    (7, 1, 256, 16, True, False), (128, 2, 128, 128, False, False)])
def test_decode_step_against_the_definition(kv_lens, hq, hkv, D, page, e4m3, gate):
    run_attention(lib(), [1] * len(kv_lens), kv_lens, hq, hkv, D, page, e4m3, gate, decode=True)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D", [128, 256])
def test_sharp_scores_and_growing_maximum(D, e4m3):
    """Queries that make one key's weight 1 and the rest 0, with the maximum found late."""
    run_attention(lib(), [70], [1500], 8, 2, D, 32, e4m3, False, q_std=12.0)


@pytest.mark.parametrize("e4m3", [False, True])
def test_rows_without_keys_are_zero(e4m3):
    g = lib()
    out = run_attention(g, [9, 2], [4, 0], 8, 2, 128, 16, e4m3, True)
    assert torch.count_nonzero(out[:5]) == 0 and torch.count_nonzero(out[9:]) == 0
    assert torch.count_nonzero(out[5:9]) > 0


def test_rows_behind_the_last_sequence_are_left():
    g = lib()
    gen = torch.Generator(device=DEV).manual_seed(1)
    cache, table = make_cache(g, gen, [3], [40], 2, 16, 128, False)
    q = torch.randn(8, 4, 128, generator=gen, device=DEV).bfloat16()
    out = torch.full_like(q, 7.0)
    g.gdn_attn_prefill(q, cache, table, ints([40]), ints([0, 3]), 0.1, out=out)
    assert torch.equal(out[3:], torch.full_like(out[3:], 7.0)) and not torch.equal(out[:3], torch.full_like(out[:3], 7.0))
    q_out = torch.full_like(q, 7.0)
    kv = torch.randn(8, 2, 128, generator=gen, device=DEV).bfloat16()
    before = cache.k.clone()
    g.gdn_attn_prepare(q, kv, kv, cache, table, ints([40]), ints([0, 3]), q_out=q_out)
    g.gdn_check_device_errors()
    assert torch.equal(q_out[3:], torch.full_like(q_out[3:], 7.0)) and torch.equal(q_out[:3], q[:3])
    changed = (cache.k != before).any(-1).any(1)  # [pages, rows]
    assert int(changed.sum()) == 3


def test_two_calls_give_the_same_bits():
    g = lib()
    a = run_attention(g, [100, 3, 50], [3000, 2000, 50], 16, 2, 256, 64, False, True, seed=3).clone()
    b = run_attention(g, [100, 3, 50], [3000, 2000, 50], 16, 2, 256, 64, False, True, seed=3)
    assert torch.equal(a, b)


# ------------------------------------------------------------------------------------ prepare and read

PREPARE = [
    # hq, hkv, D, page, e4m3, rot, interleaved, norm
    (16, 2, 256, 64, True, 64, False, True), (16, 2, 256, 16, False, 256, True, True),
    (4, 4, 128, 32, False, 128, False, True), (6, 2, 128, 128, True, 96, False, False),
    (3, 1, 128, 16, True, 32, True, True), (5, 5, 256, 32, False, 0, False, False),
    (2, 1, 256, 64, True, 16, True, False), (7, 7, 128, 16, False, 48, True, True)]


@pytest.mark.parametrize("q_lens,kv_lens", [([1], [1]), ([1, 1, 1], [5, 1000000, 0]), ([40, 0, 7, 300], [90, 12, 3, 300]),
                                            ([1500], [2000000])])
@pytest.mark.parametrize("hq,hkv,D,page,e4m3,rot,interleaved,norm", PREPARE)
def test_prepare_against_the_definition(q_lens, kv_lens, hq, hkv, D, page, e4m3, rot, interleaved, norm):
    g = lib()
    gen = torch.Generator(device=DEV).manual_seed(rot + D)
    T = sum(q_lens)
    qkv = torch.randn(T, hq + 2 * hkv, D, generator=gen, device=DEV) * 3
    qkv = (qkv * torch.exp2(torch.randint(-8, 8, (T, hq + 2 * hkv, 1), generator=gen, device=DEV))).bfloat16()
    q, k, v = qkv.split([hq, hkv, hkv], dim=1)
    wq, wk = (1 + 0.3 * torch.randn(2, D, generator=gen, device=DEV)).bfloat16() if norm else (None, None)
    freqs, mag = None, 1.0
    if rot:
        freqs, mag = g.gdn_attn_rope_frequencies(rot, 1e6, "ramp", factor=8.0, original_positions=32768)
        freqs = freqs.to(DEV)
    # only the pages the new tokens lie in exist
    page_of = [[max(kv - ql, 0) // page, -(-kv // page)] for ql, kv in zip(q_lens, kv_lens)]
    pool = sum(b - a for a, b in page_of) + 2
    table = torch.full((len(q_lens), max(b for _, b in page_of) + 1), -1, dtype=torch.int32, device=DEV)
    order, at = torch.randperm(pool, generator=gen, device=DEV).to(torch.int32), 0
    for n, (a, b) in enumerate(page_of):
        table[n, a:b] = order[at:at + b - a]
        at += b - a
    cache = g.KVCache.allocate(pool, hkv, page, D, torch.float8_e4m3fn if e4m3 else torch.bfloat16)
    for x in (cache.k, cache.v):
        x.view(torch.uint8).fill_(0x5A)
    q_out = Guarded((T, hq, D), torch.bfloat16)
    cu = None if all(x == 1 for x in q_lens) else cu_of(q_lens)
    g.gdn_attn_prepare(q, k, v, cache, table, ints(kv_lens), cu, wq, wk, freqs, interleaved, mag, EPS, q_out.t)
    g.gdn_check_device_errors()
    q_out.check("q_out")

    seq, pos = positions(q_lens, kv_lens)
    want, size = norm_rotate(q, wq, pos, freqs, interleaved, mag, EPS)
    # fp32 arithmetic and the angle's 2^-23 turns (2 pi 2^-23 of the pair), then one rounding to bf16
    assert_within(q_out.t, want, 2.0 ** -8 * want.abs() + 2.0 ** -18 * size, "q")
    want_k, size_k = norm_rotate(k, wk, pos, freqs, interleaved, mag, EPS)
    tol_k = 2.0 ** -8 * want_k.abs() + 2.0 ** -18 * size_k
    written = torch.zeros(pool, page, dtype=torch.bool, device=DEV)
    for t, (n, p) in enumerate(zip(seq, pos)):
        if p < 0:
            continue
        pg, row = int(table[n, p // page]), p % page
        written[pg, row] = True
        if t % max(1, T // 50):
            continue
        got_k, got_v = cache.k[pg, :, row], cache.v[pg, :, row]
        if e4m3:
            ks, vs = (two(s[pg, :, row].long() - 127)[:, None] for s in (cache.k_scale, cache.v_scale))
            c, b = quantise(v[t].double())
            assert torch.equal(cache.v_scale[pg, :, row], b) and torch.equal(got_v.double(), c)
            # half a step of e4m3 on top: 2^-4 of the value, or half its smallest step
            assert_within(got_k.double() * ks, want_k[t], tol_k[t] + 2.0 ** -4 * (want_k[t].abs() + tol_k[t]) + 2.0 ** -10 * ks,
                          "k")
            top = got_k.double().abs().amax(-1)
            assert bool(((top >= 208) & (top <= 448)).all())  # the least power of two: the top code is over 448 / 2, less half a step
        else:
            assert_within(got_k, want_k[t], tol_k[t], "k")
            assert torch.equal(got_v, v[t])
    for x in (cache.k, cache.v):  # nothing else in the pool was touched
        rest = x.view(torch.uint8).permute(0, 2, 1, 3)[~written]
        assert bool((rest == 0x5A).all())


def test_prepare_in_place_and_without_queries():
    g = lib()
    gen = torch.Generator(device=DEV).manual_seed(0)
    cache, table = make_cache(g, gen, [50], [50], 2, 16, 128, False, fill=False)
    q = torch.randn(50, 4, 128, generator=gen, device=DEV).bfloat16()
    k, v = (torch.randn(50, 2, 128, generator=gen, device=DEV).bfloat16() for _ in range(2))
    freqs = g.gdn_attn_rope_frequencies(64, 1e4)[0].to(DEV)
    w = torch.ones(128, dtype=torch.bfloat16, device=DEV)
    a = g.gdn_attn_prepare(q, k, v, cache, table, ints([50]), ints([0, 50]), w, w, freqs)
    keys = cache.k.clone()
    b = q.clone()
    assert g.gdn_attn_prepare(b, k, v, cache, table, ints([50]), ints([0, 50]), w, w, freqs, q_out=b) is b
    assert torch.equal(a, b)
    cache.k.zero_()
    assert g.gdn_attn_prepare(None, k, v, cache, table, ints([50]), ints([0, 50]), None, w, freqs) is None
    g.gdn_check_device_errors()
    assert torch.equal(cache.k, keys)


def test_quantised_rows_of_every_kind():
    """Rows of zeros, of the smallest and largest bf16 values, at a power's border, with infinities and NaN."""
    g = lib()
    D, big = 128, 3.3895e38
    tops = [0.0, 2.0 ** -133, 2.0 ** -126, 1.75, 1.7578125, 448.0, 450.0, 1.0, 3.5, 3.515625, big, 1e-30]
    gen = torch.Generator(device=DEV).manual_seed(0)
    x = torch.rand(len(tops), 1, D, generator=gen, device=DEV) * 2 - 1
    x = (x.double() * torch.tensor(tops, device=DEV)[:, None, None]).bfloat16()
    x[:, 0, 3] = torch.tensor(tops, device=DEV).bfloat16()
    x[4, 0, 7], x[5, 0, 8], x[6, 0, 9] = math.inf, -math.inf, math.nan
    x[0, 0, 5] = -0.0
    T = len(tops)
    cache, table = make_cache(g, gen, [T], [T], 1, 16, D, True, fill=False)
    g.gdn_attn_prepare(None, x, x.flip(-1).contiguous(), cache, table, ints([T]), ints([0, T]))
    codes, byte = quantise(x[:, 0].double())
    pg = int(table[0, 0])
    assert torch.equal(cache.k_scale[pg, 0, :T], byte)
    assert torch.equal(torch.nan_to_num(cache.k[pg, 0, :T].double(), nan=999.), torch.nan_to_num(codes, nan=999.))
    k_out, v_out = (torch.empty(T, 1, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    g.gdn_attn_cache_read(cache, table, ints([0, T]), k_out, v_out)
    g.gdn_check_device_errors()
    value = codes * two(byte.long() - 127)[:, None]
    # exact in bf16, but for the largest row: 255 * 2^120 is rounded to the code 256, and 2^128 is no bf16 number
    over = value.abs() >= 2.0 ** 128
    assert set(over.any(-1).nonzero().flatten().tolist()) <= {tops.index(big)}
    value = torch.where(over, value * math.inf, value)
    assert torch.equal(value.bfloat16().double().nan_to_num(nan=999.), value.nan_to_num(nan=999.))
    assert torch.equal(k_out[:, 0].double().nan_to_num(nan=999.), value.nan_to_num(nan=999.))
    assert torch.equal(v_out.flip(-1).double().nan_to_num(nan=999.), k_out.double().nan_to_num(nan=999.))


@pytest.mark.parametrize("hkv,D,page,e4m3", [(2, 256, 64, True), (8, 128, 16, False), (3, 128, 128, True), (1, 256, 32, False)])
def test_cache_read_from_the_middle(hkv, D, page, e4m3):
    from tests.attn_reference import dense_rows
    g = lib()
    gen = torch.Generator(device=DEV).manual_seed(0)
    kv, starts, lens = [300, 1, 2000, 77], [13, 0, 900, 77], [287, 1, 700, 0]
    cache, table = make_cache(g, gen, lens, kv, hkv, page, D, e4m3)
    outs = [Guarded((sum(lens), hkv, D), torch.bfloat16) for _ in range(2)]
    g.gdn_attn_cache_read(cache, table, cu_of(lens), outs[0].t, outs[1].t, starts=ints(starts))
    g.gdn_check_device_errors()
    at = 0
    for n, (s, c) in enumerate(zip(starts, lens)):
        for o, x in zip(outs, dense_rows(cache, table[n], kv[n])):
            assert torch.equal(o.t[at:at + c].double(), x[:, s:s + c].transpose(0, 1))
        at += c
    for o in outs:
        o.check("read")


# ------------------------------------------------------------------------------------ faults, streams, graphs

def test_bad_pages_and_lengths_are_reported():
    g = lib()
    gen = torch.Generator(device=DEV).manual_seed(0)
    cache, table = make_cache(g, gen, [1, 1], [40, 40], 2, 16, 128, False)
    q = torch.randn(2, 4, 128, generator=gen, device=DEV).bfloat16()
    good = g.gdn_attn_decode_step(q, cache, table, ints([40, 40]), 0.1)
    g.gdn_check_device_errors()
    pages = cache.k.shape[0]
    for bad in (-1, pages, 2 ** 31 - 1):
        broken = table.clone()
        broken[1, 1] = bad
        out = g.gdn_attn_decode_step(q, cache, broken, ints([40, 40]), 0.1)
        with pytest.raises(g.GdnError) as e:
            g.gdn_check_device_errors()
        assert e.value.status == 6 and torch.equal(out[0], good[0])
        before = cache.k.clone()
        g.gdn_attn_prepare(None, q[:, :2].contiguous(), q[:, 2:].contiguous(), cache, broken, ints([0, 20]))
        with pytest.raises(g.GdnError):
            g.gdn_check_device_errors()
        assert torch.equal(cache.k, before)
        rows = torch.zeros(2, 2, 128, dtype=torch.bfloat16, device=DEV)
        g.gdn_attn_cache_read(cache, broken, ints([0, 1, 2]), rows, rows.clone(), starts=ints([0, 20]))
        with pytest.raises(g.GdnError):
            g.gdn_check_device_errors()
    for kv in (-5, table.shape[1] * 16 + 1, 2 ** 31 - 1):
        out = g.gdn_attn_decode_step(q, cache, table, ints([40, kv]), 0.1)
        with pytest.raises(g.GdnError):
            g.gdn_check_device_errors()
        assert torch.equal(out[0], good[0])
    for cu in ([0, 3, 2], [0, -1, 2], [0, 1, 7]):
        g.gdn_attn_prefill(q, cache, table, ints([40, 40]), ints(cu), 0.1)
        with pytest.raises(g.GdnError):
            g.gdn_check_device_errors()
    g.gdn_check_device_errors()


def test_captured_and_replayed_with_other_lengths():
    """One captured decode step replayed as the sequences grow, as a server does."""
    g = lib()
    gen = torch.Generator(device=DEV).manual_seed(0)
    B, hq, hkv, D = 5, 8, 2, 256
    longest = [900, 40, 3000, 0, 128]
    cache, table = make_cache(g, gen, [1] * B, longest, hkv, 64, D, True)
    q = torch.randn(B, hq, D, generator=gen, device=DEV).bfloat16()
    kv = ints([1, 1, 1, 0, 1])  # the fourth slot is unused: it has no page
    out = torch.empty_like(q)
    ws = torch.empty(g.gdn_attn_workspace_size(hq, hkv, D), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g.gdn_attn_decode_step(q, cache, table, kv, 0.07, out=out, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.gdn_attn_decode_step(q, cache, table, kv, 0.07, out=out, workspace=ws)
    for lens in ([1, 1, 1, 0, 1], longest, [33, 40, 129, 0, 65]):
        kv.copy_(ints(lens))
        graph.replay()
        g.gdn_check_device_errors()
        want, tol = attention(q, cache, table, [1] * B, lens, 0.07)
        assert_within(out, want, tol, "replayed")


def test_on_two_streams_at_once():
    g = lib()
    gen = torch.Generator(device=DEV).manual_seed(0)
    cases = []
    for i in range(2):
        cache, table = make_cache(g, gen, [200, 9], [1000, 4000], 2, 32, 128, bool(i))
        cases.append((cache, table, torch.randn(209, 8, 128, generator=gen, device=DEV).bfloat16(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        for cache, table, q, st in cases:
            with torch.cuda.stream(st):
                outs.append(g.gdn_attn_prefill(q, cache, table, ints([1000, 4000]), ints([0, 200, 209]), 0.08))
    torch.cuda.synchronize()
    g.gdn_check_device_errors()
    for i, (cache, table, q, _) in enumerate(cases):
        want, tol = attention(q, cache, table, [200, 9], [1000, 4000], 0.08)
        for o in outs[i::2]:
            assert_within(o, want, tol, "stream")


@pytest.mark.parametrize("e4m3", [False, True])
def test_a_layer_as_a_server_runs_it(e4m3):
    """A prompt in two chunks, then decode steps, beside a second sequence: every output against the
    whole sequence's attention from the cache that the calls left."""
    g = lib()
    gen = torch.Generator(device=DEV).manual_seed(0)
    hq, hkv, D, page = 16, 2, 256, 64
    cache, table = make_cache(g, gen, [0, 0], [400, 260], hkv, page, D, e4m3, fill=False)
    wq, wk = (1 + 0.1 * torch.randn(2, D, generator=gen, device=DEV)).bfloat16()
    freqs, mag = g.gdn_attn_rope_frequencies(64, 1e7)
    freqs = freqs.to(DEV)
    done = [0, 0]
    for step, q_lens in enumerate([[150, 5], [100, 250], [1, 1], [1, 1], [1, 1]]):
        T = sum(q_lens)
        done = [a + b for a, b in zip(done, q_lens)]
        proj = torch.randn(T, hq + 2 * hkv, D, generator=gen, device=DEV).bfloat16()
        z = torch.randn(T, hq, D, generator=gen, device=DEV).bfloat16()
        q, k, v = proj.split([hq, hkv, hkv], dim=1)
        cu = None if step >= 2 else cu_of(q_lens)
        qr = g.gdn_attn_prepare(q, k, v, cache, table, ints(done), cu, wq, wk, freqs, rope_scale=mag)
        if cu is None:
            out = g.gdn_attn_decode_step(qr, cache, table, ints(done), D ** -0.5, z=z)
        else:
            out = g.gdn_attn_prefill(qr, cache, table, ints(done), cu, D ** -0.5, z=z)
        want, tol = attention(qr, cache, table, q_lens, done, D ** -0.5, z)
        assert_within(out, want, tol, f"step {step}")
    g.gdn_check_device_errors()


def test_far_positions_and_strides():
    """The rotation at positions beyond 2^24, keys and values with their own strides."""
    g = lib()
    gen = torch.Generator(device=DEV).manual_seed(0)
    D, far = 128, 30_000_000
    freqs = g.gdn_attn_rope_frequencies(D, 1e6)[0].to(DEV)
    table = torch.full((1, far // 128 + 2), -1, dtype=torch.int32, device=DEV)
    table[0, far // 128:] = ints([0, 1])
    cache = g.KVCache.allocate(2, 1, 128, D)
    wide = torch.randn(4, 3, 2, D, generator=gen, device=DEV).bfloat16()
    q, k, v = wide[:, :, 1], wide[:, 1:2, 0], wide[:, 2:, 0]
    out = g.gdn_attn_prepare(q, k, v, cache, table, ints([far + 4]), ints([0, 4]), rope_freqs=freqs)
    g.gdn_check_device_errors()
    want, size = norm_rotate(q, None, [far + i for i in range(4)], freqs, False, 1.0, EPS)
    assert_within(out, want, 2.0 ** -8 * want.abs() + 2.0 ** -14 * size, "q")
    at = far % 128
    assert torch.equal(cache.v[0, 0, at:at + 4], v[:, 0])
