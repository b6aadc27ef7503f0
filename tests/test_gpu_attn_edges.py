"""The paged-cache attention layer where a call can go wrong: values that are not finite in rows behind the
last key, outputs on 16-byte boundaries, more sequences than a CTA has threads, pools beyond 2^32 bytes,
shared pages, a stream given by the caller, empty batches, a graph of several calls."""
from __future__ import annotations

import concurrent.futures
import math

import pytest
import torch

from tests.attn_reference import DEV, assert_within, attention, dense_rows
from tests.gpu_common import lib
from tests.test_gpu_attn import cu_of, ints, make_cache

pytestmark = pytest.mark.gpu


def randn(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV).bfloat16()


def call(g, q, cache, table, q_lens, kv_lens, scale, **kw):
    if all(x == 1 for x in q_lens):
        return g.gdn_attn_decode_step(q, cache, table, ints(kv_lens), scale, **kw)
    return g.gdn_attn_prefill(q, cache, table, ints(kv_lens), cu_of(q_lens), scale, **kw)


def poison(cache, table, kv_lens, page):
    """Every row that no position of a sequence has: NaN codes, infinities and NaN in turn; scale bytes at both ends."""
    used = torch.zeros(cache.k.shape[0], page, dtype=torch.bool, device=DEV)
    for n, kv in enumerate(kv_lens):
        pos = torch.arange(kv, device=DEV)
        used[table[n, pos // page].long(), pos % page] = True
    free = ~used[:, None, :].expand(-1, cache.k.shape[1], -1)
    if cache.k_scale is not None:
        for x, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
            x.view(torch.uint8)[free] = 0x7F
            s[free] = 254
            s[..., 1::2][free[..., 1::2]] = 10
    else:
        for x in (cache.k, cache.v):
            x[free] = math.nan
            x[..., 1::2, :][free[..., 1::2]] = math.inf


@pytest.mark.parametrize("q_lens,kv_lens", [([40, 3], [200, 77]), ([200], [1100]), ([1, 1, 1], [130, 1, 64]), ([1] * 5, [33] * 5)])
@pytest.mark.parametrize("hq,hkv,D,page,e4m3", [(8, 2, 128, 16, False), (8, 2, 128, 128, True), (8, 1, 256, 64, False),
                                                (8, 1, 256, 32, True), (24, 1, 256, 16, False), (24, 1, 128, 64, True)])
def test_rows_behind_the_last_key_may_hold_anything(q_lens, kv_lens, hq, hkv, D, page, e4m3):
    g = lib()
    gen = torch.Generator(device=DEV).manual_seed(2)
    cache, table = make_cache(g, gen, q_lens, kv_lens, hkv, page, D, e4m3)
    poison(cache, table, kv_lens, page)
    q = randn(gen, sum(q_lens), hq, D)
    out = call(g, q, cache, table, q_lens, kv_lens, D ** -0.5)
    g.gdn_check_device_errors()
    assert bool(torch.isfinite(out).all())
    want, tol = attention(q, cache, table, q_lens, kv_lens, D ** -0.5)
    assert_within(out, want, tol, "attention")


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1], [100, 900]), ([30, 2], [700, 5]), ([150, 140], [150, 600])])
def test_outputs_and_gates_on_16_byte_boundaries(q_lens, kv_lens, D, e4m3):
    g = lib()
    gen = torch.Generator(device=DEV).manual_seed(4)
    T, hq, hkv, page = sum(q_lens), 6, 2, 32
    cache, table = make_cache(g, gen, q_lens, kv_lens, hkv, page, D, e4m3)

    def odd(*shape):  # 16 bytes past a 32-byte boundary
        n = math.prod(shape)
        return torch.zeros(n + 24, dtype=torch.bfloat16, device=DEV)[8:8 + n].view(shape)
    q, z, out = odd(T, hq, D), odd(T, hq, D), odd(T, hq, D)
    assert out.data_ptr() % 32 == 16
    q.copy_(randn(gen, T, hq, D))
    z.copy_(randn(gen, T, hq, D))
    call(g, q, cache, table, q_lens, kv_lens, D ** -0.5, z=z, out=out)
    want, tol = attention(q, cache, table, q_lens, kv_lens, D ** -0.5, z)
    assert_within(out, want, tol, "attention")
    k, v = odd(T, hkv, D), odd(T, hkv, D)
    g.gdn_attn_cache_read(cache, table, cu_of(q_lens), k, v)
    g.gdn_check_device_errors()
    lo = 0
    for n, ql in enumerate(q_lens):
        dk, dv = dense_rows(cache, table[n], ql)
        assert torch.equal(k[lo:lo + ql], dk.transpose(0, 1).bfloat16()) and torch.equal(v[lo:lo + ql], dv.transpose(0, 1).bfloat16())
        lo += ql


@pytest.mark.parametrize("hq,hkv,D,e4m3", [(4, 2, 128, False), (4, 2, 128, True), (8, 1, 256, False), (20, 1, 256, True)])
@pytest.mark.parametrize("decode", [False, True])
def test_more_sequences_than_threads(hq, hkv, D, e4m3, decode):
    g = lib()
    gen = torch.Generator(device=DEV).manual_seed(5)
    n, page = 1301, 16
    q_lens = [1] * n if decode else [(7 * i) % 4 for i in range(n)]
    kv_lens = [ql + (13 * i) % 150 for i, ql in enumerate(q_lens)]
    cache, table = make_cache(g, gen, q_lens, kv_lens, hkv, page, D, e4m3)
    q = randn(gen, sum(q_lens), hq, D)
    out = call(g, q, cache, table, q_lens, kv_lens, D ** -0.5)
    g.gdn_check_device_errors()
    want, tol = attention(q, cache, table, q_lens, kv_lens, D ** -0.5)
    assert_within(out, want, tol, "attention")


@pytest.mark.parametrize("e4m3", [False, True])
def test_a_pool_beyond_4_gib(e4m3):
    """The pages used are the last ones of a pool whose offsets pass 32 bits."""
    g = lib()
    gen = torch.Generator(device=DEV).manual_seed(6)
    hq, hkv, D, page = 8, 2, 256, 128
    pages = (5 << 30) // (hkv * page * D * (1 if e4m3 else 2))
    cache = g.KVCache.allocate(pages, hkv, page, D, torch.float8_e4m3fn if e4m3 else torch.bfloat16)
    q_lens, kv_lens = [60, 40], [300, 50]
    table = torch.tensor([[pages - 1, pages - 3, 2], [pages - 2, 0, 0]], dtype=torch.int32, device=DEV)
    freqs = g.gdn_attn_rope_frequencies(64, 1e6)[0].to(DEV)
    keys = randn(gen, sum(kv_lens), hkv, D)
    g.gdn_attn_prepare(None, keys, keys, cache, table, ints(kv_lens), cu_of(kv_lens), rope_freqs=freqs)
    q = randn(gen, sum(q_lens), hq, D)
    out = g.gdn_attn_prefill(q, cache, table, ints(kv_lens), cu_of(q_lens), D ** -0.5)
    one = g.gdn_attn_decode_step(q[[59, 99]].contiguous(), cache, table, ints(kv_lens), D ** -0.5)
    k, v = (torch.empty(300, hkv, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    g.gdn_attn_cache_read(cache, table[:1].contiguous(), ints([0, 300]), k, v)
    g.gdn_check_device_errors()
    want, tol = attention(q, cache, table, q_lens, kv_lens, D ** -0.5)
    assert_within(out, want, tol, "prefill")
    assert_within(one, want[[59, 99]], tol[[59, 99]], "decode")
    dk, dv = dense_rows(cache, table[0], 300)
    assert torch.equal(k, dk.transpose(0, 1).bfloat16()) and torch.equal(v, dv.transpose(0, 1).bfloat16())
    if not e4m3:
        assert torch.equal(v, keys[:300])


def test_sequences_that_share_pages():
    """A prefix that three sequences read from the same pages, each with pages of its own behind it."""
    g = lib()
    gen = torch.Generator(device=DEV).manual_seed(7)
    hq, hkv, D, page = 8, 2, 128, 32
    cache, table = make_cache(g, gen, [5, 60, 1], [500, 500, 500], hkv, page, D, False)
    table[1:, :10] = table[0, :10]
    q = randn(gen, 66, hq, D)
    out = g.gdn_attn_prefill(q, cache, table, ints([500, 500, 500]), ints([0, 5, 65, 66]), 0.1)
    g.gdn_check_device_errors()
    want, tol = attention(q, cache, table, [5, 60, 1], [500, 500, 500], 0.1)
    assert_within(out, want, tol, "attention")


def test_the_callers_stream_and_memory_of_its_own():
    """stream= another than the current one: the memory that a call takes belongs to that stream, so that work
    queued on the current one cannot have it too."""
    g = lib()
    gen = torch.Generator(device=DEV).manual_seed(8)
    hq, hkv, D, page = 8, 2, 256, 64
    cache, table = make_cache(g, gen, [300], [5000], hkv, page, D, True)
    q = randn(gen, 300, hq, D)
    want, tol = attention(q, cache, table, [300], [5000], 0.06)
    kv, cu = ints([5000]), ints([0, 300])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        outs = []
        for _ in range(4):
            outs.append(g.gdn_attn_prefill(q, cache, table, kv, cu, 0.06, stream=stream))
            for _ in range(3):  # what the allocator gives the current stream is written at once
                torch.empty(g.gdn_attn_workspace_size(hq, hkv, D), dtype=torch.uint8, device=DEV).fill_(255)
        torch.cuda.synchronize()
        g.gdn_check_device_errors()
        for o in outs:
            assert_within(o, want, tol, "attention")


def test_empty_batches():
    g = lib()
    cache = g.KVCache.allocate(4, 2, 16, 128)
    q, kv = torch.empty(0, 4, 128, dtype=torch.bfloat16, device=DEV), torch.empty(0, 2, 128, dtype=torch.bfloat16, device=DEV)
    for n in (0, 3):
        table, lens, cu = torch.zeros(n, 2, dtype=torch.int32, device=DEV), ints([0] * n), ints([0] * (n + 1))
        assert g.gdn_attn_prefill(q, cache, table, lens, cu, 0.1).shape == q.shape
        assert g.gdn_attn_prepare(q, kv, kv, cache, table, lens, cu).shape == q.shape
        g.gdn_attn_cache_read(cache, table, cu, kv, kv.clone())
    none = torch.zeros(0, 2, dtype=torch.int32, device=DEV)
    assert g.gdn_attn_decode_step(q, cache, none, ints([]), 0.1).shape == q.shape
    torch.cuda.synchronize()
    g.gdn_check_device_errors()


def test_a_captured_layer_advances_by_itself():
    """prepare, decode and the lengths' increment in one graph, replayed: each replay is the next position."""
    g = lib()
    gen = torch.Generator(device=DEV).manual_seed(9)
    hq, hkv, D, page, n = 8, 2, 128, 16, 3
    kv0 = [15, 40, 1]
    cache, table = make_cache(g, gen, [1] * n, [x + 20 for x in kv0], hkv, page, D, False)
    q, k, v = randn(gen, n, hq, D), randn(gen, n, hkv, D), randn(gen, n, hkv, D)
    freqs = g.gdn_attn_rope_frequencies(D, 1e4)[0].to(DEV)
    lens = ints(kv0)
    ws = torch.empty(g.gdn_attn_workspace_size(hq, hkv, D), dtype=torch.uint8, device=DEV)
    qr, out = torch.empty_like(q), torch.empty_like(q)

    def step():
        lens.add_(1)
        g.gdn_attn_prepare(q, k, v, cache, table, lens, None, rope_freqs=freqs, q_out=qr)
        g.gdn_attn_decode_step(qr, cache, table, lens, 0.09, out=out, workspace=ws)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(2, 8):
        q.copy_(randn(gen, n, hq, D))
        k.copy_(randn(gen, n, hkv, D))
        graph.replay()
        torch.cuda.synchronize()
        now = [x + i for x in kv0]
        assert lens.tolist() == now
        want, tol = attention(qr, cache, table, [1] * n, now, 0.09)
        assert_within(out, want, tol, f"replay {i}")
    g.gdn_check_device_errors()


def test_a_captured_step_on_two_branches():
    """Queries from one branch of a graph, keys and values from another (the attention's first kernel has two
    predecessors there, one of them a copy), replayed with new inputs."""
    g = lib()
    gen = torch.Generator(device=DEV).manual_seed(10)
    hq, hkv, D, page, kv = 8, 2, 256, 32, [300, 7]
    cache, table = make_cache(g, gen, [1, 1], kv, hkv, page, D, True)
    q, k, v = randn(gen, 2, hq, D), randn(gen, 2, hkv, D), randn(gen, 2, hkv, D)
    qin, qs, out = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
    dense = [torch.empty(4, hkv, D, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    lens, cu, starts = ints(kv), ints([0, 2, 4]), ints([100, 3])
    ws = torch.empty(g.gdn_attn_workspace_size(hq, hkv, D), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()

    def step():
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            qs.copy_(q)
            g.gdn_attn_cache_read(cache, table, cu, *dense, starts=starts)
        g.gdn_attn_prepare(None, k, v, cache, table, lens)
        qin.copy_(q)
        here.wait_stream(side)
        g.gdn_attn_decode_step(qs, cache, table, lens, 0.06, out=out, workspace=ws)
    first = torch.cuda.Stream()
    with torch.cuda.stream(first):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(5):
        for x in (q, k, v):
            x.copy_(randn(gen, *x.shape))
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        want, tol = attention(q, cache, table, [1, 1], kv, 0.06)
        assert_within(out, want, tol, f"replay {i}")
    assert torch.equal(dense[0][:2], dense_rows(cache, table[0], 102)[0][:, 100:].transpose(0, 1).bfloat16())
    g.gdn_check_device_errors()


def test_threads_that_share_a_stream():
    """Calls from several threads on one stream, whose kernels interleave there: no call works in another's memory."""
    g = lib()
    gen = torch.Generator(device=DEV).manual_seed(11)
    hq, hkv, D, page = 8, 2, 128, 32
    q_lens, kv_lens = [40, 3], [3000, 900]
    cases = []
    for i in range(4):
        cache, table = make_cache(g, gen, q_lens, kv_lens, hkv, page, D, bool(i & 1))
        cases.append((cache, table, randn(gen, 43, hq, D)))
    kv, cu = ints(kv_lens), cu_of(q_lens)
    torch.cuda.synchronize()

    def work(i):
        cache, table, q = cases[i]
        return [g.gdn_attn_prefill(q, cache, table, kv, cu, 0.08) for _ in range(30)]
    with concurrent.futures.ThreadPoolExecutor(4) as pool:
        outs = list(pool.map(work, range(4)))
    torch.cuda.synchronize()
    g.gdn_check_device_errors()
    for (cache, table, q), got in zip(cases, outs):
        want, tol = attention(q, cache, table, q_lens, kv_lens, 0.08)
        for o in got:
            assert_within(o, want, tol, "thread")


def test_two_graphs_replayed_at_once():
    """Graphs captured without a workspace of the caller's have one each."""
    g = lib()
    gen = torch.Generator(device=DEV).manual_seed(12)
    hq, hkv, D, page = 16, 2, 256, 64
    q_lens, kv_lens = [50], [6000]
    graphs = []
    for i in range(2):
        cache, table = make_cache(g, gen, q_lens, kv_lens, hkv, page, D, False)
        q, out = randn(gen, 50, hq, D), torch.empty(50, hq, D, dtype=torch.bfloat16, device=DEV)
        kv, cu = ints(kv_lens), cu_of(q_lens)
        g.gdn_attn_prefill(q, cache, table, kv, cu, 0.06, out=out)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            g.gdn_attn_prefill(q, cache, table, kv, cu, 0.06, out=out)
        graphs.append((graph, torch.cuda.Stream(), cache, table, q, out, kv, cu))
    for _ in range(10):
        for graph, stream, *_ in graphs:
            with torch.cuda.stream(stream):
                graph.replay()
        g.gdn_attn_prefill(*[graphs[0][i] for i in (4, 2, 3, 6, 7)], 0.06)  # and a call beside them
    torch.cuda.synchronize()
    g.gdn_check_device_errors()
    for _, _, cache, table, q, out, *_ in graphs:
        want, tol = attention(q, cache, table, q_lens, kv_lens, 0.06)
        assert_within(out, want, tol, "graph")
