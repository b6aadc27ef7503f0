"""The attention calls' own memory on streams of every kind: the per-thread default stream in several threads, side
streams, streams given by handle, and the release of what is kept."""
from __future__ import annotations

import concurrent.futures

import pytest
import torch

from tests.attn_reference import DEV, assert_within, attention
from tests.gpu_common import lib
from tests.test_gpu_attn import cu_of, ints, make_cache
from tests.test_gpu_attn_edges import randn

pytestmark = pytest.mark.gpu
PER_THREAD = 2  # cudaStreamPerThread


@pytest.mark.parametrize("given", [False, True])
def test_threads_on_their_per_thread_streams(given):
    """One handle, a queue in each thread: calls that run at the same time have memory of their own."""
    g = lib()
    gen = torch.Generator(device=DEV).manual_seed(30)
    hq, hkv, D, page = 16, 2, 256, 64
    cases = []
    for i, (q_lens, kv_lens) in enumerate([([40, 3], [5000, 900]), ([43], [7000]), ([20, 23], [300, 9000])]):
        cache, table = make_cache(g, gen, q_lens, kv_lens, hkv, page, D, bool(i & 1))
        cases.append((cache, table, randn(gen, 43, hq, D), q_lens, kv_lens, ints(kv_lens), cu_of(q_lens)))
    torch.cuda.synchronize()

    def work(i):
        cache, table, q, _, _, kv, cu = cases[i]
        mine = torch.cuda.ExternalStream(PER_THREAD)
        if given:
            outs = [g.gdn_attn_prefill(q, cache, table, kv, cu, 0.08, stream=PER_THREAD) for _ in range(40)]
        else:
            with torch.cuda.stream(mine):
                outs = [g.gdn_attn_prefill(q, cache, table, kv, cu, 0.08) for _ in range(40)]
        mine.synchronize()
        return outs
    with concurrent.futures.ThreadPoolExecutor(3) as pool:
        results = list(pool.map(work, range(3)))
    torch.cuda.synchronize()
    g.gdn_check_device_errors()
    for (cache, table, q, q_lens, kv_lens, *_), outs in zip(cases, results):
        want, tol = attention(q, cache, table, q_lens, kv_lens, 0.08)
        for o in outs:
            assert_within(o, want, tol, "thread")


def test_what_the_default_stream_keeps():
    """Calls on the default stream and on side streams in turn, with a release between them."""
    g = lib()
    from linear_attention_ssm_gb300 import binding
    gen = torch.Generator(device=DEV).manual_seed(31)
    cache, table = make_cache(g, gen, [30], [3000], 2, 32, 128, False)
    q, kv, cu = randn(gen, 30, 8, 128), ints([3000]), ints([0, 30])
    want, tol = attention(q, cache, table, [30], [3000], 0.08)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g.gdn_attn_release_workspaces()
    outs = []
    for i in range(6):
        outs.append(g.gdn_attn_prefill(q, cache, table, kv, cu, 0.08))
        with torch.cuda.stream(side):
            outs.append(g.gdn_attn_prefill(q, cache, table, kv, cu, 0.08))
            outs.append(g.gdn_attn_prefill(q, cache, table, kv, cu, 0.08, stream=0))
        if i == 3:
            g.gdn_attn_release_workspaces()
            torch.empty(g.gdn_attn_workspace_size(8, 2, 128), dtype=torch.uint8, device=DEV).fill_(255)
        assert list(binding._kept_workspaces) == ([0] if i != 3 else [])
    torch.cuda.synchronize()
    g.gdn_check_device_errors()
    for o in outs:
        assert_within(o, want, tol, "attention")
