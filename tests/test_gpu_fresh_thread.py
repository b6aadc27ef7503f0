"""Calls whose first CUDA work on their host thread is the call itself (a thread pool's worker, with outputs and
workspaces made elsewhere): tensor maps are encoded before the first launch there."""
from __future__ import annotations

import threading

import pytest
import torch

from linear_attention_ssm_gb300.synth import prefill_inputs
from tests.gpu_common import DEV, lib
from tests.test_gpu_attn import cu_of, ints, make_cache
from tests.test_gpu_attn_edges import randn

pytestmark = pytest.mark.gpu


def on_a_fresh_thread(fn):
    """fn's result, from a thread that has done nothing before."""
    box = []

    def work():
        try:
            box.append(fn())
        except BaseException as e:  # handed on
            box.append(e)
    t = threading.Thread(target=work)
    t.start()
    t.join()
    if isinstance(box[0], BaseException):
        raise box[0]
    return box[0]


@pytest.mark.parametrize("hq,D,e4m3", [(8, 128, False), (8, 256, True), (40, 128, True)])
def test_attention(hq, D, e4m3):
    g = lib()
    gen = torch.Generator(device=DEV).manual_seed(40)
    cache, table = make_cache(g, gen, [9], [400], 2, 32, D, e4m3)
    q, out = randn(gen, 9, hq, D), torch.empty(9, hq, D, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(g.gdn_attn_workspace_size(hq, 2, D), dtype=torch.uint8, device=DEV)
    kv, cu, one, stream = ints([400]), cu_of([9]), q[8:].clone(), torch.cuda.current_stream()
    want = g.gdn_attn_prefill(q, cache, table, kv, cu, 0.1)
    last = g.gdn_attn_decode_step(one, cache, table, kv, 0.1)
    torch.cuda.synchronize()
    on_a_fresh_thread(lambda: g.gdn_attn_prefill(q, cache, table, kv, cu, 0.1, out=out, workspace=ws, stream=stream))
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    on_a_fresh_thread(lambda: g.gdn_attn_decode_step(one, cache, table, kv, 0.1, out=out[:1], workspace=ws, stream=stream))
    torch.cuda.synchronize()
    g.gdn_check_device_errors()
    assert torch.equal(out[:1], last)


def test_conv_and_chunk_prefill():
    g = lib()
    inp = prefill_inputs([130, 64, 7], seed=41)
    d = {k: v.to(DEV) for k, v in inp.items() if torch.is_tensor(v)}
    y, out = torch.empty_like(d["x"]), torch.empty_like(d["z"])
    want_y = g.gdn_conv1d_prefill(d["x"], d["conv_w"], d["cu_seqlens"])
    T = d["x"].shape[0]
    args = (want_y, d["g"], d["beta"], d["cu_seqlens"], inp["q_scale"])
    want = g.gdn_chunk_prefill(*args, z=d["z"], norm_w=d["norm_w"])
    ws = torch.empty(g.gdn_chunk_prefill_workspace_size(3, T), dtype=torch.uint8, device=DEV)
    stream = torch.cuda.current_stream()
    torch.cuda.synchronize()
    on_a_fresh_thread(lambda: g.gdn_conv1d_prefill(d["x"], d["conv_w"], d["cu_seqlens"], y=y, stream=stream))
    on_a_fresh_thread(lambda: g.gdn_chunk_prefill(*args, z=d["z"], norm_w=d["norm_w"], out=out, workspace=ws, stream=stream))
    torch.cuda.synchronize()
    g.gdn_check_device_errors()
    assert torch.equal(y, want_y) and torch.equal(out, want)
