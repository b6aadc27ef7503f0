"""A workspace given to a binding is memory of its own, as many bytes as its elements: without a GPU, the calls are
stand-ins that say what they were given."""
from __future__ import annotations

import types

import pytest
import torch

from linear_attention_ssm_gb300 import binding

CPU = torch.device("cpu")


@pytest.fixture
def calls(monkeypatch):
    given = []
    monkeypatch.setattr(binding, "_L", lambda: types.SimpleNamespace(
        gdn_attn_workspace_size=lambda geo: 64, gdn_attn_decode_step=None, gdn_attn_prefill=None,
        gdn_moe_workspace_size=lambda *a: 64, gdn_moe_step=None, gdn_moe_step_routed=None))
    monkeypatch.setattr(binding, "_cache_arg", lambda cache: (None, 2, 128, CPU))
    monkeypatch.setattr(binding, "_rows_of", lambda t, name: (1, 4))
    monkeypatch.setattr(binding, "_flat", lambda *a: 0)
    monkeypatch.setattr(binding, "_matrix", lambda *a: (0, 0))
    monkeypatch.setattr(binding, "_batch_args", lambda *a: (1, 0, 0, None, 1))
    monkeypatch.setattr(binding, "_call", lambda fn, dev, stream, *args: given.append(args[-2:]))
    experts = types.SimpleNamespace(_device=CPU, _geo=types.SimpleNamespace(hidden=16), _weights=None, router=object())
    x = torch.zeros(2, 16, dtype=torch.bfloat16)

    def attention(workspace):
        binding._attention(None, None, None, None, None, 0.1, None, torch.zeros(1), workspace, None)

    def layer(workspace):
        binding.gdn_moe_step(x, experts, 2, out=x, workspace=workspace)

    def routed(workspace):
        binding.gdn_moe_step_routed(x, experts, torch.zeros(2, 2, dtype=torch.int32), x, out=x, workspace=workspace)
    return {"attention": attention, "layer": layer, "routed": routed}, given


@pytest.mark.parametrize("name", ["attention", "layer", "routed"])
def test_a_workspace_is_contiguous_memory(calls, name):
    call, given = calls[0][name], calls[1]
    room = torch.empty(256, dtype=torch.uint8)
    for t in (room, room[64:192], room.view(4, 64), room.view(torch.float32)):
        call(t)
        assert given.pop() == (t.data_ptr(), t.numel() * t.element_size())
    for t in (room[::2], room[:64].expand(4, 64), room.view(4, 64).t(), room.view(4, 64)[:, :32]):
        with pytest.raises(ValueError):
            call(t)
    with pytest.raises(ValueError):
        call(torch.empty(256, dtype=torch.uint8, device="meta"))
    with pytest.raises(TypeError):
        call(b"256")
    assert not given


class _Library:
    """Every workspace is of 64 bytes, every call succeeds."""
    def __init__(self, given):
        self.given = given

    def __getattr__(self, name):
        if name.endswith("workspace_size"):
            return lambda *a: 64
        return lambda *a: self.given.append(a[-3:-1])


@pytest.mark.parametrize("name", ["gdn_chunk_prefill", "gdn_kda_chunk_prefill", "gdn_chunk_prefill_fused_gates", "gdn_prefill",
                                  "gdn_kda_prefill"])
def test_the_prefills_workspaces_too(monkeypatch, name):
    given = []
    monkeypatch.setattr(binding, "_L", lambda: _Library(given))
    monkeypatch.setattr(binding, "_dev", lambda t, *a, **kw: t)
    monkeypatch.setattr(binding, "_stream", lambda stream: None)
    monkeypatch.setattr(binding, "_check", lambda status: None)
    monkeypatch.setattr(binding, "_p", lambda t: None if t is None else t.data_ptr())
    x, cu = torch.zeros(2, 16, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    args = {"gdn_chunk_prefill": (x, None, None, cu, 0.1), "gdn_kda_chunk_prefill": (x, None, None, cu, 0.1),
            "gdn_chunk_prefill_fused_gates": (x, None, None, None, None, cu, 0.1),
            "gdn_prefill": (x, None, cu, None, None, None, None, 0.1), "gdn_kda_prefill": (x, None, cu, None, None, None, None, 0.1)}

    def call(workspace):
        getattr(binding, name)(*args[name], workspace=workspace)
    room = torch.empty(256, dtype=torch.uint8)
    for t in (room, room.view(torch.float32)):
        call(t)
        assert given.pop() == (t.data_ptr(), 256)
    call(None)
    assert given.pop()[1] == 64
    for t in (room[::2], room[:64].expand(4, 64), torch.empty(256, dtype=torch.uint8, device="meta")):
        with pytest.raises(ValueError):
            call(t)
    assert not given
