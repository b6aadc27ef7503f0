"""The attention binding's workspaces, without a GPU: the library and the stream's handle are stand-ins, so that
each call says which memory it was given."""
from __future__ import annotations

import types

import pytest
import torch

from linear_attention_ssm_gb300 import binding

NEED = 4096


@pytest.fixture
def calls(monkeypatch):
    """A stand-in for the GPU; .handle is the current stream's, .used the memory of every call, kept alive."""
    state = types.SimpleNamespace(handle=0, used=[], device=torch.device("cuda", 0))

    def memory(shape, dtype, device=None, stream=None):
        state.used.append(torch.empty(shape, dtype=dtype))
        return state.used[-1]
    lib = types.SimpleNamespace(gdn_attn_workspace_size=lambda geo: NEED, gdn_attn_decode_step=None, gdn_attn_prefill=None)
    monkeypatch.setattr(binding, "_L", lambda: lib)
    monkeypatch.setattr(binding, "_raw_stream", lambda index: state.handle)
    monkeypatch.setattr(binding, "_cache_arg", lambda cache: (None, 2, 128, state.device))
    monkeypatch.setattr(binding, "_rows_of", lambda t, name: (1, 4))
    monkeypatch.setattr(binding, "_flat", lambda *a: 0)
    monkeypatch.setattr(binding, "_batch_args", lambda *a: (1, 0, 0, None, 1))
    monkeypatch.setattr(binding, "_empty", memory)
    monkeypatch.setattr(binding.torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(binding.torch.cuda, "is_current_stream_capturing", lambda: False)
    real_empty = torch.empty

    def empty(*a, device=None, **kw):
        t = real_empty(*a, **kw)
        if device is not None:
            state.used.append(t)
        return t
    monkeypatch.setattr(binding.torch, "empty", empty)
    given = []
    monkeypatch.setattr(binding, "_call", lambda fn, dev, stream, *args: given.append(args[-2]))  # (workspace, bytes)
    state.given = given
    for name in ("_kept_workspaces", "_spare_workspaces"):
        if hasattr(binding, name):
            getattr(binding, name).clear()
    yield state
    for name in ("_kept_workspaces", "_spare_workspaces"):
        if hasattr(binding, name):
            getattr(binding, name).clear()


def step(state, handle, stream=None):
    state.handle = handle
    binding._attention(None, None, None, None, None, 0.1, None, torch.zeros(1), None, stream)
    return state.given[-1]


@pytest.mark.parametrize("handle", [2, 0x7F12345600])
def test_only_the_default_stream_keeps_a_workspace(calls, handle):
    """The per-thread stream has one handle and a queue in each thread; another stream's handle may come back as a
    new stream's after it is destroyed: their calls never get the memory of an earlier one."""
    assert step(calls, handle) != step(calls, handle)
    assert step(calls, 0, stream=handle) != step(calls, 0, stream=handle)
    first = step(calls, 0)
    assert step(calls, handle) != first
    assert step(calls, 0) == first and step(calls, 0, stream=0) == first
    assert step(calls, handle, stream=0) == first


def test_what_is_kept_is_one_workspace_and_can_be_released(calls):
    for handle in range(0x1000, 0x9000, 0x100):
        step(calls, handle)
    step(calls, 0)
    assert sum(w.numel() for w in binding._kept_workspaces.values()) == NEED
    first = step(calls, 0)
    binding.gdn_attn_release_workspaces()
    assert not binding._kept_workspaces
    assert step(calls, 0) != first
