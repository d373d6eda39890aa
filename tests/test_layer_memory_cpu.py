"""Where the layer calls take the memory that their callers do not give, with the
allocator and the native calls replaced by recorders (no GPU)."""
from __future__ import annotations

import contextlib
import types

import pytest
import torch

from mamba2_ssm_decode_gb300 import layer_api as api

X, I32 = torch.zeros(6, 32), torch.zeros(3, dtype=torch.int32)
CALLS = {
    "conv_update": lambda **kw: api.conv_update(None, X, None, **kw),
    "conv_update_varlen": lambda **kw: api.conv_update_varlen(None, X, None, **kw),
    "conv_fwd_varlen": lambda **kw: api.conv_fwd_varlen(X, None, I32, **kw),
    "scan_update": lambda **kw: api.scan_update(None, X, X, None, X, X, **kw),
    "scan_update_varlen": lambda **kw: api.scan_update_varlen(None, X, X, None, X, X, **kw),
    "scan_fwd_varlen": lambda **kw: api.scan_fwd_varlen(X, X, None, X, X, I32, **kw),
    "slots_compact": lambda **kw: api.slots_compact([X], I32, **kw),
    "slots_compact, in place": lambda **kw: api.slots_compact([X], I32, out=I32, **kw),
}


@pytest.fixture
def streams(monkeypatch):
    """The stream that is current at each allocation of a call."""
    current, seen, empty = [None], [], torch.empty

    @contextlib.contextmanager
    def use(stream):
        before, current[0] = current[0], stream
        yield
        current[0] = before

    def recorded(*a, **kw):
        seen.append(current[0])
        return empty(*a, **kw)

    nothing = lambda *a: None  # noqa: E731
    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch, "empty", recorded)
    monkeypatch.setattr(torch, "empty_like", lambda t, **kw: recorded(t.shape, dtype=t.dtype, **kw))
    monkeypatch.setattr(torch.Tensor, "record_stream", nothing)
    monkeypatch.setattr(api, "slots_compact_workspace_bytes", lambda *a, **kw: 64)
    monkeypatch.setattr(api, "_module", types.SimpleNamespace(conv=nothing, scan=nothing,
                                                              slots_compact=nothing))
    return seen


@pytest.mark.parametrize("call", CALLS)
def test_memory_of_the_call_is_of_its_stream(call, streams):
    side = types.SimpleNamespace(cuda_stream=1)
    CALLS[call](stream=side)
    assert streams and all(s is side for s in streams)
    del streams[:]
    CALLS[call]()
    assert streams and all(s is None for s in streams)


def test_memory_of_the_older_calls_is_of_their_stream(streams, monkeypatch):
    """The state update, the checkpointing update with its zeroed scratch, and the
    SSD prefill with its workspace, up to the library's own call."""
    from mamba2_ssm_decode_gb300 import api as old

    zeros = torch.zeros
    monkeypatch.setattr(torch, "zeros", lambda *a, **kw: torch.empty(*a, **kw).zero_())
    monkeypatch.setattr(old, "_require_cuda", lambda *a: torch.device("cpu"))
    monkeypatch.setattr(old, "ssd_workspace_bytes", lambda *a, **kw: 64)

    class Library:
        def __getattr__(self, name):
            return lambda *a: 0

    monkeypatch.setattr(old._abi, "lib", Library)
    monkeypatch.setattr(old, "_stream", lambda dev, stream: None)
    S, H, P, N, G, R = 2, 2, 64, 64, 1, 4
    f = lambda *shape: zeros(*shape, dtype=torch.bfloat16)  # noqa: E731
    ints = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    state, x, dt, A = zeros(4, H, P, N), f(S, H, P), zeros(S, H), zeros(H)
    B = f(S, G, N)
    cu = ints(0, 1, 2)
    rows = [x, dt, A, B, B]
    calls = [lambda **kw: old.ssu_update(state, *rows, **kw),
             lambda **kw: old.ssu_update_varlen(state, *rows, cu_seqlens=cu, **kw),
             lambda **kw: old.ssu_replay_update(state, *rows, f(4, H, R, P), f(4, G, R, N),
                                                zeros(4, H, R), ints(0, 0, 0, 0), ints(0, 0, 0, 0), R,
                                                **kw),
             lambda **kw: old.ssd_combined_fwd_varlen(*rows, 64, cu, cu, ints(0, 1), ints(0, 1), **kw)]
    side = types.SimpleNamespace(cuda_stream=1)
    for call, most in zip(calls, (1, 1, 2, 3)):
        del streams[:]
        call(stream=side)
        assert len(streams) == most and all(s is side for s in streams)


def test_compaction_into_a_view_of_the_table_is_in_place(monkeypatch):
    """The workspace is the one that the library asks for, which compares addresses."""
    asked = []
    monkeypatch.setattr(api, "slots_compact_workspace_bytes",
                        lambda slots, n, in_place: asked.append(bool(in_place)) or 0)
    monkeypatch.setattr(api, "_module", types.SimpleNamespace(slots_compact=lambda *a: None))
    for out in (I32, I32.view(3), I32[:], torch.zeros_like(I32), None):
        api.slots_compact([X], I32, out=out)
    assert asked == [True, True, True, False, False]
