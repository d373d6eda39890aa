"""Memory for what a caller does not give: results and workspaces of a call."""
from __future__ import annotations

import torch


def empty(stream, shape, dtype, device):
    """Memory that a call on ``stream`` (None: the current one) writes.  It comes
    from that stream's share of the allocator: a block of the current stream's
    could still be in use there, and nothing orders ``stream`` behind that use."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def zeros(stream, shape, dtype, device):
    """... zeroed in that stream's order."""
    if stream is None:
        return torch.zeros(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.zeros(shape, dtype=dtype, device=device)


def result(stream, shape, dtype, device):
    """As ``empty``, for what the caller's current stream goes on with: it is not handed out
    again while work queued there by the time it is freed may still read it."""
    t = empty(stream, shape, dtype, device)
    if stream is not None and t.is_cuda:
        t.record_stream(torch.cuda.current_stream(t.device))
    return t
