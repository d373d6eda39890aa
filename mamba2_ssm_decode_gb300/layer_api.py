"""Python binding of the calls around the state update (include/ssu.h): the
causal convolution, the selective scan with a full A, and the moves of slots.

Like ``api``: argument marshalling only.  Each function checks that its CUDA
tensors describe the layout the ABI expects (no hidden copies, no compute) and
calls the library on the current torch stream of the tensors' device.
ValueError for a rejected argument, NotImplementedError for a capability the
library does not implement, RuntimeError for a failed launch.
"""
from __future__ import annotations

import ctypes

import torch

from . import _abi
from .api import _FLOAT_DT, _float_dtype, _int_dtype, _ptr, _require_cuda, _stream, _table

_ACTIVATIONS = {None: 0, "none": 0, "silu": 1}


def _rows2(t, name, rows, dim):
    """Row stride of a [rows, dim] operand with unit dim stride."""
    if t.dim() != 2 or t.shape[0] != rows or t.shape[1] != dim:
        raise ValueError(f"{name} must be [{rows}, {dim}], got {tuple(t.shape)}")
    if dim > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must be contiguous along channels (stride 1), got {t.stride()}")
    return t.stride(0)


def _vector(t, name, n, dtype=None):
    """A contiguous [n] tensor."""
    if t.dim() != 1 or t.shape[0] != n:
        raise ValueError(f"{name} must be [{n}], got {tuple(t.shape)}")
    if n > 1 and t.stride(0) != 1:
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise NotImplementedError(f"{name} must be {dtype}, got {t.dtype}")


def _slot_vectors(src, dst, nseqs):
    """Common index dtype of the read and write slots of ``nseqs`` sequences."""
    idx = 0
    for name, t in (("state_batch_indices", src), ("dst_state_batch_indices", dst)):
        if t is not None:
            _vector(t, name, nseqs)
            d = _int_dtype(t, name)
            if idx and d != idx:
                raise ValueError("state_batch_indices and dst_state_batch_indices must share a dtype")
            idx = d
    return idx or _abi.SSU_I32


def _flags(t, nseqs):
    """has_initial_state: one byte per sequence."""
    if t is None:
        return None
    _vector(t, "has_initial_state", nseqs)
    if t.dtype not in (torch.bool, torch.uint8):
        raise ValueError(f"has_initial_state must be bool or uint8, got {t.dtype}")
    return ctypes.c_void_p(t.data_ptr())


def _no_overlap(out, *operands):
    for t in operands:
        if t is not None and t.numel() and t.data_ptr() == out.data_ptr():
            raise ValueError("out must not overlap an operand of a prompt call")


def _dense(t, name, rows):
    """The [rows, ...] view of a dense [batch, steps, ...] operand."""
    if t is None:
        return None
    if t.dim() < 3 or t.shape[0] * t.shape[1] != rows:
        raise ValueError(f"a dense x requires a dense {name} as well, got {tuple(t.shape)}")
    return t.view(rows, *t.shape[2:])


def _packed(nseqs, cu_seqlens, num_accepted_tokens, state_batch_indices,
            dst_state_batch_indices):
    """Sequences of a packed decode call: (nseqs, meta dtype, src, dst, index dtype)."""
    if nseqs is None:
        if cu_seqlens is not None:
            nseqs = cu_seqlens.numel() - 1
        elif num_accepted_tokens is not None:
            nseqs = num_accepted_tokens.numel()
        elif state_batch_indices is not None:
            nseqs = state_batch_indices.shape[0]
        elif dst_state_batch_indices is not None:
            nseqs = dst_state_batch_indices.shape[0]
        else:
            raise ValueError("a packed multi-token call must carry per-sequence metadata: "
                             "state_batch_indices, dst_state_batch_indices, "
                             "num_accepted_tokens or cu_seqlens")
    meta = 0
    if cu_seqlens is not None:
        _vector(cu_seqlens, "cu_seqlens", nseqs + 1)
        meta = _int_dtype(cu_seqlens, "cu_seqlens")
    if num_accepted_tokens is not None:
        _vector(num_accepted_tokens, "num_accepted_tokens", nseqs)
        d = _int_dtype(num_accepted_tokens, "num_accepted_tokens")
        if meta and d != meta:
            raise ValueError("cu_seqlens and num_accepted_tokens must share a dtype")
        meta = d
    src, sd = _table(state_batch_indices, "state_batch_indices")
    dst, dd = _table(dst_state_batch_indices, "dst_state_batch_indices")
    if sd and dd and sd != dd:
        raise ValueError("state_batch_indices and dst_state_batch_indices must share a dtype")
    for t, name in ((state_batch_indices, "state_batch_indices"),
                    (dst_state_batch_indices, "dst_state_batch_indices")):
        if t is not None and t.dim() == 2 and t.shape[0] < nseqs:
            raise ValueError(f"{name} must have a row for each of the {nseqs} sequences, got "
                             f"{tuple(t.shape)}")
    return nseqs, meta or _abi.SSU_I32, src, dst, sd or dd or _abi.SSU_I32


def _prompts(cu_seqlens):
    if cu_seqlens is None or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must hold the start of every sequence and the end of the last")
    n = cu_seqlens.numel() - 1
    _vector(cu_seqlens, "cu_seqlens", n + 1)
    return n, _int_dtype(cu_seqlens, "cu_seqlens")


# ---------------------------------------------------------------------------
# causal convolution
# ---------------------------------------------------------------------------

def _conv_params(conv_state, x, weight, bias, activation, disable_state_update, pad_slot_id, out):
    if x.dim() != 2:
        raise ValueError(f"x must be [rows, channels], got {tuple(x.shape)}")
    rows, C = x.shape
    io = _float_dtype(x, "x")
    if weight.dim() != 2 or weight.shape[0] != C:
        raise ValueError(f"weight must be [{C}, width], got {tuple(weight.shape)}")
    if not weight.is_contiguous():
        raise ValueError("weight must be contiguous")
    W = weight.shape[1]
    if weight.dtype not in (x.dtype, torch.float32):
        raise ValueError(f"weight must be {x.dtype} or fp32, got {weight.dtype}")
    if bias is not None:
        _vector(bias, "bias", C)
        if bias.dtype != weight.dtype:
            raise ValueError(f"bias must have weight's dtype ({weight.dtype}), got {bias.dtype}")
    if activation not in _ACTIVATIONS:
        raise ValueError(f"activation must be None or 'silu', got {activation!r}")
    p = _abi.ConvParams()
    if conv_state is not None:
        if conv_state.dim() != 3 or conv_state.shape[1] != W - 1 or conv_state.shape[2] != C:
            raise ValueError(f"conv_state must be [slots, {W - 1}, {C}], got "
                             f"{tuple(conv_state.shape)}")
        if conv_state.dtype != x.dtype:
            raise ValueError(f"conv_state must be {x.dtype}, got {conv_state.dtype}")
        if not conv_state.is_contiguous():
            raise ValueError("conv_state must be contiguous")
        p.conv_state, p.slots = conv_state.data_ptr(), conv_state.shape[0]
    p.channels, p.width, p.io_dtype = C, W, io
    p.x, p.x_row_stride = x.data_ptr(), x.stride(0)
    if out.dtype != x.dtype:
        raise ValueError(f"out must be {x.dtype}, got {out.dtype}")
    p.out, p.out_row_stride = out.data_ptr(), _rows2(out, "out", rows, C)
    if C > 1 and x.stride(1) != 1:
        raise ValueError(f"x must be contiguous along channels (stride 1), got {x.stride()}")
    p.weight, p.weight_dtype = weight.data_ptr(), _FLOAT_DT[weight.dtype]
    p.bias = bias.data_ptr() if bias is not None else None
    p.activation = _ACTIVATIONS[activation]
    p.disable_state_update = int(bool(disable_state_update))
    p.pad_slot_id = int(pad_slot_id)
    return p


def conv_update(conv_state, x, weight, bias=None, activation="silu", state_batch_indices=None,
                dst_state_batch_indices=None, pad_slot_id=-1, out=None,
                disable_state_update=False, stream=None):
    """One-token causal convolution (C ABI ``ssu_conv_update``).

    conv_state [slots, W - 1, C] (updated in place, x's dtype); x [batch, C]
    (fp32, bf16 or fp16; a column slice of a wider tensor is fine); weight
    [C, W] and bias [C] in x's dtype or fp32; W 2, 3 or 4; ``activation``
    "silu" or None.  Slot vectors [batch] int32/int64.  Returns ``out``
    [batch, C] (which may be x itself)."""
    dev = _require_cuda(conv_state, x, weight, bias, state_batch_indices,
                        dst_state_batch_indices, out)
    batch = x.shape[0]
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=dev)
    p = _conv_params(conv_state, x, weight, bias, activation, disable_state_update, pad_slot_id,
                     out)
    idx = _slot_vectors(state_batch_indices, dst_state_batch_indices, batch)
    src, _ = _table(state_batch_indices, "state_batch_indices")
    dst, _ = _table(dst_state_batch_indices, "dst_state_batch_indices")
    _abi.check(_abi.lib().ssu_conv_update(
        ctypes.byref(p), batch, batch, None, 1, None, _abi.SSU_I32, ctypes.byref(src),
        ctypes.byref(dst), idx, _stream(dev, stream)))
    return out


def conv_update_varlen(conv_state, x, weight, bias=None, activation="silu", cu_seqlens=None,
                       num_accepted_tokens=None, state_batch_indices=None,
                       dst_state_batch_indices=None, pad_slot_id=-1, out=None, nseqs=None,
                       disable_state_update=False, stream=None):
    """Packed / speculative causal convolution (C ABI ``ssu_conv_update``).

    x is packed [rows, C] with ``cu_seqlens`` [S + 1], or dense
    [batch, steps, C].  Slot tables ([S, T] or flat) and
    ``num_accepted_tokens`` as in ssu_update_varlen: the rows before a
    sequence's first come from its read slot, step t's slot takes the last
    W - 1 rows after it."""
    dev = _require_cuda(conv_state, x, weight, bias, cu_seqlens, num_accepted_tokens,
                        state_batch_indices, dst_state_batch_indices, out)
    steps, shape = 1, None
    if x.dim() == 3:
        shape = x.shape
        batch, steps = x.shape[:2]
        x = x.view(batch * steps, x.shape[2])
        if out is not None:
            out = _dense(out, "out", batch * steps)
        if cu_seqlens is None:
            nseqs = batch
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=dev)
    p = _conv_params(conv_state, x, weight, bias, activation, disable_state_update, pad_slot_id,
                     out)
    nseqs, meta, src, dst, idx = _packed(nseqs, cu_seqlens, num_accepted_tokens,
                                         state_batch_indices, dst_state_batch_indices)
    _abi.check(_abi.lib().ssu_conv_update(
        ctypes.byref(p), nseqs, x.shape[0], _ptr(cu_seqlens), steps, _ptr(num_accepted_tokens),
        meta, ctypes.byref(src), ctypes.byref(dst), idx, _stream(dev, stream)))
    return out if shape is None else out.view(shape)


def conv_fwd_varlen(x, weight, cu_seqlens, bias=None, activation="silu", conv_state=None,
                    state_batch_indices=None, has_initial_state=None,
                    dst_state_batch_indices=None, pad_slot_id=-1, out=None, stream=None):
    """Causal convolution of packed prompts (C ABI ``ssu_conv_fwd_varlen``).

    x [rows, C] packed by ``cu_seqlens`` [S + 1]; weight, bias, activation as
    for conv_update.  With ``conv_state`` each sequence starts from its slot
    (``has_initial_state`` [S] bool: False starts it from zeros; None reads
    every slot) and its slot -- ``dst_state_batch_indices`` or the same --
    takes its last W - 1 rows.  Returns ``out`` [rows, C], which must not
    overlap x."""
    dev = _require_cuda(conv_state, x, weight, bias, cu_seqlens, state_batch_indices,
                        dst_state_batch_indices, has_initial_state, out)
    nseqs, meta = _prompts(cu_seqlens)
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=dev)
    p = _conv_params(conv_state, x, weight, bias, activation, False, pad_slot_id, out)
    _no_overlap(out, x)
    idx = _slot_vectors(state_batch_indices, dst_state_batch_indices, nseqs)
    _abi.check(_abi.lib().ssu_conv_fwd_varlen(
        ctypes.byref(p), nseqs, x.shape[0], _ptr(cu_seqlens), meta, _ptr(state_batch_indices),
        _ptr(dst_state_batch_indices), idx, _flags(has_initial_state, nseqs),
        _stream(dev, stream)))
    return out


# ---------------------------------------------------------------------------
# selective scan
# ---------------------------------------------------------------------------

def _scan_params(state, x, dt, A, B, C, D, z, dt_bias, dt_softplus, disable_state_update,
                 pad_slot_id, out):
    if x.dim() != 2:
        raise ValueError(f"x must be [rows, channels], got {tuple(x.shape)}")
    rows, dim = x.shape
    io = _float_dtype(x, "x")
    if A.dim() != 2 or A.shape[0] != dim:
        raise ValueError(f"A must be [{dim}, dstate], got {tuple(A.shape)}")
    if A.dtype != torch.float32:
        raise NotImplementedError(f"A must be fp32, got {A.dtype}")
    N = A.shape[1]
    if N > 1 and A.stride(1) != 1:
        raise ValueError("A must be contiguous along dstate")
    if B.dim() == 2:   # one group
        B = B.unsqueeze(1)
    if C.dim() == 2:
        C = C.unsqueeze(1)
    if B.dim() != 3 or C.shape != B.shape or B.shape[0] != rows or B.shape[2] != N:
        raise ValueError(f"B/C must be [{rows}, groups, {N}]; got B={tuple(B.shape)}, "
                         f"C={tuple(C.shape)}")
    if B.dtype != x.dtype or C.dtype != x.dtype:
        raise ValueError("B and C must share the x dtype")
    if N > 1 and (B.stride(2) != 1 or C.stride(2) != 1):
        raise ValueError("B and C must be contiguous along dstate")
    if dt.dtype not in (x.dtype, torch.float32):
        raise ValueError(f"dt must be {x.dtype} or fp32, got {dt.dtype}")
    if z is not None and z.dtype != x.dtype:
        raise ValueError("z must match x in shape and dtype")
    if out.dtype not in (x.dtype, torch.float32):
        raise ValueError(f"out must be {x.dtype} (or fp32), got {out.dtype}")
    for name, t in (("D", D), ("dt_bias", dt_bias)):
        if t is not None:
            _vector(t, name, dim, torch.float32)
    p = _abi.ScanParams()
    if state is not None:
        if state.dim() != 3 or state.shape[1] != dim or state.shape[2] != N:
            raise ValueError(f"state must be [slots, {dim}, {N}], got {tuple(state.shape)}")
        if not state.is_contiguous():
            raise ValueError("state must be contiguous")
        p.state, p.state_dtype = state.data_ptr(), _float_dtype(state, "state")
        p.slots = state.shape[0]
    p.channels, p.dstate, p.ngroups, p.io_dtype = dim, N, B.shape[1], io
    p.x, p.x_row_stride = x.data_ptr(), _rows2(x, "x", rows, dim)
    if z is not None:
        p.z, p.z_row_stride = z.data_ptr(), _rows2(z, "z", rows, dim)
    p.out, p.out_dtype = out.data_ptr(), _FLOAT_DT[out.dtype]
    p.out_row_stride = _rows2(out, "out", rows, dim)
    p.dt, p.dt_dtype, p.dt_row_stride = dt.data_ptr(), _FLOAT_DT[dt.dtype], _rows2(dt, "dt", rows,
                                                                                  dim)
    p.B, p.B_row_stride, p.B_group_stride = B.data_ptr(), B.stride(0), B.stride(1)
    p.C, p.C_row_stride, p.C_group_stride = C.data_ptr(), C.stride(0), C.stride(1)
    p.A, p.A_row_stride = A.data_ptr(), A.stride(0)
    p.D = D.data_ptr() if D is not None else None
    p.dt_bias = dt_bias.data_ptr() if dt_bias is not None else None
    p.dt_softplus = int(bool(dt_softplus))
    p.disable_state_update = int(bool(disable_state_update))
    p.pad_slot_id = int(pad_slot_id)
    return p


def scan_update(state, x, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus=False,
                state_batch_indices=None, dst_state_batch_indices=None, pad_slot_id=-1, out=None,
                out_dtype=None, disable_state_update=False, stream=None):
    """One-token selective scan with a full A (C ABI ``ssu_scan_update``).

    state [slots, dim, N] (updated in place; fp32, bf16 or fp16); x, z
    [batch, dim]; dt [batch, dim] in x's dtype or fp32; A [dim, N] fp32; B, C
    [batch, groups, N] or [batch, N]; D, dt_bias [dim] fp32.  Slot vectors
    [batch] int32/int64.  Returns ``out`` [batch, dim] (x's dtype, or
    ``out_dtype=torch.float32``)."""
    dev = _require_cuda(state, x, dt, A, B, C, D, z, dt_bias, state_batch_indices,
                        dst_state_batch_indices, out)
    batch = x.shape[0]
    if out is None:
        out = torch.empty(x.shape, dtype=out_dtype or x.dtype, device=dev)
    p = _scan_params(state, x, dt, A, B, C, D, z, dt_bias, dt_softplus, disable_state_update,
                     pad_slot_id, out)
    idx = _slot_vectors(state_batch_indices, dst_state_batch_indices, batch)
    src, _ = _table(state_batch_indices, "state_batch_indices")
    dst, _ = _table(dst_state_batch_indices, "dst_state_batch_indices")
    _abi.check(_abi.lib().ssu_scan_update(
        ctypes.byref(p), batch, batch, None, 1, None, _abi.SSU_I32, ctypes.byref(src),
        ctypes.byref(dst), idx, _stream(dev, stream)))
    return out


def scan_update_varlen(state, x, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus=False,
                       cu_seqlens=None, num_accepted_tokens=None, state_batch_indices=None,
                       dst_state_batch_indices=None, pad_slot_id=-1, out=None, out_dtype=None,
                       nseqs=None, disable_state_update=False, stream=None):
    """Packed / speculative selective scan with a full A (C ABI
    ``ssu_scan_update``): operands as for scan_update over packed [rows, ...]
    or dense [batch, steps, ...] rows, sequences and slot tables as in
    ssu_update_varlen."""
    dev = _require_cuda(state, x, dt, A, B, C, D, z, dt_bias, cu_seqlens, num_accepted_tokens,
                        state_batch_indices, dst_state_batch_indices, out)
    steps, shape = 1, None
    if x.dim() == 3:
        shape = x.shape
        batch, steps = x.shape[:2]
        rows = batch * steps
        x, dt, z = x.view(rows, x.shape[2]), _dense(dt, "dt", rows), _dense(z, "z", rows)
        B, C = _dense(B, "B", rows), _dense(C, "C", rows)
        if out is not None:
            out = _dense(out, "out", rows)
        if cu_seqlens is None:
            nseqs = batch
    if out is None:
        out = torch.empty(x.shape, dtype=out_dtype or x.dtype, device=dev)
    p = _scan_params(state, x, dt, A, B, C, D, z, dt_bias, dt_softplus, disable_state_update,
                     pad_slot_id, out)
    nseqs, meta, src, dst, idx = _packed(nseqs, cu_seqlens, num_accepted_tokens,
                                         state_batch_indices, dst_state_batch_indices)
    _abi.check(_abi.lib().ssu_scan_update(
        ctypes.byref(p), nseqs, x.shape[0], _ptr(cu_seqlens), steps, _ptr(num_accepted_tokens),
        meta, ctypes.byref(src), ctypes.byref(dst), idx, _stream(dev, stream)))
    return out if shape is None else out.view(shape)


def scan_fwd_varlen(x, dt, A, B, C, cu_seqlens, out=None, D=None, z=None, dt_bias=None,
                    dt_softplus=False, state=None, state_batch_indices=None,
                    has_initial_state=None, dst_state_batch_indices=None, pad_slot_id=-1,
                    out_dtype=None, stream=None):
    """Selective scan of packed prompts with a full A (C ABI
    ``ssu_scan_fwd_varlen``).

    Operands as for scan_update over rows packed by ``cu_seqlens`` [S + 1].
    With ``state`` each sequence starts from its slot (``has_initial_state``
    [S] bool: False starts it from zeros; None reads every slot) and its slot
    -- ``dst_state_batch_indices`` or the same -- takes its final state.
    Returns ``out`` [rows, dim], which must not overlap an operand."""
    dev = _require_cuda(state, x, dt, A, B, C, D, z, dt_bias, cu_seqlens, state_batch_indices,
                        dst_state_batch_indices, has_initial_state, out)
    nseqs, meta = _prompts(cu_seqlens)
    if out is None:
        out = torch.empty(x.shape, dtype=out_dtype or x.dtype, device=dev)
    p = _scan_params(state, x, dt, A, B, C, D, z, dt_bias, dt_softplus, False, pad_slot_id, out)
    _no_overlap(out, x, dt, z)
    idx = _slot_vectors(state_batch_indices, dst_state_batch_indices, nseqs)
    _abi.check(_abi.lib().ssu_scan_fwd_varlen(
        ctypes.byref(p), nseqs, x.shape[0], _ptr(cu_seqlens), meta, _ptr(state_batch_indices),
        _ptr(dst_state_batch_indices), idx, _flags(has_initial_state, nseqs),
        _stream(dev, stream)))
    return out


# ---------------------------------------------------------------------------
# slots
# ---------------------------------------------------------------------------

def _pools(pools):
    """(array of ssu_pool, its length, slots) of tensors [slots, ...]."""
    if not pools:
        raise ValueError("at least one pool is required")
    slots = pools[0].shape[0] if pools[0].dim() else 0
    arr = (_abi.Pool * len(pools))()
    for i, t in enumerate(pools):
        if t.dim() < 1 or t.shape[0] != slots:
            raise ValueError(f"pool {i} must hold {slots} slots like the first, got "
                             f"{tuple(t.shape)}")
        per = t.numel() // slots if slots else 0
        if not t.is_contiguous() and not (slots and t[0].is_contiguous()):
            raise ValueError(f"pool {i}: a slot must be contiguous")
        es = t.element_size()
        arr[i].data, arr[i].slot_bytes = t.data_ptr(), per * es
        arr[i].slot_stride_bytes = t.stride(0) * es
    return arr, len(pools), slots


def _ids(t, name):
    _vector(t, name, t.numel())
    return _int_dtype(t, name)


def slots_copy(pools, src, dst, pad_slot_id=-1, stream=None):
    """Copy slot ``src[i]`` to slot ``dst[i]`` in every pool, in one launch (C
    ABI ``ssu_slots_copy``).

    ``pools``: tensors [slots, ...] of any dtype that share the slot ids (the
    state and convolution pools of all layers, ring caches, trackers).  One
    source may be copied to many slots; pairs with a pad / out-of-range id are
    skipped; a slot that one pair writes must not occur in another."""
    dev = _require_cuda(src, dst, *pools)
    arr, n, slots = _pools(pools)
    d = _ids(src, "src")
    if _ids(dst, "dst") != d or src.numel() != dst.numel():
        raise ValueError("src and dst must share their length and dtype")
    _abi.check(_abi.lib().ssu_slots_copy(arr, n, slots, _ptr(src), _ptr(dst), d, src.numel(),
                                         int(pad_slot_id), _stream(dev, stream)))


def slots_clear(pools, slots, pad_slot_id=-1, stream=None):
    """Zero the slots whose ids are given in every pool, in one launch (C ABI
    ``ssu_slots_clear``)."""
    dev = _require_cuda(slots, *pools)
    arr, n, count = _pools(pools)
    d = _ids(slots, "slots")
    _abi.check(_abi.lib().ssu_slots_clear(arr, n, count, _ptr(slots), d, slots.numel(),
                                          int(pad_slot_id), _stream(dev, stream)))


def slots_compact_workspace_bytes(slots):
    """Bytes of workspace slots_compact needs (C ABI
    ``ssu_slots_compact_workspace_bytes``)."""
    return int(_abi.lib().ssu_slots_compact_workspace_bytes(slots))


def slots_compact(pools, table, pad_slot_id=-1, out=None, num_live=None, workspace=None,
                  stream=None):
    """Close the pools up (C ABI ``ssu_slots_compact``): the m distinct valid
    slots in ``table`` (any shape, contiguous, int32/int64) end up in slots
    0 .. m - 1 of every pool.  Slots below m stay; the others move, in ascending
    order, into the free slots below m.

    Returns (``out``, ``num_live``): the table under the new ids (``out`` may be
    ``table``) and m as a one-element int32 CUDA tensor.  ``workspace``: a CUDA
    uint8 tensor of slots_compact_workspace_bytes(slots), allocated when not
    given."""
    dev = _require_cuda(table, out, num_live, workspace, *pools)
    arr, n, slots = _pools(pools)
    d = _int_dtype(table, "table")
    if not table.is_contiguous():
        raise ValueError("table must be contiguous")
    if out is None:
        out = torch.empty_like(table)
    if out.shape != table.shape or out.dtype != table.dtype or not out.is_contiguous():
        raise ValueError("out must match table's shape and dtype")
    if num_live is None:
        num_live = torch.empty(1, dtype=torch.int32, device=dev)
    if num_live.dtype != torch.int32 or num_live.numel() != 1:
        raise ValueError("num_live must be one int32")
    if workspace is None:
        workspace = torch.empty(slots_compact_workspace_bytes(slots), dtype=torch.uint8, device=dev)
    _abi.check(_abi.lib().ssu_slots_compact(
        arr, n, slots, _ptr(table), _ptr(out), d, table.numel(), int(pad_slot_id),
        _ptr(num_live), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(dev, stream)))
    return out, num_live
