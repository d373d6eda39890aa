"""The calls around the state update (include/ssu.h) for CUDA torch tensors: the
causal convolution, the selective scan with a full A, and the moves of slots.

Argument marshalling only: the checks that tensors describe the layout the ABI
expects (no hidden copies, no compute) are in csrc/layer_binding.cpp, the calls
go to ``stream``, or to the current torch stream of the tensors' device; what a
caller does not give (``out``, a workspace) is allocated for that stream.
ValueError for a rejected argument, NotImplementedError for a capability the
library does not implement, RuntimeError for a failed launch.
"""
from __future__ import annotations

import importlib.util
import os

import torch

from . import _abi
from ._alloc import empty, result

_ACTIVATIONS = {None: 0, "none": 0, "silu": 1}
_ONE_TOKEN, _PACKED, _PROMPT = 0, 1, 2
_module = None


def _binding():
    """The native module (loaded once); there is no fallback."""
    global _module
    if _module is None:
        _abi.lib()   # the library it is linked to, with the check of its ABI version
        path = os.path.join(os.path.dirname(_abi.LIB_PATH), "_layer_binding.so")
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is not built; run `python -m mamba2_ssm_decode_gb300.build`")
        spec = importlib.util.spec_from_file_location("_layer_binding", path)
        _module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(_module)
    return _module


def _activation(name):
    act = _ACTIVATIONS.get(name)
    if act is None:
        raise ValueError(f"activation must be None or 'silu', got {name!r}")
    return act


def _raw(stream):
    return None if stream is None else stream.cuda_stream


def _dense(t, name, rows):
    """The [rows, ...] view of a dense [batch, steps, ...] operand."""
    if t is None:
        return None
    if t.dim() < 3 or t.shape[0] * t.shape[1] != rows:
        raise ValueError(f"a dense x requires a dense {name} as well, got {tuple(t.shape)}")
    return t.view(rows, *t.shape[2:])


# ---------------------------------------------------------------------------
# causal convolution
# ---------------------------------------------------------------------------

def conv_update(conv_state, x, weight, bias=None, activation="silu", state_batch_indices=None,
                dst_state_batch_indices=None, pad_slot_id=-1, out=None,
                disable_state_update=False, stream=None):
    """One-token causal convolution (C ABI ``ssu_conv_update``).

    conv_state [slots, W - 1, C] (updated in place, x's dtype); x [batch, C]
    (fp32, bf16 or fp16; a column slice of a wider tensor is fine); weight
    [C, W] and bias [C] in x's dtype or fp32; W 2, 3 or 4; ``activation``
    "silu" or None.  Slot vectors [batch] int32/int64.  Returns ``out``
    [batch, C] (which may be x itself)."""
    if out is None:
        out = result(stream, x.shape, x.dtype, x.device)
    (_module or _binding()).conv(
        _ONE_TOKEN, conv_state, x, weight, bias, _activation(activation), None, None,
        state_batch_indices, dst_state_batch_indices, None, pad_slot_id, out, -1, 1,
        disable_state_update, _raw(stream))
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
        out = result(stream, x.shape, x.dtype, x.device)
    (_module or _binding()).conv(
        _PACKED, conv_state, x, weight, bias, _activation(activation), cu_seqlens,
        num_accepted_tokens, state_batch_indices, dst_state_batch_indices, None, pad_slot_id, out,
        -1 if nseqs is None else nseqs, steps, disable_state_update, _raw(stream))
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
    if out is None:
        out = result(stream, x.shape, x.dtype, x.device)
    (_module or _binding()).conv(
        _PROMPT, conv_state, x, weight, bias, _activation(activation), cu_seqlens, None,
        state_batch_indices, dst_state_batch_indices, has_initial_state, pad_slot_id, out, -1, 1,
        False, _raw(stream))
    return out


# ---------------------------------------------------------------------------
# selective scan
# ---------------------------------------------------------------------------

def scan_update(state, x, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus=False,
                state_batch_indices=None, dst_state_batch_indices=None, pad_slot_id=-1, out=None,
                out_dtype=None, disable_state_update=False, stream=None):
    """One-token selective scan with a full A (C ABI ``ssu_scan_update``).

    state [slots, dim, N] (updated in place; fp32, bf16 or fp16); x, z
    [batch, dim]; dt [batch, dim] in x's dtype or fp32; A [dim, N] fp32; B, C
    [batch, groups, N] or [batch, N]; D, dt_bias [dim] fp32.  Slot vectors
    [batch] int32/int64.  Returns ``out`` [batch, dim] (x's dtype, or
    ``out_dtype=torch.float32``; it may be x, dt or z itself)."""
    if out is None:
        out = result(stream, x.shape, out_dtype or x.dtype, x.device)
    (_module or _binding()).scan(
        _ONE_TOKEN, state, x, dt, A, B, C, D, z, dt_bias, dt_softplus, None, None,
        state_batch_indices, dst_state_batch_indices, None, pad_slot_id, out, -1, 1,
        disable_state_update, _raw(stream))
    return out


def scan_update_varlen(state, x, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus=False,
                       cu_seqlens=None, num_accepted_tokens=None, state_batch_indices=None,
                       dst_state_batch_indices=None, pad_slot_id=-1, out=None, out_dtype=None,
                       nseqs=None, disable_state_update=False, stream=None):
    """Packed / speculative selective scan with a full A (C ABI
    ``ssu_scan_update``): operands as for scan_update over packed [rows, ...]
    or dense [batch, steps, ...] rows, sequences and slot tables as in
    ssu_update_varlen."""
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
        out = result(stream, x.shape, out_dtype or x.dtype, x.device)
    (_module or _binding()).scan(
        _PACKED, state, x, dt, A, B, C, D, z, dt_bias, dt_softplus, cu_seqlens,
        num_accepted_tokens, state_batch_indices, dst_state_batch_indices, None, pad_slot_id, out,
        -1 if nseqs is None else nseqs, steps, disable_state_update, _raw(stream))
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
    if out is None:
        out = result(stream, x.shape, out_dtype or x.dtype, x.device)
    (_module or _binding()).scan(
        _PROMPT, state, x, dt, A, B, C, D, z, dt_bias, dt_softplus, cu_seqlens, None,
        state_batch_indices, dst_state_batch_indices, has_initial_state, pad_slot_id, out, -1, 1,
        False, _raw(stream))
    return out


# ---------------------------------------------------------------------------
# slots
# ---------------------------------------------------------------------------

def slots_copy(pools, src, dst, pad_slot_id=-1, stream=None):
    """Copy slot ``src[i]`` to slot ``dst[i]`` in every pool, in one launch (C
    ABI ``ssu_slots_copy``).

    ``pools``: tensors [slots, ...] of any dtype that share the slot ids (the
    state and convolution pools of all layers, ring caches, trackers).  One
    source may be copied to many slots; pairs with a pad / out-of-range id are
    skipped; a slot that one pair writes must not occur in another."""
    (_module or _binding()).slots_copy(pools, src, dst, pad_slot_id, _raw(stream))


def slots_clear(pools, slots, pad_slot_id=-1, stream=None):
    """Zero the slots whose ids are given in every pool, in one launch (C ABI
    ``ssu_slots_clear``)."""
    (_module or _binding()).slots_clear(pools, slots, pad_slot_id, _raw(stream))


def slots_compact_workspace_bytes(slots, entries, in_place=False):
    """Bytes of workspace slots_compact needs for a table of ``entries`` entries
    (C ABI ``ssu_slots_compact_workspace_bytes``); 0 where it takes one launch."""
    return int(_abi.lib().ssu_slots_compact_workspace_bytes(slots, entries, int(in_place)))


def slots_compact(pools, table, pad_slot_id=-1, out=None, num_live=None, workspace=None,
                  stream=None):
    """Close the pools up (C ABI ``ssu_slots_compact``): the m distinct valid
    slots in ``table`` (any shape, contiguous, int32/int64) end up in slots
    0 .. m - 1 of every pool.  Slots below m stay; the others move, in ascending
    order, into the free slots below m.

    Returns (``out``, ``num_live``): the table under the new ids (``out`` may be
    ``table``) and m as a one-element int32 CUDA tensor.  ``workspace``: a CUDA
    uint8 tensor of slots_compact_workspace_bytes(...), allocated when needed and
    not given."""
    if out is None:
        out = result(stream, table.shape, table.dtype, table.device)
    if num_live is None:
        num_live = result(stream, 1, torch.int32, table.device)
    if workspace is None:
        n = pools[0].shape[0] if len(pools) and pools[0].dim() else 0
        in_place = out.data_ptr() == table.data_ptr()   # as the library sees it
        need = slots_compact_workspace_bytes(n, table.numel(), in_place)
        if need > 0:
            workspace = empty(stream, need, torch.uint8, table.device)
    (_module or _binding()).slots_compact(pools, table, out, num_live, workspace, pad_slot_id,
                                          _raw(stream))
    return out, num_live
