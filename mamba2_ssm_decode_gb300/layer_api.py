"""The calls around the state update (include/ssu.h) for CUDA torch tensors: the
causal convolution, the selective scan with a full A, linear attention, the moves
and assignment of slots, the maps of a batch and the verification of drafts.

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
from typing import NamedTuple

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
# linear attention
# ---------------------------------------------------------------------------

def _scale(scale, q):
    return q.shape[-1] ** -0.5 if scale is None else scale


def linattn_update(state, q, k, v, log_decay=None, scale=None, state_batch_indices=None,
                   dst_state_batch_indices=None, pad_slot_id=-1, out=None,
                   disable_state_update=False, stream=None):
    """One-token linear attention with a decay for each head (C ABI
    ``ssu_linattn_update``).

    state [slots, heads, dv, dk] (updated in place; fp32, bf16 or fp16); q, k
    [batch, groups, dk] and v [batch, heads, dv] (fp32, bf16 or fp16; slices of
    a wider tensor are fine); log_decay [heads] or [batch, heads] fp32, or None;
    ``scale`` of the outputs (dk ** -0.5 when None).  Slot vectors [batch]
    int32/int64.  Returns ``out`` [batch, heads, dv], which must not overlap an
    operand."""
    if out is None:
        out = result(stream, v.shape, v.dtype, v.device)
    (_module or _binding()).linattn(
        _ONE_TOKEN, state, q, k, v, log_decay, _scale(scale, q), None, None, state_batch_indices,
        dst_state_batch_indices, None, pad_slot_id, out, -1, 1, disable_state_update, None,
        _raw(stream))
    return out


def linattn_update_varlen(state, q, k, v, log_decay=None, scale=None, cu_seqlens=None,
                          num_accepted_tokens=None, state_batch_indices=None,
                          dst_state_batch_indices=None, pad_slot_id=-1, out=None, nseqs=None,
                          disable_state_update=False, stream=None):
    """Packed / speculative linear attention (C ABI ``ssu_linattn_update``):
    operands as for linattn_update over packed [rows, ...] or dense
    [batch, steps, ...] rows (log_decay [heads] or one value per row and head),
    sequences and slot tables as in ssu_update_varlen."""
    steps, shape = 1, None
    if v.dim() == 4:
        shape = v.shape
        batch, steps = v.shape[:2]
        rows = batch * steps
        v, q, k = v.view(rows, *v.shape[2:]), _dense(q, "q", rows), _dense(k, "k", rows)
        if log_decay is not None and log_decay.dim() == 3:
            log_decay = _dense(log_decay, "log_decay", rows)
        if out is not None:
            out = _dense(out, "out", rows)
        if cu_seqlens is None:
            nseqs = batch
    if out is None:
        out = result(stream, v.shape, v.dtype, v.device)
    (_module or _binding()).linattn(
        _PACKED, state, q, k, v, log_decay, _scale(scale, q), cu_seqlens, num_accepted_tokens,
        state_batch_indices, dst_state_batch_indices, None, pad_slot_id, out,
        -1 if nseqs is None else nseqs, steps, disable_state_update, None, _raw(stream))
    return out if shape is None else out.view(shape)


_IO = {torch.float32: _abi.SSU_F32, torch.bfloat16: _abi.SSU_BF16, torch.float16: _abi.SSU_F16}


def linattn_workspace_bytes(rows, nseqs, nheads, dv, dk, dtype):
    """Bytes of workspace linattn_fwd_varlen needs for ``rows`` packed rows of
    ``nseqs`` sequences in ``dtype`` (C ABI ``ssu_linattn_workspace_bytes``)."""
    if dtype not in _IO:
        raise NotImplementedError(f"v dtype {dtype} is not supported")
    return int(_abi.lib().ssu_linattn_workspace_bytes(rows, nseqs, nheads, dv, dk, _IO[dtype]))


def linattn_fwd_varlen(q, k, v, cu_seqlens, log_decay=None, scale=None, state=None,
                       state_batch_indices=None, has_initial_state=None,
                       dst_state_batch_indices=None, pad_slot_id=-1, out=None, workspace=None,
                       stream=None):
    """Linear attention of packed prompts (C ABI ``ssu_linattn_fwd_varlen``).

    Operands as for linattn_update over rows packed by ``cu_seqlens`` [S + 1].
    With ``state`` each sequence starts from its slot (``has_initial_state``
    [S] bool: False starts it from zeros; None reads every slot) and its slot
    -- ``dst_state_batch_indices`` or the same -- takes its final state.
    ``workspace``: a CUDA uint8 tensor of linattn_workspace_bytes(...),
    allocated when needed and not given.  Returns ``out`` [rows, heads, dv],
    which must not overlap an operand."""
    if out is None:
        out = result(stream, v.shape, v.dtype, v.device)
    if (workspace is None and cu_seqlens is not None and v.dim() == 3 and q.dim() == 3
            and v.dtype in _IO):
        need = linattn_workspace_bytes(v.shape[0], max(cu_seqlens.numel() - 1, 0), v.shape[1],
                                       v.shape[2], q.shape[2], v.dtype)
        if need > 0:
            workspace = empty(stream, need, torch.uint8, v.device)
    (_module or _binding()).linattn(
        _PROMPT, state, q, k, v, log_decay, _scale(scale, q), cu_seqlens, None,
        state_batch_indices, dst_state_batch_indices, has_initial_state, pad_slot_id, out, -1, 1,
        False, workspace, _raw(stream))
    return out


# ---------------------------------------------------------------------------
# drafts and maps
# ---------------------------------------------------------------------------

def drafts_verify(target_probs, draft_tokens, uniform, draft_probs=None, cu_seqlens=None,
                  greedy=None, out=None, num_accepted=None, stream=None):
    """Drafted tokens against the target's probabilities (C ABI
    ``ssu_drafts_verify``).

    target_probs [rows, V] (fp32, bf16 or fp16): a sequence with n drafts has
    n + 1 rows, packed by ``cu_seqlens`` [S + 1] (None: K + 1 each);
    draft_tokens [S, K] int32/int64; draft_probs [S, K, V], what the drafts were
    drawn from (None: certain); ``uniform`` [S, K + 1] fp32 random numbers in
    [0, 1), the last column for the token that is drawn; ``greedy`` [S] bool:
    True takes drafts while they are the row's largest value.

    Returns (``out``, ``num_accepted``): [S, K + 1] tokens -- the drafts taken,
    the next token, then -1 -- and [S] how many they are (int32, or cu_seqlens'
    dtype), the ``num_accepted_tokens`` of the next packed call."""
    if out is None:
        out = result(stream, (draft_tokens.shape[0], draft_tokens.shape[-1] + 1),
                     draft_tokens.dtype, draft_tokens.device)
    if num_accepted is None:
        dtype = torch.int32 if cu_seqlens is None else cu_seqlens.dtype
        num_accepted = result(stream, draft_tokens.shape[0], dtype, draft_tokens.device)
    (_module or _binding()).drafts_verify(target_probs, draft_tokens, uniform, draft_probs,
                                          cu_seqlens, greedy, out, num_accepted, _raw(stream))
    return out, num_accepted


class PromptMaps(NamedTuple):
    """What prompt_maps makes of a batch's lengths (integers in their dtype)."""
    cu_seqlens: torch.Tensor           # [S + 1] row starts
    cu_chunk_seqlens: torch.Tensor     # [max_chunks + 1] chunk starts
    seq_idx: torch.Tensor              # [max_chunks] each chunk's sequence
    last_chunk_indices: torch.Tensor   # [S]
    has_initial_state: torch.Tensor    # [S] bool
    num_chunks: torch.Tensor           # [1]; the chunks behind are empty
    row_seq: torch.Tensor              # [rows] each row's sequence, -1 behind the last
    row_pos: torch.Tensor              # [rows] each row's position, context included, or -1


def prompt_maps(lens, chunk_size, rows, context_lens=None, max_chunks=None, out=None, stream=None):
    """The maps of a packed batch of prompts, from the lengths on the GPU (C ABI
    ``ssu_prompt_maps``): what conv_fwd_varlen, scan_fwd_varlen,
    linattn_fwd_varlen and ssd_combined_fwd_varlen (``chunk_size``) take.

    lens [S] int32/int64: each sequence's tokens in this call; ``rows``: the rows
    of the packed tensors, at least their sum (what is beyond is cut off);
    context_lens [S]: tokens before this call (positions have to fit lens' dtype);
    ``max_chunks``: room for chunks (None: as many as there can be); ``out``: the
    PromptMaps of an earlier call with the same sizes to write again.  Returns a
    PromptMaps."""
    n = lens.numel()
    if max_chunks is None:
        if out is not None:
            max_chunks = out.seq_idx.numel()
        else:
            max_chunks = rows // max(chunk_size, 1) + (1 if context_lens is None else 2) * n
    if out is None:
        def ints(size):
            return result(stream, max(size, 0), lens.dtype, lens.device)
        out = PromptMaps(ints(n + 1), ints(max_chunks + 1), ints(max_chunks), ints(n),
                         result(stream, n, torch.bool, lens.device), ints(1), ints(rows),
                         ints(rows))
    (_module or _binding()).prompt_maps(lens, context_lens, chunk_size, rows, max_chunks, *out,
                                        _raw(stream))
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


def slots_assign(table, counts, slots, pad_slot_id=-1, out=None, fresh=None, num_missing=None,
                 stream=None):
    """Give sequences their slots (C ABI ``ssu_slots_assign``): row s of ``table``
    [S, T] (int32/int64) is to hold ``counts[s]`` of the pools' ``slots``.  Valid
    entries among the first counts[s] stay; the others take the lowest free slots
    in ascending order; the rest of the row becomes pad_slot_id and its slots free.

    Returns (``out``, ``fresh``, ``num_missing``): the new table (``out`` may be
    ``table``), the slots newly given (pad_slot_id elsewhere; slots_clear takes
    it flattened), and how many entries got none, as a one-element int32 CUDA
    tensor."""
    if out is None:
        out = result(stream, table.shape, table.dtype, table.device)
    if fresh is None:
        fresh = result(stream, table.shape, table.dtype, table.device)
    if num_missing is None:
        num_missing = result(stream, 1, torch.int32, table.device)
    (_module or _binding()).slots_assign(table, counts, slots, pad_slot_id, out, fresh, num_missing,
                                         _raw(stream))
    return out, fresh, num_missing
