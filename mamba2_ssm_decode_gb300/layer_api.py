"""Python binding of the calls around the state update (include/ssu.h): the
causal convolution, the selective scan with a full A, and the moves of slots.

Like ``api``: argument marshalling only.  Each function checks that its CUDA
tensors describe the layout the ABI expects (no hidden copies, no compute) and
calls the library on the current torch stream of the tensors' device.
ValueError for a rejected argument, NotImplementedError for a capability the
library does not implement, RuntimeError for a failed launch.
"""
from __future__ import annotations

import struct

import torch

from . import _abi

_FLOAT = {torch.float32: _abi.SSU_F32, torch.bfloat16: _abi.SSU_BF16, torch.float16: _abi.SSU_F16}
_INT = {torch.int32: _abi.SSU_I32, torch.int64: _abi.SSU_I64}
_ACTIVATIONS = {None: 0, "none": 0, "silu": 1}
_current_stream = torch._C._cuda_getCurrentRawStream
_pack_conv = _abi.packer(_abi.ConvParams)
_pack_scan = _abi.packer(_abi.ScanParams)
_pack_table = _abi.packer(_abi.SlotTable)
_NO_TABLE = _pack_table(0, 0, 0, 0, 0)


# These calls take a few microseconds on the device, so the checks below are
# written for few and cheap looks at each tensor.

def _device(first, *others):
    """The CUDA device index that every tensor is on."""
    d = first.get_device()
    for t in others:
        if t is not None and t.get_device() != d:
            if t.get_device() < 0 or d < 0:
                break
            raise ValueError(f"all tensors must be on one device, got {first.device} and {t.device}")
    else:
        if d >= 0:
            return d
    raise ValueError("libssu_gb300 works on CUDA tensors only (there is no CPU path)")


def _stream(d, stream):
    return _current_stream(d) if stream is None else stream.cuda_stream


def _call(name, d, *args):
    """Call the library with device d current (a launch goes to the current device)."""
    f = getattr(_abi.lib(), name)
    if d == torch._C._cuda_getDevice():
        status = f(*args)
    else:
        with torch.cuda.device(d):
            status = f(*args)
    if status:
        _abi.check(status)


def _rows2(t, name, rows, dim):
    """Row stride of a [rows, dim] operand with unit dim stride."""
    if t.dim() != 2 or t.shape != (rows, dim):
        raise ValueError(f"{name} must be [{rows}, {dim}], got {tuple(t.shape)}")
    rs, cs = t.stride()
    if cs != 1 and dim > 1:
        raise ValueError(f"{name} must be contiguous along channels (stride 1), got {t.stride()}")
    return rs


def _vector(t, name, n):
    """A contiguous [n] tensor's address."""
    if t.dim() != 1 or t.shape[0] != n:
        raise ValueError(f"{name} must be [{n}], got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _index(t, name):
    d = _INT.get(t.dtype)
    if d is None:
        raise ValueError(f"{name} must be int32 or int64, got {t.dtype}")
    return d


def _same_index(src, dst):
    """Common index dtype of the read and write slots."""
    if src is None and dst is None:
        return _abi.SSU_I32
    a = dst if src is None else src
    d = _index(a, "state_batch_indices")
    if dst is not None and dst is not a and _index(dst, "dst_state_batch_indices") != d:
        raise ValueError("state_batch_indices and dst_state_batch_indices must share a dtype")
    return d


def _address(t):
    return 0 if t is None else t.data_ptr()


def _flags(t, nseqs):
    """has_initial_state: one byte per sequence."""
    if t is None:
        return 0
    at = _vector(t, "has_initial_state", nseqs)
    if t.dtype is not torch.bool and t.dtype is not torch.uint8:
        raise ValueError(f"has_initial_state must be bool or uint8, got {t.dtype}")
    return at


def _no_overlap(out, *operands):
    at = out.data_ptr()
    for t in operands:
        if t is not None and at and t.data_ptr() == at:
            raise ValueError("out must not overlap an operand of a prompt call")


def _dense(t, name, rows):
    """The [rows, ...] view of a dense [batch, steps, ...] operand."""
    if t is None:
        return None
    if t.dim() < 3 or t.shape[0] * t.shape[1] != rows:
        raise ValueError(f"a dense x requires a dense {name} as well, got {tuple(t.shape)}")
    return t.view(rows, *t.shape[2:])


def _slots_of(t, name, nseqs):
    """Slot vector of a one-token call as a table of one step."""
    if t is None:
        return _NO_TABLE
    at = _vector(t, name, nseqs)
    return _pack_table(at, nseqs, 1, 1, 1)


def _table(t, name, nseqs):
    """Slot table of a packed call: [S, T], or flat with entry (s, t) = s + t."""
    if t is None:
        return _NO_TABLE
    if t.dim() == 1:
        n, step = t.shape[0], t.stride(0)
        return _pack_table(t.data_ptr(), (n - 1) * step + 1 if n else 0, step, step, n)
    if t.dim() != 2:
        raise ValueError(f"{name} must be the flat [rows] or the 2-D [sequences, steps] slot "
                         f"table; got {tuple(t.shape)}")
    (S, T), (ss, ts) = t.shape, t.stride()
    if S < nseqs:
        raise ValueError(f"{name} must have a row for each of the {nseqs} sequences, got "
                         f"{tuple(t.shape)}")
    return _pack_table(t.data_ptr(), (S - 1) * ss + (T - 1) * ts + 1 if S and T else 0, ss, ts, T)


def _packed(nseqs, cu_seqlens, num_accepted_tokens, src, dst):
    """Sequences of a packed decode call: (nseqs, meta dtype)."""
    if nseqs is None:
        if cu_seqlens is not None:
            nseqs = cu_seqlens.numel() - 1
        elif num_accepted_tokens is not None:
            nseqs = num_accepted_tokens.numel()
        elif src is not None:
            nseqs = src.shape[0]
        elif dst is not None:
            nseqs = dst.shape[0]
        else:
            raise ValueError("a packed multi-token call must carry per-sequence metadata: "
                             "state_batch_indices, dst_state_batch_indices, "
                             "num_accepted_tokens or cu_seqlens")
    meta = None
    if cu_seqlens is not None:
        _vector(cu_seqlens, "cu_seqlens", nseqs + 1)
        meta = _index(cu_seqlens, "cu_seqlens")
    if num_accepted_tokens is not None:
        _vector(num_accepted_tokens, "num_accepted_tokens", nseqs)
        d = _index(num_accepted_tokens, "num_accepted_tokens")
        if meta is not None and d != meta:
            raise ValueError("cu_seqlens and num_accepted_tokens must share a dtype")
        meta = d
    return nseqs, _abi.SSU_I32 if meta is None else meta


def _prompts(cu_seqlens):
    if cu_seqlens is None or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must hold the start of every sequence and the end of the last")
    if not cu_seqlens.is_contiguous():
        raise ValueError("cu_seqlens must be contiguous")
    return cu_seqlens.shape[0] - 1, _index(cu_seqlens, "cu_seqlens")


# ---------------------------------------------------------------------------
# causal convolution
# ---------------------------------------------------------------------------

def _conv_params(conv_state, x, weight, bias, activation, disable_state_update, pad_slot_id, out):
    if x.dim() != 2:
        raise ValueError(f"x must be [rows, channels], got {tuple(x.shape)}")
    rows, C = x.shape
    dtype = x.dtype
    io = _FLOAT.get(dtype)
    if io is None:
        raise NotImplementedError(f"x dtype {dtype} is not supported")
    if weight.dim() != 2 or weight.shape[0] != C:
        raise ValueError(f"weight must be [{C}, width], got {tuple(weight.shape)}")
    if not weight.is_contiguous():
        raise ValueError("weight must be contiguous")
    W = weight.shape[1]
    wt = weight.dtype
    if wt is not dtype and wt is not torch.float32:
        raise ValueError(f"weight must be {dtype} or fp32, got {wt}")
    b = 0
    if bias is not None:
        b = _vector(bias, "bias", C)
        if bias.dtype is not wt:
            raise ValueError(f"bias must have weight's dtype ({wt}), got {bias.dtype}")
    act = _ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation must be None or 'silu', got {activation!r}")
    state = slots = 0
    if conv_state is not None:
        if conv_state.dim() != 3 or conv_state.shape[1:] != (W - 1, C):
            raise ValueError(f"conv_state must be [slots, {W - 1}, {C}], got "
                             f"{tuple(conv_state.shape)}")
        if conv_state.dtype is not dtype:
            raise ValueError(f"conv_state must be {dtype}, got {conv_state.dtype}")
        if not conv_state.is_contiguous():
            raise ValueError("conv_state must be contiguous")
        state, slots = conv_state.data_ptr(), conv_state.shape[0]
    if out.dtype is not dtype:
        raise ValueError(f"out must be {dtype}, got {out.dtype}")
    return _pack_conv(state, slots, C, W, io, x.data_ptr(), _rows2(x, "x", rows, C), out.data_ptr(),
                      _rows2(out, "out", rows, C), weight.data_ptr(), b, _FLOAT[wt], act,
                      1 if disable_state_update else 0, int(pad_slot_id))


def conv_update(conv_state, x, weight, bias=None, activation="silu", state_batch_indices=None,
                dst_state_batch_indices=None, pad_slot_id=-1, out=None,
                disable_state_update=False, stream=None):
    """One-token causal convolution (C ABI ``ssu_conv_update``).

    conv_state [slots, W - 1, C] (updated in place, x's dtype); x [batch, C]
    (fp32, bf16 or fp16; a column slice of a wider tensor is fine); weight
    [C, W] and bias [C] in x's dtype or fp32; W 2, 3 or 4; ``activation``
    "silu" or None.  Slot vectors [batch] int32/int64.  Returns ``out``
    [batch, C] (which may be x itself)."""
    dev = _device(x, conv_state, weight, bias, state_batch_indices, dst_state_batch_indices, out)
    batch = x.shape[0]
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    p = _conv_params(conv_state, x, weight, bias, activation, disable_state_update, pad_slot_id,
                     out)
    _call("ssu_conv_update", dev, p, batch, batch, None, 1, None, _abi.SSU_I32,
          _slots_of(state_batch_indices, "state_batch_indices", batch),
          _slots_of(dst_state_batch_indices, "dst_state_batch_indices", batch),
          _same_index(state_batch_indices, dst_state_batch_indices), _stream(dev, stream))
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
    dev = _device(x, conv_state, weight, bias, cu_seqlens, num_accepted_tokens,
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
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    p = _conv_params(conv_state, x, weight, bias, activation, disable_state_update, pad_slot_id,
                     out)
    nseqs, meta = _packed(nseqs, cu_seqlens, num_accepted_tokens, state_batch_indices,
                          dst_state_batch_indices)
    _call("ssu_conv_update", dev, p, nseqs, x.shape[0], _address(cu_seqlens), steps,
          _address(num_accepted_tokens), meta,
          _table(state_batch_indices, "state_batch_indices", nseqs),
          _table(dst_state_batch_indices, "dst_state_batch_indices", nseqs),
          _same_index(state_batch_indices, dst_state_batch_indices), _stream(dev, stream))
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
    dev = _device(x, conv_state, weight, bias, cu_seqlens, state_batch_indices,
                  dst_state_batch_indices, has_initial_state, out)
    nseqs, meta = _prompts(cu_seqlens)
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    p = _conv_params(conv_state, x, weight, bias, activation, False, pad_slot_id, out)
    _no_overlap(out, x)
    _call("ssu_conv_fwd_varlen", dev, p, nseqs, x.shape[0], cu_seqlens.data_ptr(), meta,
          *_prompt_slots(state_batch_indices, dst_state_batch_indices, nseqs),
          _flags(has_initial_state, nseqs), _stream(dev, stream))
    return out


def _prompt_slots(src, dst, nseqs):
    """Addresses of the read and write slots, and their dtype."""
    return (0 if src is None else _vector(src, "state_batch_indices", nseqs),
            0 if dst is None else _vector(dst, "dst_state_batch_indices", nseqs),
            _same_index(src, dst))


# ---------------------------------------------------------------------------
# selective scan
# ---------------------------------------------------------------------------

def _scan_params(state, x, dt, A, B, C, D, z, dt_bias, dt_softplus, disable_state_update,
                 pad_slot_id, out):
    if x.dim() != 2:
        raise ValueError(f"x must be [rows, channels], got {tuple(x.shape)}")
    rows, dim = x.shape
    dtype = x.dtype
    io = _FLOAT.get(dtype)
    if io is None:
        raise NotImplementedError(f"x dtype {dtype} is not supported")
    if A.dim() != 2 or A.shape[0] != dim:
        raise ValueError(f"A must be [{dim}, dstate], got {tuple(A.shape)}")
    f32 = torch.float32
    if A.dtype is not f32:
        raise NotImplementedError(f"A must be fp32, got {A.dtype}")
    N = A.shape[1]
    a_row, a_col = A.stride()
    if a_col != 1 and N > 1:
        raise ValueError("A must be contiguous along dstate")
    bs, bstride, cstride = B.shape, B.stride(), C.stride()
    if C.shape != bs or len(bs) not in (2, 3) or bs[0] != rows or bs[-1] != N:
        raise ValueError(f"B/C must be [{rows}, groups, {N}] or [{rows}, {N}]; got B={tuple(bs)}, "
                         f"C={tuple(C.shape)}")
    if B.dtype is not dtype or C.dtype is not dtype:
        raise ValueError("B and C must share the x dtype")
    if N > 1 and (bstride[-1] != 1 or cstride[-1] != 1):
        raise ValueError("B and C must be contiguous along dstate")
    groups, b_group, c_group = (1, N, N) if len(bs) == 2 else (bs[1], bstride[1], cstride[1])
    ddt = dt.dtype
    if ddt is not dtype and ddt is not f32:
        raise ValueError(f"dt must be {dtype} or fp32, got {ddt}")
    if z is not None and z.dtype is not dtype:
        raise ValueError("z must match x in shape and dtype")
    odt = out.dtype
    if odt is not dtype and odt is not f32:
        raise ValueError(f"out must be {dtype} (or fp32), got {odt}")
    skip = bias = 0
    if D is not None:
        skip = _vector(D, "D", dim)
        if D.dtype is not f32:
            raise NotImplementedError(f"D must be fp32, got {D.dtype}")
    if dt_bias is not None:
        bias = _vector(dt_bias, "dt_bias", dim)
        if dt_bias.dtype is not f32:
            raise NotImplementedError(f"dt_bias must be fp32, got {dt_bias.dtype}")
    pool = pool_dt = slots = 0
    if state is not None:
        if state.dim() != 3 or state.shape[1:] != (dim, N):
            raise ValueError(f"state must be [slots, {dim}, {N}], got {tuple(state.shape)}")
        if not state.is_contiguous():
            raise ValueError("state must be contiguous")
        pool, pool_dt, slots = state.data_ptr(), _FLOAT.get(state.dtype), state.shape[0]
        if pool_dt is None:
            raise NotImplementedError(f"state dtype {state.dtype} is not supported")
    return _pack_scan(pool, pool_dt, slots, dim, N, groups, io, x.data_ptr(),
                      _rows2(x, "x", rows, dim), _address(z),
                      0 if z is None else _rows2(z, "z", rows, dim), out.data_ptr(), _FLOAT[odt],
                      _rows2(out, "out", rows, dim), dt.data_ptr(), _FLOAT[ddt],
                      _rows2(dt, "dt", rows, dim), B.data_ptr(), bstride[0], b_group, C.data_ptr(),
                      cstride[0], c_group, A.data_ptr(), a_row, skip, bias,
                      1 if dt_softplus else 0, 1 if disable_state_update else 0, int(pad_slot_id))


def scan_update(state, x, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus=False,
                state_batch_indices=None, dst_state_batch_indices=None, pad_slot_id=-1, out=None,
                out_dtype=None, disable_state_update=False, stream=None):
    """One-token selective scan with a full A (C ABI ``ssu_scan_update``).

    state [slots, dim, N] (updated in place; fp32, bf16 or fp16); x, z
    [batch, dim]; dt [batch, dim] in x's dtype or fp32; A [dim, N] fp32; B, C
    [batch, groups, N] or [batch, N]; D, dt_bias [dim] fp32.  Slot vectors
    [batch] int32/int64.  Returns ``out`` [batch, dim] (x's dtype, or
    ``out_dtype=torch.float32``)."""
    dev = _device(x, state, dt, A, B, C, D, z, dt_bias, state_batch_indices,
                  dst_state_batch_indices, out)
    batch = x.shape[0]
    if out is None:
        out = torch.empty(x.shape, dtype=out_dtype or x.dtype, device=x.device)
    p = _scan_params(state, x, dt, A, B, C, D, z, dt_bias, dt_softplus, disable_state_update,
                     pad_slot_id, out)
    _call("ssu_scan_update", dev, p, batch, batch, None, 1, None, _abi.SSU_I32,
          _slots_of(state_batch_indices, "state_batch_indices", batch),
          _slots_of(dst_state_batch_indices, "dst_state_batch_indices", batch),
          _same_index(state_batch_indices, dst_state_batch_indices), _stream(dev, stream))
    return out


def scan_update_varlen(state, x, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus=False,
                       cu_seqlens=None, num_accepted_tokens=None, state_batch_indices=None,
                       dst_state_batch_indices=None, pad_slot_id=-1, out=None, out_dtype=None,
                       nseqs=None, disable_state_update=False, stream=None):
    """Packed / speculative selective scan with a full A (C ABI
    ``ssu_scan_update``): operands as for scan_update over packed [rows, ...]
    or dense [batch, steps, ...] rows, sequences and slot tables as in
    ssu_update_varlen."""
    dev = _device(x, state, dt, A, B, C, D, z, dt_bias, cu_seqlens, num_accepted_tokens,
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
        out = torch.empty(x.shape, dtype=out_dtype or x.dtype, device=x.device)
    p = _scan_params(state, x, dt, A, B, C, D, z, dt_bias, dt_softplus, disable_state_update,
                     pad_slot_id, out)
    nseqs, meta = _packed(nseqs, cu_seqlens, num_accepted_tokens, state_batch_indices,
                          dst_state_batch_indices)
    _call("ssu_scan_update", dev, p, nseqs, x.shape[0], _address(cu_seqlens), steps,
          _address(num_accepted_tokens), meta,
          _table(state_batch_indices, "state_batch_indices", nseqs),
          _table(dst_state_batch_indices, "dst_state_batch_indices", nseqs),
          _same_index(state_batch_indices, dst_state_batch_indices), _stream(dev, stream))
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
    dev = _device(x, state, dt, A, B, C, D, z, dt_bias, cu_seqlens, state_batch_indices,
                  dst_state_batch_indices, has_initial_state, out)
    nseqs, meta = _prompts(cu_seqlens)
    if out is None:
        out = torch.empty(x.shape, dtype=out_dtype or x.dtype, device=x.device)
    p = _scan_params(state, x, dt, A, B, C, D, z, dt_bias, dt_softplus, False, pad_slot_id, out)
    _no_overlap(out, x, dt, z)
    _call("ssu_scan_fwd_varlen", dev, p, nseqs, x.shape[0], cu_seqlens.data_ptr(), meta,
          *_prompt_slots(state_batch_indices, dst_state_batch_indices, nseqs),
          _flags(has_initial_state, nseqs), _stream(dev, stream))
    return out


# ---------------------------------------------------------------------------
# slots
# ---------------------------------------------------------------------------

def _pools(pools):
    """(packed array of ssu_pool, its length, slots) of tensors [slots, ...]."""
    if not pools:
        raise ValueError("at least one pool is required")
    slots = pools[0].shape[0] if pools[0].dim() else 0
    fields = []
    for i, t in enumerate(pools):
        if t.dim() < 1 or t.shape[0] != slots:
            raise ValueError(f"pool {i} must hold {slots} slots like the first, got "
                             f"{tuple(t.shape)}")
        if t.is_contiguous():
            size = stride = t.nbytes // slots if slots else 0
        elif t[0].is_contiguous():
            size, stride = t.nbytes // slots, t.stride(0) * t.element_size()
        else:
            raise ValueError(f"pool {i}: a slot must be contiguous")
        fields += (t.data_ptr(), size, stride)
    return struct.pack(f"{len(fields)}q", *fields), len(pools), slots


def _ids(t, name):
    """(address, dtype) of a vector of slot ids."""
    return _vector(t, name, t.numel()), _index(t, name)


def slots_copy(pools, src, dst, pad_slot_id=-1, stream=None):
    """Copy slot ``src[i]`` to slot ``dst[i]`` in every pool, in one launch (C
    ABI ``ssu_slots_copy``).

    ``pools``: tensors [slots, ...] of any dtype that share the slot ids (the
    state and convolution pools of all layers, ring caches, trackers).  One
    source may be copied to many slots; pairs with a pad / out-of-range id are
    skipped; a slot that one pair writes must not occur in another."""
    dev = _device(src, dst, *pools)
    arr, n, slots = _pools(pools)
    s, d = _ids(src, "src")
    t, dd = _ids(dst, "dst")
    if dd != d or src.numel() != dst.numel():
        raise ValueError("src and dst must share their length and dtype")
    _call("ssu_slots_copy", dev, arr, n, slots, s, t, d, src.numel(), int(pad_slot_id),
          _stream(dev, stream))


def slots_clear(pools, slots, pad_slot_id=-1, stream=None):
    """Zero the slots whose ids are given in every pool, in one launch (C ABI
    ``ssu_slots_clear``)."""
    dev = _device(slots, *pools)
    arr, n, count = _pools(pools)
    at, d = _ids(slots, "slots")
    _call("ssu_slots_clear", dev, arr, n, count, at, d, slots.numel(), int(pad_slot_id),
          _stream(dev, stream))


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
    dev = _device(table, out, num_live, workspace, *pools)
    arr, n, slots = _pools(pools)
    d = _index(table, "table")
    if not table.is_contiguous():
        raise ValueError("table must be contiguous")
    if out is None:
        out = torch.empty_like(table)
    elif out.shape != table.shape or out.dtype is not table.dtype or not out.is_contiguous():
        raise ValueError("out must match table's shape and dtype")
    if num_live is None:
        num_live = torch.empty(1, dtype=torch.int32, device=table.device)
    elif num_live.dtype is not torch.int32 or num_live.numel() != 1:
        raise ValueError("num_live must be one int32")
    if workspace is None:
        workspace = torch.empty(slots_compact_workspace_bytes(slots), dtype=torch.uint8,
                                device=table.device)
    _call("ssu_slots_compact", dev, arr, n, slots, table.data_ptr(), out.data_ptr(), d,
          table.numel(), int(pad_slot_id), num_live.data_ptr(), workspace.data_ptr(),
          workspace.nbytes, _stream(dev, stream))
    return out, num_live
