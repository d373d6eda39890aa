"""Linear attention, verification, maps and slot assignment without a GPU: struct
layout, the refusals that the host makes before any launch, the memory that the
binding allocates."""
from __future__ import annotations

import ctypes
import subprocess
import types

import pytest
import torch

from mamba2_ssm_decode_gb300 import _abi
from mamba2_ssm_decode_gb300 import layer_api as api

from .test_layer_abi_cpu import FAKE, HEADER, INVALID, UNSUPPORTED, decode, lib  # noqa: F401
from .test_layer_memory_cpu import streams  # noqa: F401
from .test_layer_overlap_cpu import touched

FAR = FAKE + (1 << 40)
I32, I64, F32, BF16, F16 = (_abi.SSU_I32, _abi.SSU_I64, _abi.SSU_F32, _abi.SSU_BF16, _abi.SSU_F16)


def test_struct_layout_matches_header(tmp_path):
    structs = {"ssu_linattn_params": _abi.LinattnParams, "ssu_drafts_params": _abi.DraftsParams,
               "ssu_prompt_maps_params": _abi.PromptMapsParams}
    src, want = ['#include <stdio.h>', '#include <stddef.h>', f'#include "{HEADER}"',
                 'int main(void){'], []
    for name, cls in structs.items():
        src.append(f'printf("%zu\\n", sizeof({name}));')
        want.append(ctypes.sizeof(cls))
        for f, _ in cls._fields_:
            src.append(f'printf("%zu\\n", offsetof({name}, {f}));')
            want.append(getattr(cls, f).offset)
    src.append('printf("%d\\n", SSU_PROMPT_MAPS_MAX_SEQS); return 0; }')
    want.append(_abi.PROMPT_MAPS_MAX_SEQS)
    c, exe = tmp_path / "layout.c", tmp_path / "layout"
    c.write_text("\n".join(src))
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-o", str(exe), str(c)], check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    assert [int(v) for v in got] == want


# ---------------------------------------------------------------------------
# linear attention
# ---------------------------------------------------------------------------

def lin(**over):
    p = _abi.LinattnParams()
    p.state, p.q, p.k, p.v, p.out = FAKE, FAKE, FAKE, FAKE, FAR
    p.slots, p.nheads, p.ngroups, p.dv, p.dk = 8, 4, 2, 64, 64
    p.io_dtype = BF16
    p.q_row_stride = p.k_row_stride = 128
    p.q_group_stride = p.k_group_stride = 64
    p.v_row_stride = p.out_row_stride = 256
    p.v_head_stride = p.out_head_stride = 64
    p.scale, p.pad_slot_id = 1.0, -1
    for k, v in over.items():
        setattr(p, k, v)
    return p


def fwd(lib, p, nseqs=2, rows=4, cu=FAKE, meta=I32, src=None, dst=None, idx=I32, ws=FAR + 4096,  # noqa: F811
        size=1 << 30):
    return lib.ssu_linattn_fwd_varlen(ctypes.byref(p), nseqs, rows, cu, meta, src, dst, idx, None, ws,
                                      size, None)


REFUSED = [
    (dict(state_dtype=I32), UNSUPPORTED, "state dtype"),
    (dict(io_dtype=I64), UNSUPPORTED, "q/k/v dtype"),
    (dict(dv=0), INVALID, "positive sizes"),
    (dict(slots=-1), INVALID, "positive sizes"),
    (dict(ngroups=3), INVALID, "multiple of the groups"),
    (dict(nheads=8192), UNSUPPORTED, "4096 heads"),
    (dict(dv=257, out_head_stride=257, out_row_stride=1028), UNSUPPORTED, "dv at most 256"),
    (dict(dk=48), UNSUPPORTED, "dk 48"),
    (dict(q=None), INVALID, "NULL"),
    (dict(state=FAKE + 8), INVALID, "16-byte"),
    (dict(k=FAKE + 1), INVALID, "aligned"),
    (dict(log_decay=FAKE + 2), INVALID, "aligned"),
    (dict(out_row_stride=63), INVALID, "out's rows or heads overlap"),
    (dict(out_head_stride=63), INVALID, "out's rows or heads overlap"),
    (dict(out_row_stride=128), INVALID, "out's rows and heads overlap"),
    (dict(out_row_stride=64, out_head_stride=128), INVALID, "out's rows and heads overlap"),
    (dict(out=FAKE), INVALID, "out must not overlap q"),
    (dict(q=FAR + (1 << 30), k=FAR + 64), INVALID, "out must not overlap k"),
    (dict(v=FAR - 2), INVALID, "out must not overlap v"),
    (dict(log_decay=FAR + 4, log_decay_head_stride=1), INVALID, "out must not overlap log_decay"),
    (dict(state=FAR - 16), INVALID, "out must not overlap state"),
    (dict(state=FAR + 4 * 512 - 16), INVALID, "out must not overlap state"),
]


@pytest.mark.parametrize("over,code,needle", REFUSED)
def test_linattn_refusals(lib, over, code, needle):  # noqa: F811
    assert decode(lib, "ssu_linattn_update", lin(**over)) == code
    assert needle in lib.ssu_last_error().decode()
    assert fwd(lib, lin(**over)) == code
    assert needle in lib.ssu_last_error().decode()


def test_linattn_sequence_refusals(lib):  # noqa: F811
    p, err = lin(), lambda: lib.ssu_last_error().decode()  # noqa: E731
    call = lambda p, **kw: decode(lib, "ssu_linattn_update", p, **kw)  # noqa: E731
    assert call(p, na=FAKE) == INVALID and "needs state_batch_indices" in err()
    assert call(p, rows=5) == INVALID and "cannot be split" in err()
    assert call(p, cu=FAKE, meta=F32) == INVALID
    assert call(p, nseqs=9, rows=18) == INVALID and "exceed 8 slots" in err()
    assert call(lin(state=None)) == INVALID and "state must not be NULL" in err()
    assert call(p, nseqs=0, rows=0) == _abi.SSU_OK and err() == ""
    assert fwd(lib, p, cu=None) == INVALID and "cu_seqlens" in err()
    assert fwd(lib, p, nseqs=9) == INVALID
    assert fwd(lib, lin(state=None, slots=0), dst=FAKE) == INVALID and "state pool" in err()
    assert fwd(lib, p, rows=0) == _abi.SSU_OK
    need = lib.ssu_linattn_workspace_bytes(4, 2, 4, 64, 64, BF16)
    assert need > 0
    assert fwd(lib, p, size=need - 1) == INVALID and "workspace" in err()
    assert fwd(lib, p, ws=None) == INVALID and fwd(lib, p, ws=FAR + 8) == INVALID


def test_linattn_workspace():
    lib = _abi.lib()
    size = lib.ssu_linattn_workspace_bytes
    for args in ((-1, 1, 1, 64, 64), (1, -1, 1, 64, 64), (1, 1, -1, 64, 64), (1, 1, 1, -1, 64),
                 (1, 1, 1, 64, -1)):
        assert size(*args, BF16) == -1
    assert size(0, 4, 4, 64, 64, BF16) == size(64, 0, 4, 64, 64, BF16) == 0
    for args in ((64, 1, 4, 64, 64, F32), (64, 1, 4, 65, 64, BF16), (64, 1, 4, 64, 32, F16)):
        assert size(*args) == 0                     # walked row by row
    # room for what any lengths can be cut into: it grows with the rows, not with lengths
    assert size(1 << 20, 1, 4, 128, 128, F16) >= size(1 << 16, 1, 4, 128, 128, F16) > 0
    assert api.linattn_workspace_bytes(64, 1, 4, 64, 64, torch.bfloat16) == size(64, 1, 4, 64, 64, BF16)
    with pytest.raises(NotImplementedError, match="float64"):
        api.linattn_workspace_bytes(64, 1, 4, 64, 64, torch.float64)


def test_linattn_out_against_every_byte(lib):  # noqa: F811
    """A refusal exactly where a byte is shared, with v the columns of a wider tensor."""
    rows, H, dv = 3, 2, 2
    base = dict(nheads=H, ngroups=1, dv=dv, dk=16, q=FAR * 2, k=FAR * 3, q_row_stride=16,
                k_row_stride=16, v=FAKE + 4096, v_row_stride=12, v_head_stride=4)
    theirs = touched(FAKE + 4096, 24, 2 * dv, rows, H, 8)
    for rs, hs in ((4, 2), (12, 4), (2, 8), (10, 5)):
        for at in range(FAKE + 4096 - 80, FAKE + 4096 + 80, 2):
            mine = touched(at, 2 * rs, 2 * dv, rows, H, 2 * hs)
            p = lin(out=at, out_row_stride=rs, out_head_stride=hs, **base)
            st = decode(lib, "ssu_linattn_update", p, nseqs=0, rows=rows, cu=FAKE, dense=0)
            assert (st == INVALID) == bool(mine & theirs), (rs, hs, at - FAKE - 4096)


# ---------------------------------------------------------------------------
# verification
# ---------------------------------------------------------------------------

def drafts(**over):
    p = _abi.DraftsParams()
    p.target_probs, p.draft_probs, p.draft_tokens, p.uniform = FAKE, FAKE, FAKE, FAKE
    p.rows, p.vocab, p.target_row_stride = 6, 100, 100
    p.draft_seq_stride, p.draft_step_stride, p.draft_tokens_seq_stride = 200, 100, 2
    p.nseqs, p.drafts, p.uniform_seq_stride = 2, 2, 3
    p.probs_dtype, p.token_dtype, p.count_dtype, p.meta_dtype = F32, I32, I32, I32
    p.out, p.out_seq_stride, p.num_accepted = FAR, 3, FAR + 4096
    for k, v in over.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("over,code,needle", [
    (dict(probs_dtype=I32), UNSUPPORTED, "probabilities"),
    (dict(token_dtype=F32), INVALID, "int32 or int64"),
    (dict(count_dtype=BF16), INVALID, "int32 or int64"),
    (dict(cu_seqlens=FAKE, meta_dtype=F32), INVALID, "int32 or int64"),
    (dict(vocab=0), INVALID, "vocab positive"),
    (dict(rows=-1), INVALID, ">= 0"),
    (dict(vocab=(1 << 19) + 1), UNSUPPORTED, "2^19"),
    (dict(nseqs=65536, rows=65536 * 3), UNSUPPORTED, "65535"),
    (dict(drafts=4097, rows=2 * 4098, out_seq_stride=4098), UNSUPPORTED, "4096"),
    (dict(rows=5), INVALID, "cannot be split"),
    (dict(out=None), INVALID, "NULL"),
    (dict(uniform=None), INVALID, "NULL"),
    (dict(target_probs=None), INVALID, "NULL"),
    (dict(draft_tokens=None), INVALID, "NULL"),
    (dict(out_seq_stride=2), INVALID, "out's rows overlap"),
    (dict(target_probs=FAKE + 2), INVALID, "aligned"),
    (dict(uniform=FAKE + 1), INVALID, "aligned"),
    (dict(num_accepted=FAR + 2), INVALID, "aligned"),
    (dict(draft_tokens=FAR + 4), INVALID, "must not overlap"),
    (dict(uniform=FAR + 20), INVALID, "must not overlap"),
    (dict(num_accepted=FAR + 8), INVALID, "must not overlap"),
    (dict(target_probs=FAR - 4), INVALID, "out must not overlap target_probs"),
    (dict(draft_probs=FAR + 20), INVALID, "out must not overlap draft_probs"),
    (dict(cu_seqlens=FAR + 20), INVALID, "out must not overlap cu_seqlens"),
    (dict(greedy=FAR + 23), INVALID, "out must not overlap greedy"),
    (dict(num_accepted=FAKE + 4), INVALID, "num_accepted must not overlap"),
])
def test_verify_refusals(lib, over, code, needle):  # noqa: F811
    assert lib.ssu_drafts_verify(ctypes.byref(drafts(**over)), None) == code
    assert needle in lib.ssu_last_error().decode()


def test_verify_of_nothing(lib):  # noqa: F811
    p = drafts(nseqs=0, rows=0, target_probs=None, draft_tokens=None, uniform=None, out=None,
               num_accepted=None)
    assert lib.ssu_drafts_verify(ctypes.byref(p), None) == _abi.SSU_OK
    assert lib.ssu_drafts_verify(None, None) == INVALID


# ---------------------------------------------------------------------------
# maps and assignment
# ---------------------------------------------------------------------------

def maps(**over):
    p = _abi.PromptMapsParams()
    at = FAKE
    for name in ("lens", "context_lens", "cu_seqlens", "cu_chunk_seqlens", "seq_idx",
                 "last_chunk_indices", "has_initial_state", "num_chunks", "row_seq", "row_pos"):
        setattr(p, name, at)
        at += 1 << 20
    p.index_dtype, p.nseqs, p.rows, p.chunk_size, p.max_chunks = I32, 3, 100, 16, 12
    for k, v in over.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("over,code,needle", [
    (dict(index_dtype=F32), INVALID, "int32 or int64"),
    (dict(nseqs=-1), INVALID, ">= 0"),
    (dict(chunk_size=0), INVALID, "chunk_size positive"),
    (dict(nseqs=16385, max_chunks=1 << 20), UNSUPPORTED, "16384"),
    (dict(rows=1 << 31, max_chunks=1 << 28), UNSUPPORTED, "rows"),
    (dict(chunk_size=(1 << 20) + 1), UNSUPPORTED, "2^20"),
    (dict(max_chunks=11), INVALID, "room for 11"),
    (dict(context_lens=None, max_chunks=8), INVALID, "room for 8"),
    (dict(lens=None), INVALID, "NULL"),
    (dict(cu_seqlens=None), INVALID, "NULL"),
    (dict(num_chunks=None), INVALID, "NULL"),
    (dict(has_initial_state=None), INVALID, "NULL"),
    (dict(seq_idx=FAKE + 2), INVALID, "aligned"),
    (dict(cu_seqlens=FAKE), INVALID, "overlap"),
    (dict(row_seq=FAKE + 9 * (1 << 20) + 396), INVALID, "overlap"),
    (dict(context_lens=FAKE + 2 * (1 << 20) + 12), INVALID, "overlap"),
])
def test_maps_refusals(lib, over, code, needle):  # noqa: F811
    assert lib.ssu_prompt_maps(ctypes.byref(maps(**over)), None) == code
    assert needle in lib.ssu_last_error().decode()


def test_assign_refusals(lib):  # noqa: F811
    def call(table=FAKE, counts=FAKE + 4096, idx=I32, n=4, steps=2, slots=8, out=FAR, fresh=FAR + 4096,
             missing=FAR + 8192):
        return lib.ssu_slots_assign(table, counts, idx, n, steps, slots, -1, out, fresh, missing, None)

    err = lambda: lib.ssu_last_error().decode()  # noqa: E731
    assert call(idx=F32) == INVALID and "int32 or int64" in err()
    assert call(n=-1) == INVALID and call(steps=-1) == INVALID and call(slots=-1) == INVALID
    assert call(slots=(1 << 20) + 1) == UNSUPPORTED and "2^20" in err()
    assert call(n=1 << 20, steps=1 << 10) == UNSUPPORTED and "2^24" in err()
    assert call(n=1 << 40, steps=1 << 40) == UNSUPPORTED
    for name in ("table", "counts", "out", "fresh", "missing"):
        assert call(**{name: None}) == INVALID and "NULL" in err()
    assert call(table=FAKE + 2) == INVALID and "aligned" in err()
    assert call(out=FAKE + 4) == INVALID and "overlap" in err()
    assert call(fresh=FAR + 28) == INVALID and "overlap" in err()
    assert call(fresh=FAKE) == INVALID and "overlap" in err()
    assert call(counts=FAR + 16) == INVALID and "overlap" in err()
    assert call(missing=FAKE + 4096) == INVALID and "overlap" in err()


# ---------------------------------------------------------------------------
# memory that the caller does not give
# ---------------------------------------------------------------------------
Q, V4, INTS = torch.zeros(6, 2, 64), torch.zeros(6, 2, 64), torch.zeros(3, dtype=torch.int32)
CALLS = {
    "linattn_update": lambda **kw: api.linattn_update(None, Q, Q, V4, **kw),
    "linattn_update_varlen": lambda **kw: api.linattn_update_varlen(None, Q, Q, V4, **kw),
    "linattn_fwd_varlen": lambda **kw: api.linattn_fwd_varlen(Q, Q, V4, INTS, **kw),
    "linattn_fwd_varlen, workspace": lambda **kw: api.linattn_fwd_varlen(
        Q.bfloat16(), Q.bfloat16(), V4.bfloat16(), INTS, **kw),
    "drafts_verify": lambda **kw: api.drafts_verify(Q[0], torch.zeros(2, 3, dtype=torch.int64),
                                                    Q[0], **kw),
    "prompt_maps": lambda **kw: api.prompt_maps(INTS, 16, 6, **kw),
    "slots_assign": lambda **kw: api.slots_assign(INTS[:, None], INTS, 4, **kw),
}


@pytest.mark.parametrize("call", CALLS)
def test_memory_of_the_call_is_of_its_stream(call, streams, monkeypatch):  # noqa: F811
    nothing = lambda *a: None  # noqa: E731
    monkeypatch.setattr(api, "_module", types.SimpleNamespace(
        linattn=nothing, drafts_verify=nothing, prompt_maps=nothing, slots_assign=nothing))
    side = types.SimpleNamespace(cuda_stream=1)
    CALLS[call](stream=side)
    assert streams and all(s is side for s in streams)
    del streams[:]
    CALLS[call]()
    assert streams and all(s is None for s in streams)
