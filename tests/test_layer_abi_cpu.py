"""The C ABI of the calls around the state update without a GPU: struct layout
and the refusals that the host makes before any launch."""
from __future__ import annotations

import ctypes
import os
import subprocess

import pytest

from mamba2_ssm_decode_gb300 import _abi

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "ssu.h")
FAKE = 0x10000  # a 16-byte aligned address the host code never dereferences
INVALID, UNSUPPORTED = _abi.SSU_ERR_INVALID_ARGUMENT, _abi.SSU_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    from mamba2_ssm_decode_gb300 import build
    build.build()
    return _abi.lib()


def test_struct_layout_matches_header(tmp_path):
    structs = {"ssu_conv_params": _abi.ConvParams, "ssu_scan_params": _abi.ScanParams,
               "ssu_pool": _abi.Pool}
    src, want = ['#include <stdio.h>', '#include <stddef.h>', f'#include "{HEADER}"',
                 'int main(void){'], []
    for name, cls in structs.items():
        src.append(f'printf("%zu\\n", sizeof({name}));')
        want.append(ctypes.sizeof(cls))
        for f, _ in cls._fields_:
            src.append(f'printf("%zu\\n", offsetof({name}, {f}));')
            want.append(getattr(cls, f).offset)
    src.append('printf("%d\\n", SSU_SLOTS_MAX_POOLS); return 0; }')
    want.append(_abi.SLOTS_MAX_POOLS)
    c, exe = tmp_path / "layout.c", tmp_path / "layout"
    c.write_text("\n".join(src))
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-o", str(exe), str(c)], check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    assert [int(v) for v in got] == want


def conv(**over):
    p = _abi.ConvParams()
    p.conv_state = p.x = p.out = p.weight = FAKE
    p.out = FAKE + 4096
    p.slots, p.channels, p.width = 8, 64, 4
    p.io_dtype = p.weight_dtype = _abi.SSU_BF16
    p.x_row_stride = p.out_row_stride = 64
    p.activation, p.pad_slot_id = 1, -1
    for k, v in over.items():
        setattr(p, k, v)
    return p


def scan(**over):
    p = _abi.ScanParams()
    p.state = p.x = p.dt = p.B = p.C = p.A = FAKE
    p.out = FAKE + 4096
    p.slots, p.channels, p.dstate, p.ngroups = 8, 64, 16, 2
    p.io_dtype = p.dt_dtype = p.out_dtype = _abi.SSU_BF16
    p.x_row_stride = p.out_row_stride = p.dt_row_stride = 64
    p.A_row_stride, p.pad_slot_id = 16, -1
    for k, v in over.items():
        setattr(p, k, v)
    return p


def decode(lib, name, p, nseqs=2, rows=4, cu=None, dense=2, na=None, meta=_abi.SSU_I32, src=None,
           dst=None, idx=_abi.SSU_I32):
    src = src or _abi.SlotTable(None, 0, 0, 0, 0)
    dst = dst or _abi.SlotTable(None, 0, 0, 0, 0)
    return getattr(lib, name)(ctypes.byref(p), nseqs, rows, cu, dense, na, meta, ctypes.byref(src),
                              ctypes.byref(dst), idx, None)


def prompt(lib, name, p, nseqs=2, rows=4, cu=FAKE, meta=_abi.SSU_I32, src=None, dst=None,
           idx=_abi.SSU_I32):
    return getattr(lib, name)(ctypes.byref(p), nseqs, rows, cu, meta, src, dst, idx, None, None)


CALLS = [("ssu_conv_update", "ssu_conv_fwd_varlen", conv),
         ("ssu_scan_update", "ssu_scan_fwd_varlen", scan)]


@pytest.mark.parametrize("update,fwd,make", CALLS)
def test_sequence_refusals(lib, update, fwd, make):
    p, err = make(), lambda: lib.ssu_last_error().decode()  # noqa: E731
    table = _abi.SlotTable(FAKE, 8, 4, 1, 4)
    assert decode(lib, update, p, na=FAKE) == INVALID and "needs state_batch_indices" in err()
    assert decode(lib, update, p, rows=5) == INVALID and "cannot be split" in err()
    assert decode(lib, update, p, dense=0) == INVALID
    assert decode(lib, update, p, cu=FAKE, meta=_abi.SSU_F32) == INVALID
    assert decode(lib, update, p, src=table, idx=_abi.SSU_BF16) == INVALID
    assert decode(lib, update, p, src=_abi.SlotTable(FAKE, -1, 4, 1, 4)) == INVALID
    assert decode(lib, update, p, nseqs=9, rows=18) == INVALID and "exceed 8 slots" in err()
    assert decode(lib, update, p, nseqs=-1) == INVALID
    assert decode(lib, update, p, nseqs=1 << 30, rows=1 << 30, dense=1) == UNSUPPORTED
    assert decode(lib, update, p, nseqs=0, rows=0) == _abi.SSU_OK and err() == ""
    assert prompt(lib, fwd, p, cu=None) == INVALID and "cu_seqlens" in err()
    assert prompt(lib, fwd, p, meta=_abi.SSU_F16) == INVALID
    assert prompt(lib, fwd, p, src=FAKE, idx=_abi.SSU_F16) == INVALID
    assert prompt(lib, fwd, p, nseqs=9) == INVALID
    assert prompt(lib, fwd, p, rows=-1) == INVALID
    assert prompt(lib, fwd, p, rows=1 << 31) == UNSUPPORTED
    no_pool = make(**{"conv_state" if make is conv else "state": None}, slots=0)
    assert prompt(lib, fwd, no_pool, dst=FAKE) == INVALID and "state pool" in err()
    assert prompt(lib, fwd, make(out=FAKE)) == INVALID and "out must not" in err()
    assert prompt(lib, fwd, p, rows=0) == _abi.SSU_OK
    assert prompt(lib, fwd, p, nseqs=0) == _abi.SSU_OK
    assert prompt(lib, fwd, make(x=None), rows=0) == _abi.SSU_OK   # no rows: nothing is read


@pytest.mark.parametrize("over,code,needle", [
    (dict(io_dtype=_abi.SSU_I32), UNSUPPORTED, "x must be"),
    (dict(weight_dtype=_abi.SSU_F16), INVALID, "weight"),
    (dict(channels=0), INVALID, "channels"),
    (dict(channels=1 << 25), UNSUPPORTED, "2^24"),
    (dict(width=1), UNSUPPORTED, "width"),
    (dict(width=5), UNSUPPORTED, "width"),
    (dict(activation=2), INVALID, "activation"),
    (dict(x=None), INVALID, "NULL"),
    (dict(conv_state=None), INVALID, "conv_state"),
    (dict(x=FAKE + 1), INVALID, "aligned"),
    (dict(out_row_stride=63), INVALID, "out rows overlap"),
])
def test_conv_refusals(lib, over, code, needle):
    assert decode(lib, "ssu_conv_update", conv(**over)) == code
    assert needle in lib.ssu_last_error().decode()


@pytest.mark.parametrize("over,code,needle", [
    (dict(io_dtype=_abi.SSU_I64), UNSUPPORTED, "dtype"),
    (dict(state_dtype=_abi.SSU_I32), UNSUPPORTED, "state dtype"),
    (dict(dt_dtype=_abi.SSU_F16), INVALID, "dt must"),
    (dict(out_dtype=_abi.SSU_F16), INVALID, "out must"),
    (dict(ngroups=3), INVALID, "multiple of ngroups"),
    (dict(dstate=24), UNSUPPORTED, "dstate 24"),
    (dict(channels=0), INVALID, "positive"),
    (dict(A=None), INVALID, "NULL"),
    (dict(state=FAKE + 8), INVALID, "16-byte"),
    (dict(dt=FAKE + 1), INVALID, "aligned"),
    (dict(out_row_stride=63), INVALID, "out rows overlap"),
])
def test_scan_refusals(lib, over, code, needle):
    assert decode(lib, "ssu_scan_update", scan(**over)) == code
    assert needle in lib.ssu_last_error().decode()


def test_slots_refusals(lib):
    def pools(*specs):
        return (_abi.Pool * len(specs))(*[_abi.Pool(*s) for s in specs])

    one = pools((FAKE, 64, 64))
    err = lambda: lib.ssu_last_error().decode()  # noqa: E731
    I32 = _abi.SSU_I32
    copy = lambda a, n=1, slots=4, idx=I32, pairs=2, src=FAKE: lib.ssu_slots_copy(  # noqa: E731
        a, n, slots, src, FAKE, idx, pairs, -1, None)
    assert copy(one, n=-1) == INVALID
    assert copy(one, n=257) == UNSUPPORTED and "256 pools" in err()
    assert copy(one, slots=(1 << 20) + 1) == UNSUPPORTED
    assert copy(pools((FAKE, 64, 32))) == INVALID and "stride" in err()
    assert copy(pools((None, 64, 64))) == INVALID
    assert copy(one, idx=_abi.SSU_F32) == INVALID
    assert copy(one, pairs=-1) == INVALID
    assert copy(one, src=None) == INVALID
    assert copy(one, pairs=0) == _abi.SSU_OK and err() == ""
    assert copy(pools((None, 0, 0))) == _abi.SSU_OK                       # no bytes to move
    assert lib.ssu_slots_clear(one, 1, 4, None, I32, 2, -1, None) == INVALID
    size = lib.ssu_slots_compact_workspace_bytes
    need = size(4, 2, 1)
    assert need > 0 and size(-1, 2, 0) == size(4, -1, 0) == -1
    assert size(4096, 8192, 0) == 0                          # one launch
    assert size(4097, 8192, 0) > 0 and size(4096, 8193, 0) > 0
    comp = lambda t=FAKE, ws=FAKE, n=need, live=FAKE, idx=I32, entries=2: (  # noqa: E731
        lib.ssu_slots_compact(one, 1, 4, t, FAKE, idx, entries, -1, live, ws, n, None))
    assert comp(n=need - 1) == INVALID and "workspace" in err()   # in place: two launches
    assert comp(ws=FAKE + 4) == INVALID
    assert comp(live=None) == INVALID
    assert comp(t=None) == INVALID
    assert comp(idx=_abi.SSU_BF16) == INVALID
    assert comp(entries=-1) == INVALID
