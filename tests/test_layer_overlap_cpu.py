"""Which `out` the layer calls take and refuse, through the C ABI without a GPU: a
call without sequences makes every check and launches nothing."""
from __future__ import annotations

import random

import pytest

from mamba2_ssm_decode_gb300 import _abi

from .test_layer_abi_cpu import FAKE, INVALID, conv, decode, lib, prompt, scan  # noqa: F401

FAR = FAKE + (1 << 30)
F32, BF16 = _abi.SSU_F32, _abi.SSU_BF16


def taken(lib, p, rows, form):  # noqa: F811
    kind = "conv" if isinstance(p, _abi.ConvParams) else "scan"
    if form == "prompt":
        st = prompt(lib, f"ssu_{kind}_fwd_varlen", p, nseqs=0, rows=rows)
    else:
        st = decode(lib, f"ssu_{kind}_update", p, nseqs=0, rows=rows, cu=FAKE)
    if st == INVALID:
        assert "out must not overlap" in lib.ssu_last_error().decode()
        return False
    assert st == _abi.SSU_OK
    return True


def touched(at, stride, run, rows, pieces=1, piece_stride=0):
    return {at + r * stride + g * piece_stride + i for r in range(rows) for g in range(pieces)
            for i in range(run)}


@pytest.mark.parametrize("form", ["prompt", "decode"])
def test_conv_out_against_every_byte(lib, form):  # noqa: F811
    """Random rows and strides against the sets of bytes: shifted by rows, by
    columns, interleaved in one wider tensor, at other strides, broadcast."""
    r, C, seen = random.Random(1), 5, set()
    for _ in range(4000):
        rows = r.randint(1, 5)
        so = r.randint(C, 14)
        sx = r.choice([so, so, so, r.randint(0, 16)])
        at = r.randint(-40, 40)
        p = conv(x=FAKE, x_row_stride=sx, out=FAKE + 2 * at, out_row_stride=so, channels=C,
                 conv_state=FAR)
        free = not touched(0, 2 * sx, 2 * C, rows) & touched(2 * at, 2 * so, 2 * C, rows)
        same = form == "decode" and at == 0 and (rows == 1 or sx == so)
        assert taken(lib, p, rows, form) == (free or same), (rows, sx, so, at)
        seen.add((free, sx == so))
    assert len(seen) == 4


@pytest.mark.parametrize("form", ["prompt", "decode"])
@pytest.mark.parametrize("name", ["x", "dt", "z", "B", "C"])
def test_scan_out_against_every_byte(lib, form, name):  # noqa: F811
    r, dim, N, seen = random.Random(2), 4, 16, set()
    for _ in range(1500):
        rows, G = r.randint(1, 3), r.choice([1, 2])
        so, at = r.randint(dim, 50), r.randint(-60, 60)
        f32 = r.random() < 0.3            # a wider out
        eo = 4 if f32 else 2
        run, pieces, gs = (N, G, r.choice([N, N + 3])) if name in "BC" else (dim, 1, 0)
        s = so * eo // 2 if r.random() < 0.7 else r.randint(0, 60)
        over = {name: FAKE, f"{name}_row_stride": s}
        if name in "BC":
            over[f"{name}_group_stride"] = gs
        p = scan(**{**dict(state=FAR, x=FAR, dt=FAR, B=FAR, C=FAR, A=FAR, B_group_stride=N,
                           C_group_stride=N, channels=dim, ngroups=G, out=FAKE + 4 * at,
                           out_row_stride=so, out_dtype=F32 if f32 else BF16), **over})
        mine = touched(0, 2 * s, 2 * run, rows, pieces, 2 * gs)
        free = not mine & touched(4 * at, eo * so, eo * dim, rows)
        same = (form == "decode" and name not in "BC" and at == 0 and not f32 and
                (rows == 1 or s == so))
        assert taken(lib, p, rows, form) == (free or same), (rows, G, s, so, at, f32)
        seen.add(free)
    assert len(seen) == 2


def test_many_rows_are_not_looked_at_one_by_one(lib):  # noqa: F811
    p = conv(x=FAKE, x_row_stride=256, out=FAKE + 128, out_row_stride=256, conv_state=1 << 50)
    assert taken(lib, p, (1 << 31) - 2048, "prompt")
    p = conv(x=FAKE, x_row_stride=256, out=FAKE + 126, out_row_stride=256, conv_state=1 << 50)
    assert not taken(lib, p, (1 << 31) - 2048, "prompt")


def test_compaction_tables_that_overlap_in_part(lib):  # noqa: F811
    one = (_abi.Pool * 1)(_abi.Pool(FAR, 64, 64))

    def refused(table, out, entries, idx):
        st = lib.ssu_slots_compact(one, 1, 4, table, out, idx, entries, -1, FAR, None, 0, None)
        return st == INVALID and "not overlap" in lib.ssu_last_error().decode()

    assert refused(FAKE, FAKE + 4, 2, _abi.SSU_I32) and refused(FAKE + 8, FAKE, 2, _abi.SSU_I64)
    for table, out, n, idx in ((FAKE, FAKE, 2, _abi.SSU_I32), (FAKE + 8, FAKE, 3, _abi.SSU_I64)):
        want = table != out
        assert refused(table, out, n, idx) == want
