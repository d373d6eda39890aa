"""Sizes and slot ids at the ends of their range, where the host answers: no GPU."""
from __future__ import annotations

import subprocess
import sys

from mamba2_ssm_decode_gb300 import _abi

from .test_layer_abi_cpu import FAKE, INVALID


def test_linattn_workspace_of_any_sizes():
    """A query of sizes that no call takes is answered (a division by zero would end the
    process, so they are asked for in another)."""
    code = """
from mamba2_ssm_decode_gb300 import _abi
f = _abi.lib().ssu_linattn_workspace_bytes
big = [1, 2, 63, 64, 4096, 4097, 2**20, 2**31 - 1, 2**31, 2**40, 64 * (3 * 2**32 - 2), 2**62, 2**63 - 1]
for rows in big:
    for nseqs in big:
        for heads in [0] + big:
            assert f(rows, nseqs, heads, 64, 64, _abi.SSU_BF16) >= 0, (rows, nseqs, heads)
print("answered")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.split() == ["answered"], r.stderr[-500:]


def test_linattn_workspace_of_refused_sizes():
    f = _abi.lib().ssu_linattn_workspace_bytes
    for rows, nseqs, heads in ((2 ** 31 - 1024, 1, 1), (64, 2 ** 30, 1), (64, 1, 4097), (64, 1, 0)):
        assert f(rows, nseqs, heads, 64, 64, _abi.SSU_BF16) == 0


def test_assignment_refuses_a_pad_that_the_table_cannot_hold():
    """2^32 would be written into an int32 table as 0: a valid slot."""
    lib = _abi.lib()

    def call(pad, idx):
        return lib.ssu_slots_assign(FAKE, FAKE + 4096, idx, 0, 2, 8, pad, FAKE + 8192, FAKE + 12288,
                                    FAKE + 16384, None)

    for pad in (1 << 32, 1 << 31, -(1 << 31) - 1):
        assert call(pad, _abi.SSU_I32) == INVALID and "int32" in lib.ssu_last_error().decode()
