"""Linear attention over fp16 prompts, whose products are brought to the middle of
fp16's range by powers of two: values that are not finite, at the ends of the range,
and decays there."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import mamba2_ssm_decode_gb300 as ssu
from oracle import serving

from .test_layer_gpu import BF16, F16, F32, cu_of, gen, same_bits, within
from .test_serving_gpu import lin_inputs, lin_prompt

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mamba2_ssm_decode_gb300 import build
    build.build()
    yield
    assert ssu.ssu_device_error() == 0


def copied(i, rows, G, dk, H, dv):
    """The inputs on a projection of their own."""
    wide = i["q"].as_strided((rows, 2 * G * dk + H * dv), (i["q"].stride(0), 1), 0).clone()
    cut = lambda a, n, d: wide[:, a:a + n * d].unflatten(1, (n, d))  # noqa: E731
    return dict(i, q=cut(0, G, dk), k=cut(G * dk, G, dk), v=cut(2 * G * dk, H, dv),
                log_decay=i["log_decay"].clone())


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("name,at", [("q", 70), ("k", 70), ("v", 70), ("v", 5), ("v", 100), ("v", 129)])
@pytest.mark.parametrize("io,dk,dv", [(F16, 64, 64), (F16, 128, 128), (F16, 128, 64), (BF16, 64, 128)])
@pytest.mark.parametrize("lens,H", [([30, 100, 40], 4), ([30, 1500], 2)])
def test_bad_values_leave_the_rest_alone(name, at, bad, io, dk, dv, lens, H):
    """Rows before the value, the other sequences, and the heads (of v: the channels) that
    it does not touch have the bits of a call with a zero in its place; small values
    beside an fp32 state, in whole sequences and in pieces."""
    T, G = sum(lens), 2
    i = lin_inputs(T, H, G, dk, dv, len(lens), io, F32, seed=12)
    i["v"].mul_(2.0 ** -10)
    i["pool"].mul_(2.0 ** -10)
    i[name][at, 0 if name != "v" else 1, 17] = 0.0
    want, want_pool = lin_prompt(i, lens)
    j = copied(i, T, G, dk, H, dv)
    j[name][at, 0 if name != "v" else 1, 17] = bad
    got, pool = lin_prompt(j, lens)
    s = 0 if at < 30 else 1
    end = sum(lens[:s + 1])
    heads = [1] if name == "v" else list(range(H // G))
    clean = torch.ones(T, H, dv, dtype=torch.bool)
    state = torch.ones_like(pool.cpu(), dtype=torch.bool)
    for h in heads:
        if name == "v":
            clean[at:end, h, 17] = state[s, h, 17] = False
        elif name == "k":
            clean[at:end, h] = state[s, h] = False
        else:
            clean[at, h] = False
    same_bits(got.cpu()[clean], want.cpu()[clean])
    same_bits(pool.cpu()[state], want_pool.cpu()[state])
    assert not bool(torch.isfinite(got.cpu()[~clean]).any())
    if name == "v":
        assert not bool(torch.isfinite(pool[s, 1, 17]).any())


def test_weighed_values_over_the_whole_range():
    """A value that grows to 2^127 before its product with k is added, and one that shrinks
    to 2^-120: the state is the value within 2^-15 (an exponent of 111 to 136 is held to
    2^-17, the parts of a value near the largest one to 2^-22)."""
    rows, d = 64, 64
    for v0, total, k0 in ((60000.0, 77.0, 2.0 ** -10), (2.0 ** -10, -76.0, 1.0)):
        q, k, v = (torch.zeros(rows, 1, d, dtype=F16) for _ in range(3))
        v[0], k[0] = v0, k0
        v[0, 0, ::2] = v0 / 4
        ld = torch.full((rows, 1), total / 63)
        pool = torch.zeros(1, 1, d, d)
        i = dict(q=q, k=k, v=v, log_decay=ld, pool=pool)
        out, got = lin_prompt(i, [rows])
        want = v[0, 0].double() * k0 * math.exp(float(ld[1:].double().sum()))
        off = (got.cpu()[0, 0].double() / want[:, None] - 1.0).abs()
        assert float(off.max()) <= 2.0 ** -15, float(off.max())
        assert not bool(out.any())


def rows_check(i, lens, got, pool, init=None):
    """As the tolerances of prompts in chunks have it, and nothing for the size of the
    sums that an exponent comes from."""
    o, bound, size, after, off, written = serving.linattn(
        i["q"], i["k"], i["v"], i["log_decay"], i["q"].shape[2] ** -0.5, prompt=True,
        eps=2.0 ** -18, pool=i["pool"], nseqs=len(lens), cu=cu_of(lens), init=init)
    bound = bound + size * 2.0 ** -15
    # from half a unit above the largest number on (65520 in fp16), a rounding gives infinity
    most = torch.finfo(got.dtype).max * (1.0 + torch.finfo(got.dtype).eps / 4)
    g = got.cpu().double().numpy()
    beyond = np.abs(o) - bound >= most
    assert (g[beyond] == np.copysign(np.inf, o[beyond])).all()
    bound[np.abs(o) + bound >= most] = np.inf
    within(got, o, bound, "out")
    w = sorted(written)
    within(pool[w], after[w], off[w], "state")


@pytest.mark.parametrize("case", ["forget", "far", "tiny", "steep", "grow", "mixed", "most", "turns"])
@pytest.mark.parametrize("io,dk,dv", [(F16, 64, 64), (F16, 128, 128), (F16, 64, 128), (BF16, 128, 64)])
@pytest.mark.parametrize("lens,H", [([200, 33], 4), ([1500], 2)])
def test_decays_at_the_ends_of_the_range(case, io, dk, dv, lens, H):
    T = sum(lens)
    i = lin_inputs(T, H, H, dk, dv, len(lens), io, F32, seed=7)
    g = gen(10)
    ld = i["log_decay"]
    if case == "forget":            # everything before is gone
        ld[torch.rand(T, H, generator=g) < 0.1] = -math.inf
    elif case == "far":             # far below what fp32's exponential holds
        ld[torch.rand(T, H, generator=g) < 0.1] = -1e30
    elif case == "tiny":
        ld.mul_(1e-7)
    elif case == "steep":
        ld.mul_(200.0)
    elif case == "grow":            # a state that grows by e^2 over a chunk
        ld.fill_(2.0 / 64)
    elif case == "mixed":           # slow heads beside ones that forget at once
        ld[:, 0], ld[:, 1] = 0.0, -math.inf
        ld[::3, H - 2], ld[:, H - 1] = -90.0, -1e-9
    elif case == "most":            # nearly every row forgotten, then slow ones
        ld[:] = -math.inf
        ld[torch.arange(T) % 64 > 55] = -1e-3
    else:                           # growth by e^10 within 16 rows, and as much lost in the next
        ld[:] = torch.where(torch.arange(T) % 32 < 16, 10.0 / 16, -10.0 / 16)[:, None]
    got, pool = lin_prompt(i, lens)
    rows_check(i, lens, got, pool)


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
@pytest.mark.parametrize("lens", [[150], [1500]])
@pytest.mark.parametrize("state", ["large", "small"])
def test_states_far_from_one(dk, dv, lens, state):
    """A state beside which fp16 has no room, and values near its smallest, also in pieces."""
    by = 1e6 if state == "large" else 1e-5
    i = lin_inputs(lens[0], 2, 2, dk, dv, 1, F16, F32, "token", seed=11)
    i["log_decay"] = i["log_decay"] / 16
    i["pool"] = i["pool"] * by
    i["q"] = (i["q"].float() * (1e-6 if state == "large" else 1.0)).to(F16)
    if state == "small":
        i["v"] = (i["v"].float() * 1e-3).to(F16)
    got, pool = lin_prompt(i, lens)
    rows_check(i, lens, got, pool)
