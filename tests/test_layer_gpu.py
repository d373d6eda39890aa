"""GPU parity of the convolution, the selective scan with a full A and the slot
moves with the fp64 oracle (oracle/layer.py) on the same seeded inputs.

Tolerances, from the arithmetic:
  * convolution: W fused multiply-adds and a bias in fp32, so |d| <= (W + 2)
    2^-24 times the sum of magnitudes; silu moves an error by at most 1.1 and
    adds a relative one of (|v| + 4) 2^-22 (its exponential's argument);
  * scan: the oracle's running bound, which grows with the chain;
  * an output or state stored in 16 bits: half a unit in its last place more
    (2^-8 bf16, 2^-11 fp16 relative, half the smallest subnormal for fp16);
  * cached convolution rows, copied slots, untouched slots: equal bits.
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import mamba2_ssm_decode_gb300 as ssu
from oracle import layer

from ._parity import graph_kernel_nodes

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
HALF_ULP = {F32: (0.0, 0.0), BF16: (2.0 ** -8, 0.0), F16: (2.0 ** -11, 2.0 ** -25)}
BITS = {F32: torch.int32, BF16: torch.int16, F16: torch.int16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mamba2_ssm_decode_gb300 import build
    build.build()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def within(got, ref, bound, label):
    """Where ref is a number and the bound finite, |got - ref| <= bound and half an ulp;
    returns where ref is a number."""
    rel, sub = HALF_ULP[got.dtype]
    g = got.detach().cpu().double().numpy()
    has = ~np.isnan(ref)
    # the stored value is the rounding of one that lies within `bound` of ref
    with np.errstate(invalid="ignore"):
        room = bound + rel * (np.abs(ref) + bound) + sub + 1e-37
        told = has & np.isfinite(room)
        worst = (np.abs(g - ref) / room)[told]
    assert np.isfinite(g[told]).all(), f"{label}: non-finite values"
    if worst.size:
        assert worst.max() <= 1.0, f"{label}: {worst.max():.3g}x the tolerance"
    return has


def same_bits(got, want):
    assert torch.equal(got.detach().cpu().contiguous().view(torch.uint8),
                       want.detach().cpu().contiguous().view(torch.uint8))


def cu_of(lens, dtype=torch.int32):
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=dtype)


# ---------------------------------------------------------------------------
# convolution
# ---------------------------------------------------------------------------

def conv_inputs(rows, C, W, slots, io=BF16, wt=None, seed=0, offset=0, extra=0):
    g = gen(seed)
    wide = torch.randn(rows, C + offset + extra, generator=g).to(io)
    return dict(x=wide[:, offset:offset + C],
                weight=(torch.randn(C, W, generator=g) / W).to(wt or io),
                bias=torch.randn(C, generator=g).to(wt or io),
                pool=torch.randn(slots, W - 1, C, generator=g).to(io))


def conv_check(i, got, held, act, label, **seqs):
    W = i["weight"].shape[1]
    y, after, mag = layer.conv(i["x"], i["weight"], i["bias"], act, **seqs)
    room = 1.1 * (W + 2) * 2.0 ** -24 * mag
    if act == "silu":   # the magnitudes bound the argument of silu
        room = room + np.abs(np.nan_to_num(y)) * (mag + 4) * 2.0 ** -22
    within(got, y, room, label)
    if held is not None:
        same_bits(held, torch.from_numpy(after).to(held.dtype))


def cuda(i, *names):
    return [None if i[n] is None else i[n].to(DEV) if i[n].is_contiguous()
            else wide_copy(i[n]) for n in names]


def wide_copy(t):
    """A column slice on the GPU with the strides and offset of `t`."""
    wide = torch.zeros(t.untyped_storage().nbytes() // t.element_size(), dtype=t.dtype, device=DEV)
    v = wide.as_strided(t.shape, t.stride(), t.storage_offset())
    v.copy_(t)
    return v


LENGTHS = [1, 0, 2, 3, 31, 4, 0, 70, 5, 129, 1, 16, 300, 33]


@pytest.mark.parametrize("io,wt", [(BF16, BF16), (BF16, F32), (F16, F16), (F16, F32), (F32, F32)])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("C", [64, 1030, 37])
def test_conv_prompts(io, wt, W, C):
    """Packed prompts of 0 to 300 rows, half continued; a fresh sequence's slot
    holds NaN, which must not get through; every channel count's vector width."""
    lens = LENGTHS
    S, T = len(lens), sum(lens)
    i = conv_inputs(T, C, W, S + 3, io, wt, seed=W + C)
    slots = torch.randperm(S + 3, generator=gen(7))[:S]
    init = torch.tensor([s % 2 == 0 for s in range(S)])
    for s in range(S):
        if not init[s]:
            i["pool"][slots[s]] = math.nan
    before = i["pool"].clone()
    x, w, b, pool = cuda(i, "x", "weight", "bias", "pool")
    got = ssu.conv_fwd_varlen(x, w, cu_of(lens).to(DEV), bias=b, conv_state=pool,
                              state_batch_indices=slots.to(DEV), has_initial_state=init.to(DEV))
    i["pool"] = before
    conv_check(i, got, None, "silu", "prompts", pool=before, init=init, nseqs=S, cu=cu_of(lens),
               src=slots, prompt=True)
    # the pool: NaN compares by bits
    _, after, _ = layer.conv(i["x"], i["weight"], i["bias"], "silu", pool=before, init=init, nseqs=S,
                             cu=cu_of(lens), src=slots, prompt=True)
    touched = [int(slots[s]) for s in range(S) if lens[s]]
    rest = [v for v in range(S + 3) if v not in touched]
    same_bits(pool[touched], torch.from_numpy(after[touched]).to(io))
    same_bits(pool[rest], before[rest])


@pytest.mark.parametrize("variant", ["no_pool", "no_bias", "no_act", "dst", "pads", "int64",
                                     "sliced", "sliced_odd", "no_table", "gaps", "all_init"])
def test_conv_prompt_variants(variant):
    lens, C, W = [40, 1, 2, 90, 0, 3], 136, 4
    S, T = len(lens), sum(lens)
    offset, extra = (24, 8) if variant == "sliced" else (3, 2) if variant == "sliced_odd" else (0, 0)
    i = conv_inputs(T, C, W, S + 2, seed=11, offset=offset, extra=extra)
    kw, seqs = {}, dict(nseqs=S, cu=cu_of(lens), prompt=True)
    slots = torch.tensor([5, 0, 3, 1, 7, 2])
    init = torch.tensor([True, False, True, True, True, False])
    act = None if variant == "no_act" else "silu"
    if variant == "no_bias":
        i["bias"] = None
    if variant == "pads":
        slots = torch.tensor([5, -1, 3, 99, 7, 2])
    if variant == "gaps":   # rows that no sequence has, in front and behind
        seqs["cu"] = torch.tensor([2, 40, 41, 50, 100, 100, 103])
        T = 136
    cu = seqs["cu"].to(torch.int64 if variant == "int64" else torch.int32).to(DEV)
    x, w, b, pool = cuda(i, "x", "weight", "bias", "pool")
    out = torch.full((i["x"].shape[0], C), 7.0, dtype=BF16, device=DEV)
    if variant == "no_pool":
        pool = None
    else:
        seqs["pool"] = i["pool"]
        kw["conv_state"] = pool
        if variant != "no_table":
            idx = torch.int64 if variant == "int64" else torch.int32
            kw["state_batch_indices"] = slots.to(idx).to(DEV)
            seqs["src"] = slots
        if variant != "all_init":
            kw["has_initial_state"] = init.to(DEV)
            seqs["init"] = init
        if variant == "dst":
            to = torch.tensor([6, 4, -1, 1, 0, 3])
            kw["dst_state_batch_indices"] = to.int().to(DEV)
            seqs["dst"] = to
    got = ssu.conv_fwd_varlen(x, w, cu, bias=b, activation=act, out=out, **kw)
    assert got is out
    conv_check(i, got, pool, act, variant, **seqs)
    y, _, _ = layer.conv(i["x"], i["weight"], i["bias"], act, **seqs)
    assert bool((out.cpu().float()[torch.from_numpy(np.isnan(y))] == 7.0).all())


@pytest.mark.parametrize("io", [BF16, F16, F32])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("C,batch", [(256, 5), (1030, 3), (37, 70), (4096, 1)])
def test_conv_one_token(io, W, C, batch):
    i = conv_inputs(batch, C, W, batch + 4, io, seed=C + W)
    slots = torch.randperm(batch + 4, generator=gen(3))[:batch]
    if batch > 2:
        slots[1] = -1
        slots[2] = batch + 50
    x, w, b, pool = cuda(i, "x", "weight", "bias", "pool")
    got = ssu.conv_update(pool, x, w, bias=b, state_batch_indices=slots.to(DEV))
    conv_check(i, got, pool, "silu", "one token", pool=i["pool"], nseqs=batch, src=slots[:, None])
    # into another slot, from x into x itself
    to = torch.arange(batch).flip(0)
    x, w, b, pool = cuda(i, "x", "weight", "bias", "pool")
    got = ssu.conv_update(pool, x, w, bias=b, activation=None, out=x, pad_slot_id=0,
                          state_batch_indices=slots.int().to(DEV),
                          dst_state_batch_indices=to.int().to(DEV))
    assert got is x
    # sequences that read a slot another one writes race: compare the rows and pads only
    y, _, mag = layer.conv(i["x"], i["weight"], i["bias"], None, pool=i["pool"], nseqs=batch,
                           src=slots[:, None], dst=to[:, None], pad=0)
    clear = [s for s in range(batch) if int(slots[s]) not in set(to.tolist()) - {int(to[s])}]
    within(got[clear], y[clear], (W + 2) * 2.0 ** -24 * mag[clear], "in place")


@pytest.mark.parametrize("io,C", [(BF16, 192), (F16, 50), (F32, 33)])
@pytest.mark.parametrize("form", ["table", "dense", "flat", "dst", "no_write"])
def test_conv_drafts(io, C, form):
    """A few drafted rows per sequence, a slot for each, read after the accepted ones."""
    S, W, steps = 9, 4, 6
    lens = [steps] * S if form == "dense" else [3, 1, 6, 0, 2, 5, 4, 1, 6]
    T = sum(lens)
    slots = S * steps + 5
    i = conv_inputs(T, C, W, slots, io, seed=5)
    ids = torch.randperm(slots, generator=gen(9))
    table = ids[:S * steps].view(S, steps).clone()
    table[2, 3] = -1
    table[5, 0] = 1000
    acc = torch.tensor([1, 6, 2, 1, 3, 1, 4, 6, 5])
    seqs, kw = dict(pool=i["pool"], nseqs=S), {}
    x, w, b, pool = cuda(i, "x", "weight", "bias", "pool")
    if form == "dense":
        x = x.view(S, steps, C)
        seqs["steps"] = steps
    else:
        seqs["cu"] = cu_of(lens)
        kw["cu_seqlens"] = seqs["cu"].to(DEV)
    if form == "flat":   # entry (s, t) of a flat table is s + t
        table = torch.arange(S)
        seqs["src"] = table
    else:
        seqs.update(src=table, accepted=acc)
        kw["num_accepted_tokens"] = acc.int().to(DEV)
    kw["state_batch_indices"] = table.int().to(DEV)
    if form == "flat":
        to = ids[ids >= S][:S].clone().view(S, 1)
        seqs["dst"] = to
        kw["dst_state_batch_indices"] = to.int().to(DEV)
    if form == "dst":
        to = torch.full((S, 8), -1)
        to[4, :2] = ids[S * steps:S * steps + 2]
        seqs["dst"] = to
        kw["dst_state_batch_indices"] = to.int().to(DEV)
    if form == "no_write":
        kw["disable_state_update"], seqs["write"] = True, False
    got = ssu.conv_update_varlen(pool, x, w, bias=b, **kw)
    if form == "dense":
        assert got.shape == (S, steps, C)
        got = got.view(T, C)
    conv_check(i, got, pool, "silu", form, **seqs)


# ---------------------------------------------------------------------------
# scan
# ---------------------------------------------------------------------------

def scan_inputs(rows, dim, N, slots, G=1, io=BF16, dt=None, state=F32, seed=0):
    g = gen(seed)
    step = torch.exp(torch.rand(dim, generator=g) * 4.6 - 6.9)
    return dict(
        x=torch.randn(rows, dim, generator=g).to(io), z=torch.randn(rows, dim, generator=g).to(io),
        dt=(0.5 * torch.randn(rows, dim, generator=g)).to(dt or io),
        A=-torch.arange(1, N + 1).float() * (0.5 + torch.rand(dim, N, generator=g)),
        B=torch.randn(rows, G, N, generator=g).to(io), C=torch.randn(rows, G, N, generator=g).to(io),
        D=torch.rand(dim, generator=g), dt_bias=step + torch.log(-torch.expm1(-step)),
        pool=(0.5 * torch.randn(slots, dim, N, generator=g)).to(state))


OPERANDS = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias")


def scan_check(i, got, held, label, softplus=True, **seqs):
    y, bound, after, off, written = layer.scan(
        i["x"], i["dt"], i["A"], i["B"], i["C"], D=i["D"], z=i["z"], dt_bias=i["dt_bias"],
        softplus=softplus, **seqs)
    has = within(got, y, bound, f"{label}: y")
    if held is not None:
        w = sorted(written)
        within(held[w], after[w], off[w], f"{label}: state")
        rest = [s for s in range(held.shape[0]) if s not in written]
        same_bits(held[rest], i["pool"][rest])
    return has


def scan_prompt(i, lens, slots=None, init=None, softplus=True, idx=torch.int32, **kw):
    d = dict(zip(OPERANDS, cuda(i, *OPERANDS)))
    pool = i["pool"].to(DEV) if i["pool"] is not None else None
    got = ssu.scan_fwd_varlen(d["x"], d["dt"], d["A"], d["B"], d["C"], cu_of(lens, idx).to(DEV),
                              D=d["D"], z=d["z"], dt_bias=d["dt_bias"], dt_softplus=softplus,
                              state=pool,
                              state_batch_indices=None if slots is None else slots.to(idx).to(DEV),
                              has_initial_state=None if init is None else init.to(DEV), **kw)
    return got, pool


PROMPTS = [1, 0, 33, 2, 64, 17, 150, 0, 3]


@pytest.mark.parametrize("io,dt,state", [(BF16, BF16, F32), (BF16, F32, BF16), (F16, F16, F16),
                                         (F16, F32, F32), (F32, F32, F32), (F32, F32, BF16)])
@pytest.mark.parametrize("N,dim,G", [(16, 160, 1), (16, 75, 1), (32, 72, 2), (64, 40, 4),
                                     (128, 24, 1), (256, 12, 3)])
def test_scan_prompts(io, dt, state, N, dim, G):
    """Packed prompts, half continued; a fresh sequence's slot holds NaN."""
    S, T = len(PROMPTS), sum(PROMPTS)
    i = scan_inputs(T, dim, N, S + 2, G, io, dt, state, seed=N + dim)
    slots = torch.randperm(S + 2, generator=gen(1))[:S]
    init = torch.tensor([s % 2 == 1 for s in range(S)])
    clean = i["pool"].clone()
    for s in range(S):
        if not init[s] and PROMPTS[s]:
            i["pool"][slots[s]] = math.nan
    got, pool = scan_prompt(i, PROMPTS, slots, init)
    i["pool"] = clean
    scan_check(i, got, pool, "prompts", pool=clean, init=init, nseqs=S, cu=cu_of(PROMPTS), src=slots,
               prompt=True)


@pytest.mark.parametrize("lens,dim", [([3000], 24), ([2049], 40), ([1500, 7], 16), ([700] * 3, 8),
                                      ([1023, 1, 513], 33)])
@pytest.mark.parametrize("N", [16, 32, 64, 128, 256])
def test_scan_long_prompts(lens, dim, N):
    """Long chains of few channels, from a slot and into it."""
    i = scan_inputs(sum(lens), dim, N, len(lens), 1, BF16, BF16, F32, seed=dim)
    got, pool = scan_prompt(i, lens)
    scan_check(i, got, pool, "long", pool=i["pool"], nseqs=len(lens), cu=cu_of(lens), prompt=True)


@pytest.mark.parametrize("variant", ["no_pool", "no_z", "no_D", "no_bias", "no_softplus",
                                     "raw_steps", "dst",
                                     "pads", "int64", "out_f32", "strided", "odd_strides", "two_d",
                                     "all_init", "gaps", "big_steps"])
@pytest.mark.parametrize("dim", [48, 29])
def test_scan_prompt_variants(variant, dim):
    lens, N, G = [40, 1, 0, 97, 5], 16, 1
    S, T = len(lens), sum(lens)
    i = scan_inputs(T, dim, N, S + 2, G, seed=21)
    kw, softplus = {}, True
    slots, init = torch.tensor([5, 0, 3, 1, 6]), torch.tensor([True, False, True, True, False])
    seqs = dict(pool=i["pool"], nseqs=S, cu=cu_of(lens), prompt=True)
    for name, key in (("no_z", "z"), ("no_D", "D"), ("no_bias", "dt_bias")):
        if variant == name:
            i[key] = None
    if variant == "no_softplus":   # with the negative bias: states that grow out of fp32's range
        softplus, i["dt"] = False, i["dt"].abs() * 0.1
    if variant == "raw_steps":
        softplus, i["dt"], i["dt_bias"] = False, i["dt"].abs() * 0.1, i["dt_bias"].abs() * 0.01
    if variant == "pads":
        slots = torch.tensor([5, -1, 3, 99, 6])
    if variant == "big_steps":   # softplus far from zero on both sides; decays that underflow
        i["dt"] = (40.0 * torch.randn(T, dim, generator=gen(2))).to(BF16)
    if variant in ("strided", "odd_strides"):
        pad = 16 if variant == "strided" else 5
        for k in ("x", "z", "dt"):
            i[k] = torch.cat([i[k], i[k][:, :pad]], 1)[:, :dim]
        for k in ("B", "C"):
            i[k] = torch.cat([i[k], i[k][:, :, :pad]], 2)[:, :, :N]
        i["A"] = torch.cat([i["A"], i["A"][:, :pad]], 1)[:, :N]
    if variant == "two_d":
        i["B"], i["C"] = i["B"][:, 0], i["C"][:, 0]
    if variant == "dst":
        to = torch.tensor([6, 4, 2, -1, 3])
        kw["dst_state_batch_indices"] = to.int().to(DEV)
        seqs["dst"] = to
    out = None
    if variant == "gaps":
        seqs["cu"] = torch.tensor([3, 40, 41, 41, 120, 121])
        lens = None
    if variant == "out_f32":
        kw["out_dtype"] = F32
    if variant == "no_pool":
        i["pool"] = None
        slots = init = None
        del seqs["pool"]
    else:
        seqs["src"] = slots
    if variant == "all_init":
        init = None
    if init is not None:
        seqs["init"] = init
    d = dict(zip(OPERANDS, cuda(i, *OPERANDS)))
    pool = None if i["pool"] is None else i["pool"].to(DEV)
    idx = torch.int64 if variant == "int64" else torch.int32
    if "out_dtype" not in kw:
        out = torch.full((T, dim), 7.0, dtype=BF16, device=DEV)
    got = ssu.scan_fwd_varlen(d["x"], d["dt"], d["A"], d["B"], d["C"], seqs["cu"].to(idx).to(DEV),
                              D=d["D"], z=d["z"], dt_bias=d["dt_bias"], dt_softplus=softplus,
                              state=pool, out=out,
                              state_batch_indices=None if slots is None else slots.to(idx).to(DEV),
                              has_initial_state=None if init is None else init.to(DEV), **kw)
    scan_check(i, got, pool, variant, softplus=softplus, **seqs)
    if out is not None:   # rows of no sequence
        cu = seqs["cu"].tolist()
        rest = [r for r in range(T) if not cu[0] <= r < cu[-1]]
        assert bool((got[rest] == 7.0).all())


@pytest.mark.parametrize("io,dt,state", [(BF16, BF16, F32), (BF16, F32, BF16), (F16, F16, F16),
                                         (F32, F32, F32)])
@pytest.mark.parametrize("N,dim,G,batch", [(16, 256, 1, 3), (16, 75, 3, 40), (32, 72, 2, 5),
                                           (64, 40, 4, 5), (128, 24, 1, 5), (256, 12, 3, 5)])
def test_scan_one_token(io, dt, state, N, dim, G, batch):
    i = scan_inputs(batch, dim, N, batch + 3, G, io, dt, state, seed=N)
    slots = torch.randperm(batch + 3, generator=gen(4))[:batch]
    slots[1], slots[2] = -1, batch + 9
    d = dict(zip(OPERANDS, cuda(i, *OPERANDS)))
    pool = i["pool"].to(DEV)
    got = ssu.scan_update(pool, d["x"], d["dt"], d["A"], d["B"], d["C"], D=d["D"], z=d["z"],
                          dt_bias=d["dt_bias"], dt_softplus=True, state_batch_indices=slots.to(DEV))
    scan_check(i, got, pool, "one token", pool=i["pool"], nseqs=batch, src=slots[:, None])


@pytest.mark.parametrize("form", ["table", "dense", "dst", "no_write", "one_row"])
@pytest.mark.parametrize("N,state", [(16, F32), (16, BF16), (64, F32)])
def test_scan_drafts(form, N, state):
    S, dim, steps = 9, 88, 6
    lens = [steps] * S if form == "dense" else [1] * S if form == "one_row" else [3, 1, 6, 0, 2, 5, 4, 1, 6]
    T, slots = sum(lens), S * steps + 5
    i = scan_inputs(T, dim, N, slots, 2, BF16, F32, state, seed=5)
    ids = torch.randperm(slots, generator=gen(9))
    table = ids[:S * steps].view(S, steps).clone()
    table[2, 3], table[5, 0] = -1, 1000
    acc = torch.tensor([1, 6, 2, 1, 3, 1, 4, 6, 5])
    seqs = dict(pool=i["pool"], nseqs=S, src=table, accepted=acc)
    kw = dict(state_batch_indices=table.int().to(DEV), num_accepted_tokens=acc.int().to(DEV))
    d = dict(zip(OPERANDS, cuda(i, *OPERANDS)))
    if form == "dense":
        seqs["steps"] = steps
        for k in ("x", "dt", "z", "B", "C"):
            d[k] = d[k].view(S, steps, *d[k].shape[1:])
    else:
        seqs["cu"] = cu_of(lens)
        kw["cu_seqlens"] = seqs["cu"].to(DEV)
    if form == "dst":
        to = torch.full((S, 2), -1)
        to[4], to[6, 1] = ids[S * steps:S * steps + 2], ids[S * steps + 3]
        seqs["dst"] = to
        kw["dst_state_batch_indices"] = to.int().to(DEV)
    if form == "no_write":
        kw["disable_state_update"], seqs["write"] = True, False
    pool = i["pool"].to(DEV)
    got = ssu.scan_update_varlen(pool, d["x"], d["dt"], d["A"], d["B"], d["C"], D=d["D"], z=d["z"],
                                 dt_bias=d["dt_bias"], dt_softplus=True, **kw)
    scan_check(i, got.view(T, dim), pool, form, **seqs)


def test_scan_prompt_then_tokens_is_one_prompt():
    """A prompt continued token by token gives what the whole prompt gives."""
    T, cut, dim, N = 96, 80, 64, 16
    i = scan_inputs(T, dim, N, 2, seed=3)
    i["pool"].zero_()
    d = dict(zip(OPERANDS, cuda(i, *OPERANDS)))
    pool = i["pool"].to(DEV)
    slot = torch.tensor([1], dtype=torch.int32, device=DEV)

    def rows(a, b):
        return [d[k][a:b] for k in ("x", "dt")] + [d["A"]] + [d[k][a:b] for k in ("B", "C")]

    kw = dict(D=d["D"], dt_bias=d["dt_bias"], dt_softplus=True, state_batch_indices=slot)
    got = [ssu.scan_fwd_varlen(*rows(0, cut), cu_of([cut]).to(DEV), z=d["z"][:cut], state=pool,
                               has_initial_state=torch.tensor([False], device=DEV), **kw)]
    for t in range(cut, T):
        got.append(ssu.scan_update(pool, *rows(t, t + 1), z=d["z"][t:t + 1], **kw))
    scan_check(i, torch.cat(got), pool, "pieces", pool=i["pool"], nseqs=1, cu=cu_of([T]),
               src=torch.tensor([1]), prompt=True)


def test_many_short_sequences():
    """More sequences than one probe finds, than are ranked by length, and than
    CTAs walk at once; several of a CTA's own one after another."""
    S, dim, N = 3000, 24, 16
    g = gen(8)
    lens = torch.randint(0, 4, (S,), generator=g).tolist()
    T = sum(lens)
    cu = cu_of(lens)
    slots = torch.randperm(S + 5, generator=g)[:S]
    slots[::9] = -1
    init = torch.rand(S, generator=g) < 0.5
    c = conv_inputs(T, dim, 4, S + 5, seed=1)
    x, w, b, pool = cuda(c, "x", "weight", "bias", "pool")
    got = ssu.conv_fwd_varlen(x, w, cu.to(DEV), bias=b, conv_state=pool, has_initial_state=init.to(DEV),
                              state_batch_indices=slots.to(DEV))
    conv_check(c, got, pool, "silu", "prompts", pool=c["pool"], nseqs=S, cu=cu, src=slots, init=init,
               prompt=True)
    i = scan_inputs(T, dim, N, S + 5, seed=1)
    d = dict(zip(OPERANDS, cuda(i, *OPERANDS)))
    got, pool = scan_prompt(i, lens, slots, init)
    scan_check(i, got, pool, "prompts", pool=i["pool"], nseqs=S, cu=cu, src=slots, init=init,
               prompt=True)
    # one token each: a row for every sequence
    c, i = conv_inputs(S, dim, 4, S + 5, seed=2), scan_inputs(S, dim, N, S + 5, seed=2)
    x, w, b, pool = cuda(c, "x", "weight", "bias", "pool")
    got = ssu.conv_update(pool, x, w, bias=b, state_batch_indices=slots.to(DEV))
    conv_check(c, got, pool, "silu", "tokens", pool=c["pool"], nseqs=S, src=slots[:, None])
    d = dict(zip(OPERANDS, cuda(i, *OPERANDS)))
    pool = i["pool"].to(DEV)
    got = ssu.scan_update(pool, d["x"], d["dt"], d["A"], d["B"], d["C"], D=d["D"], z=d["z"],
                          dt_bias=d["dt_bias"], dt_softplus=True, state_batch_indices=slots.to(DEV))
    scan_check(i, got, pool, "tokens", pool=i["pool"], nseqs=S, src=slots[:, None])


def test_conv_many_rows():
    """Enough rows for the largest row tiles; sequences that begin, end and lie
    inside them, and one of a single row at a tile's last."""
    C, lens = 2048, [63, 1, 20000, 2, 5, 40, 130, 18000, 7, 64, 3000]
    i = conv_inputs(sum(lens), C, 4, len(lens), seed=9)
    x, w, b, pool = cuda(i, "x", "weight", "bias", "pool")
    got = ssu.conv_fwd_varlen(x, w, cu_of(lens).to(DEV), bias=b, conv_state=pool)
    conv_check(i, got, pool, "silu", "many rows", pool=i["pool"], nseqs=len(lens), cu=cu_of(lens),
               prompt=True)


def test_operands_off_their_vectors():
    """weight, bias, B, C and A that do not start on 16 bytes."""
    c = conv_inputs(30, 64, 4, 2, seed=4)
    x, w, b, pool = cuda(c, "x", "weight", "bias", "pool")
    off = lambda t: torch.cat([t.flatten()[:1], t.flatten()])[1:].view(t.shape)  # noqa: E731
    got = ssu.conv_fwd_varlen(x, off(w), cu_of([30]).to(DEV), bias=off(b), conv_state=pool)
    conv_check(c, got, pool, "silu", "offset", pool=c["pool"], nseqs=1, cu=cu_of([30]), prompt=True)
    i = scan_inputs(30, 64, 16, 30, seed=4)
    d = dict(zip(OPERANDS, cuda(i, *OPERANDS)))
    d = {k: off(v) for k, v in d.items()}
    kw = dict(D=d["D"], z=d["z"], dt_bias=d["dt_bias"], dt_softplus=True)
    args = [d[k] for k in ("x", "dt", "A", "B", "C")]
    pool = i["pool"].to(DEV)
    got = ssu.scan_fwd_varlen(*args, cu_of([30]).to(DEV), state=pool, **kw)
    scan_check(i, got, pool, "offset", pool=i["pool"], nseqs=1, cu=cu_of([30]), prompt=True)
    pool = i["pool"].to(DEV)
    got = ssu.scan_update(pool, *args, **kw)
    scan_check(i, got, pool, "offset", pool=i["pool"], nseqs=30)


# ---------------------------------------------------------------------------
# slots
# ---------------------------------------------------------------------------

def make_pools(slots, seed=0):
    """Pools of every access width: wide rows, an odd number of bytes, one
    integer a slot, a strided pool, an empty slot."""
    g = gen(seed)
    strided = torch.randint(0, 255, (slots, 96), generator=g, dtype=torch.uint8)
    return [torch.randn(slots, 7, 16, 24, generator=g), torch.randn(slots, 3, 50, generator=g).half(),
            torch.randint(-9, 9, (slots,), generator=g, dtype=torch.int32),
            torch.randint(0, 255, (slots, 13), generator=g, dtype=torch.uint8),
            torch.randint(-9, 9, (slots, 5000), generator=g, dtype=torch.int64), strided[:, 8:41],
            torch.zeros(slots, 0)]


def on_gpu(pools):
    return [p.to(DEV) if p.is_contiguous() else wide_copy(p) for p in pools]


@pytest.mark.parametrize("idx", [torch.int32, torch.int64])
def test_slots_copy(idx):
    pools = make_pools(20)
    src = torch.tensor([3, 3, 3, 7, -1, 2, 19, 5, 25, 4, 0])
    dst = torch.tensor([1, 6, 8, 9, 10, -1, 11, 5, 12, 40, 13])   # a copy onto itself, pads, out of range
    gpu = on_gpu(pools)
    ssu.slots_copy(gpu, src.to(idx).to(DEV), dst.to(idx).to(DEV))
    for p, q in zip(pools, gpu):
        want = p.clone()
        for a, b in zip(src.tolist(), dst.tolist()):
            if 0 <= a < 20 and 0 <= b < 20:
                want[b] = p[a]
        same_bits(q, want)


def test_slots_copy_pad_inside_the_pool():
    pools = make_pools(6)[:1]
    gpu = on_gpu(pools)
    ssu.slots_copy(gpu, torch.tensor([0, 2], device=DEV), torch.tensor([1, 3], device=DEV), pad_slot_id=0)
    want = pools[0].clone()
    want[3] = pools[0][2]
    same_bits(gpu[0], want)


def test_slots_clear():
    pools = make_pools(12, seed=1)
    gpu = on_gpu(pools)
    ssu.slots_clear(gpu, torch.tensor([4, -1, 11, 30, 4], device=DEV))
    for p, q in zip(pools, gpu):
        want = p.clone()
        want[[4, 11]] = 0
        same_bits(q, want)
    ssu.slots_clear(gpu, torch.zeros(0, dtype=torch.int32, device=DEV))   # nothing to do


@pytest.mark.parametrize("slots,live,pads", [(1, 0, 2), (1, 1, 0), (40, 17, 4), (64, 64, 0),
                                             (65, 1, 3), (200, 0, 5), (1000, 500, 30), (3000, 2900, 0)])
@pytest.mark.parametrize("idx", [torch.int32, torch.int64])
def test_slots_compact(slots, live, pads, idx):
    g = gen(slots + live)
    pools = [torch.randn(slots, 40, generator=g), torch.arange(slots, dtype=torch.int32),
             torch.randint(0, 255, (slots, 7), generator=g, dtype=torch.uint8)]
    held = torch.randperm(slots, generator=g)[:live]
    if live > 3:   # a slot entered twice, one out of range
        held = torch.cat([held, held[:2], torch.tensor([slots + 5])])
    table = torch.cat([held, torch.full((pads,), -1)])
    table = table[torch.randperm(len(table), generator=g)].to(idx)
    want, m, moves = layer.compact(table.numpy(), slots)
    gpu = on_gpu(pools)
    out, count = ssu.slots_compact(gpu, table.to(DEV))
    assert out.cpu().tolist() == want.tolist() and count.tolist() == [m] == [live]
    for p, q in zip(pools, gpu):
        ref = p.clone()
        for a, b in moves.items():
            ref[b] = p[a]
        same_bits(q, ref)
    # in place, with a workspace of the caller's
    gpu, t = on_gpu(pools), table.to(DEV)
    need = ssu.slots_compact_workspace_bytes(slots, t.numel(), in_place=True)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    out, _ = ssu.slots_compact(gpu, t, out=t, workspace=ws)
    assert out is t and t.cpu().tolist() == want.tolist()


def test_slots_compact_many_slots():
    """More slots than the plan has threads and words, a [S, T] table."""
    slots, S, T = 1 << 20, 5000, 4
    table = torch.randperm(slots, generator=gen(3))[:S * T].view(S, T).int()
    table[::7, 3] = -1
    pool = torch.arange(slots, dtype=torch.int32)
    want, m, moves = layer.compact(table.numpy(), slots)
    p = pool.to(DEV)
    out, count = ssu.slots_compact([p], table.to(DEV))
    assert torch.equal(out.cpu(), torch.from_numpy(want).int()) and int(count) == m
    ref = pool.clone()
    ref[list(moves.values())] = torch.tensor(list(moves.keys()), dtype=torch.int32)
    assert torch.equal(p.cpu(), ref)


def test_many_pools():
    pools = [torch.full((4, 1 + i % 5), float(i), device=DEV) for i in range(256)]
    for i, p in enumerate(pools):
        p[2] = -i - 1.0
    ids = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    ssu.slots_copy(pools, ids(2, 2), ids(0, 3))
    for i, p in enumerate(pools):
        assert p[0].eq(-i - 1).all() and p[3].eq(-i - 1).all() and p[1].eq(i).all()
    with pytest.raises(NotImplementedError, match="256 pools"):
        ssu.slots_copy(pools + pools[:1], ids(2), ids(0))


# ---------------------------------------------------------------------------
# where offsets pass 32 bits
# ---------------------------------------------------------------------------

def test_offsets_beyond_32_bits():
    """Pools of more than 2^32 bytes and 2^31 elements: the last slots."""
    slots, dim, N = 1100, 8192, 256   # 2.3e9 elements, 4.6 GB in bf16
    pool = torch.zeros(slots, dim, N, dtype=BF16, device=DEV)
    i = scan_inputs(2, dim, N, 2, seed=1, state=BF16)
    at = torch.tensor([slots - 1, 0])
    pool[at.to(DEV)] = i["pool"].to(DEV)
    d = dict(zip(OPERANDS, cuda(i, *OPERANDS)))
    got = ssu.scan_update(pool, d["x"], d["dt"], d["A"], d["B"], d["C"], D=d["D"], z=d["z"],
                          dt_bias=d["dt_bias"], dt_softplus=True, state_batch_indices=at.to(DEV))
    scan_check(i, got, pool[at.to(DEV)], "large pool", pool=i["pool"], nseqs=2)
    src = torch.tensor([slots - 1], device=DEV)
    ssu.slots_copy([pool], src, torch.tensor([slots - 2], device=DEV))
    assert torch.equal(pool[slots - 2], pool[slots - 1])
    out, _ = ssu.slots_compact([pool], src)
    assert out.tolist() == [0] and torch.equal(pool[0], pool[slots - 1])
    rows = pool.view(-1)[:90000 * 3 * 8192].view(90000, 3, 8192)   # the same memory as convolution rows
    last = torch.tensor([rows.shape[0] - 1])
    c = conv_inputs(1, 8192, 4, 1, seed=2)
    rows[-1] = c["pool"][0].to(DEV)
    x, w, b = cuda(c, "x", "weight", "bias")
    got = ssu.conv_update(rows, x, w, bias=b, state_batch_indices=last.to(DEV))
    conv_check(c, got, rows[-1:], "silu", "large pool", pool=c["pool"], nseqs=1)


# ---------------------------------------------------------------------------
# streams, graphs, launches, refusals
# ---------------------------------------------------------------------------

def test_each_call_is_its_stated_launches():
    i = scan_inputs(50, 64, 16, 4)
    d = dict(zip(OPERANDS, cuda(i, *OPERANDS)))
    pool, cu, out = i["pool"].to(DEV), cu_of([30, 20]).to(DEV), torch.empty_like(d["x"])
    kw = dict(D=d["D"], z=d["z"], dt_bias=d["dt_bias"], dt_softplus=True, out=out)
    args = [d[k] for k in ("x", "dt", "A", "B", "C")]
    assert graph_kernel_nodes(lambda: ssu.scan_fwd_varlen(*args, cu, state=pool, **kw)) == 1
    assert graph_kernel_nodes(lambda: ssu.scan_update_varlen(pool, *args, cu_seqlens=cu, **kw)) == 1
    c = conv_inputs(50, 64, 4, 4)
    x, w, b, cp = cuda(c, "x", "weight", "bias", "pool")
    assert graph_kernel_nodes(lambda: ssu.conv_fwd_varlen(x, w, cu, bias=b, conv_state=cp, out=out)) == 1
    assert graph_kernel_nodes(
        lambda: ssu.conv_update_varlen(cp, x, w, bias=b, cu_seqlens=cu, out=out)) == 1
    t = torch.tensor([3, 1], dtype=torch.int32, device=DEV)
    to, n = torch.empty_like(t), torch.empty(1, dtype=torch.int32, device=DEV)
    ws = torch.empty(ssu.slots_compact_workspace_bytes(4, 2, True), dtype=torch.uint8, device=DEV)
    assert graph_kernel_nodes(lambda: ssu.slots_copy([pool, cp], t[:1], t[1:])) == 1
    assert graph_kernel_nodes(lambda: ssu.slots_clear([pool, cp], t)) == 1
    assert graph_kernel_nodes(
        lambda: ssu.slots_compact([pool, cp], t, out=to, num_live=n, workspace=ws)) == 1
    assert graph_kernel_nodes(
        lambda: ssu.slots_compact([pool, cp], t, out=t, num_live=n, workspace=ws)) == 2   # in place


def test_calls_run_on_the_given_stream():
    """Work queued behind a long kernel on a side stream is ordered after it."""
    s = torch.cuda.Stream()
    c = conv_inputs(64, 256, 4, 2, io=F32)
    x, w, b, pool = cuda(c, "x", "weight", "bias", "pool")
    busy = torch.zeros(1 << 28, device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(10):
            busy.add_(1.0)
        x.mul_(2.0)
        got = ssu.conv_fwd_varlen(x, w, cu_of([40, 24]).to(DEV), bias=b, conv_state=pool)
        ssu.slots_copy([pool], torch.tensor([0], device=DEV), torch.tensor([1], device=DEV))
    s.synchronize()
    c["x"] = c["x"] * 2.0
    conv_check(c, got, None, "silu", "side stream", pool=c["pool"], nseqs=2, cu=cu_of([40, 24]),
               prompt=True)
    assert torch.equal(pool[0], pool[1])


def test_empty_calls():
    c, i = conv_inputs(0, 16, 4, 2), scan_inputs(0, 16, 16, 2)
    x, w, b, pool = cuda(c, "x", "weight", "bias", "pool")
    d = dict(zip(OPERANDS, cuda(i, *OPERANDS)))
    args = [d[k] for k in ("x", "dt", "A", "B", "C")]
    for n in (0, 3):
        cu = torch.zeros(n + 1, dtype=torch.int32, device=DEV)
        assert ssu.conv_fwd_varlen(x, w, cu, bias=b).shape == (0, 16)
        assert ssu.scan_fwd_varlen(*args, cu).shape == (0, 16)
    assert ssu.conv_update(pool, x, w, bias=b).shape == (0, 16)
    assert ssu.scan_update(i["pool"].to(DEV), *args).shape == (0, 16)


def test_refusals():
    c = conv_inputs(6, 32, 4, 3)
    x, w, b, pool = cuda(c, "x", "weight", "bias", "pool")
    cu = cu_of([2, 4]).to(DEV)
    with pytest.raises(ValueError, match="overlap"):
        ssu.conv_fwd_varlen(x, w, cu, bias=b, out=x)
    with pytest.raises(ValueError, match="exceed"):
        ssu.conv_fwd_varlen(x, w, cu_of([1] * 6).to(DEV), conv_state=pool)
    with pytest.raises(ValueError, match="slots need the state pool"):
        ssu.conv_fwd_varlen(x, w, cu, state_batch_indices=cu[:2])
    with pytest.raises(ValueError, match="activation"):
        ssu.conv_update(pool, x[:3], w, activation="relu")
    with pytest.raises(NotImplementedError, match="width 5"):
        ssu.conv_update(torch.zeros(3, 4, 32, dtype=BF16, device=DEV), x[:3],
                        torch.zeros(32, 5, dtype=BF16, device=DEV))
    with pytest.raises(ValueError, match="conv_state must be"):
        ssu.conv_update(pool[:, :2].contiguous(), x[:3], w)
    with pytest.raises(ValueError, match="weight must be"):
        ssu.conv_update(pool, x[:3], w.half())
    with pytest.raises(ValueError, match="needs state_batch_indices"):
        ssu.conv_update_varlen(pool, x, w, cu_seqlens=cu, num_accepted_tokens=cu[1:])
    with pytest.raises(ValueError, match="contiguous along channels"):
        ssu.conv_update(pool, x.repeat(1, 2)[:3, ::2], w)
    with pytest.raises(ValueError, match="has_initial_state"):
        ssu.conv_fwd_varlen(x, w, cu, conv_state=pool, has_initial_state=cu[:2])
    i = scan_inputs(6, 32, 16, 3)
    d = dict(zip(OPERANDS, cuda(i, *OPERANDS)))
    args = [d[k] for k in ("x", "dt", "A", "B", "C")]
    sp = i["pool"].to(DEV)
    with pytest.raises(ValueError, match="overlap"):
        ssu.scan_fwd_varlen(*args, cu, out=d["x"])
    with pytest.raises(NotImplementedError, match="dstate 24"):
        ssu.scan_fwd_varlen(d["x"], d["dt"], *[torch.zeros(n, 24, device=DEV, dtype=t) for n, t in
                                               ((32, F32), (6, BF16), (6, BF16))], cu)
    with pytest.raises(NotImplementedError, match="A must be"):
        ssu.scan_update(sp, args[0][:3], args[1][:3], d["A"].bfloat16(), args[3][:3], args[4][:3])
    with pytest.raises(ValueError, match="state must be contiguous"):
        ssu.scan_update(torch.zeros(3, 32, 32, device=DEV)[:, :, :16], args[0][:3], args[1][:3], d["A"],
                        args[3][:3], args[4][:3])
    with pytest.raises(ValueError, match="share the x dtype"):
        ssu.scan_fwd_varlen(d["x"], d["dt"], d["A"], d["B"].float(), d["C"], cu)
    with pytest.raises(ValueError, match="multiple of ngroups"):
        ssu.scan_fwd_varlen(d["x"], d["dt"], d["A"], *[d[k].repeat(1, 3, 1) for k in ("B", "C")], cu)
    with pytest.raises(ValueError, match="dt must be"):
        ssu.scan_fwd_varlen(d["x"], d["dt"].half(), *args[2:], cu)
    with pytest.raises(ValueError, match="hold 3 slots"):
        ssu.slots_copy([sp, pool[:2]], cu[:1], cu[:1])
    with pytest.raises(ValueError, match="share their length"):
        ssu.slots_copy([sp], cu[:2], cu[:1])
    with pytest.raises(ValueError, match="slot must be contiguous"):
        ssu.slots_clear([sp.transpose(1, 2)], cu[:1])
    with pytest.raises(ValueError, match="workspace"):
        ssu.slots_compact([sp], cu, out=cu, workspace=torch.empty(8, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError, match="int32 or int64"):
        ssu.slots_compact([sp], cu.float())
    assert ssu.ssu_device_error() == 0
