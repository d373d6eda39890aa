"""GPU parity of linear attention with a decay for each head, the verification of
drafted tokens, the maps of a batch and the assignment of slots with their oracle
(oracle/serving.py) on the same seeded inputs.

Tolerances, from the arithmetic:
  * linear attention row by row: the oracle's running bound (eps 2^-20 a step: a
    few fp32 roundings and a fast exponential), which grows with the chain, and
    dk products more for an output;
  * over prompts in chunks: a state is carried with eps 2^-18 -- the values'
    16-bit parts leave 2^-22, 12 products of 16 tokens add with at most 2^-23
    each, the exponentials of the weights are off by 2^-21.  An output's scores
    and state enter as two parts, to 2^-17 each, and the exponent of a score is
    the difference of two fp32 sums of at most A in size, so that it is off by
    2^-24 A twice: 2^-15 + 2^-23 A of the magnitude behind the output;
  * stored in 16 bits: half a unit in its last place more;
  * tokens, counts, maps, tables, untouched slots and rows: equal.
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import mamba2_ssm_decode_gb300 as ssu
from oracle import serving

from ._parity import graph_kernel_nodes
from .test_layer_gpu import BF16, DEV, F16, F32, cu_of, gen, same_bits, wide_copy, within

pytestmark = pytest.mark.gpu
I32, I64 = torch.int32, torch.int64


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mamba2_ssm_decode_gb300 import build
    build.build()
    yield
    assert ssu.ssu_device_error() == 0


# ---------------------------------------------------------------------------
# linear attention
# ---------------------------------------------------------------------------

def lin_inputs(rows, H=4, G=2, dk=64, dv=64, slots=8, io=BF16, state=F32, decay="token", seed=0,
               offset=0):
    """q, k and v as columns of one projection, `offset` columns into it."""
    g = gen(seed)
    wide = torch.randn(rows, offset + 2 * G * dk + H * dv, generator=g).to(io)
    cut = lambda a, n, d: wide[:, a:a + n * d].unflatten(1, (n, d))  # noqa: E731
    ld = None
    if decay == "token":
        ld = torch.nn.functional.logsigmoid(2 * torch.randn(rows, H, generator=g)) / 16
    elif decay == "head":
        ld = -torch.exp2(-8.0 * torch.arange(1, H + 1) / H)
    return dict(q=cut(offset, G, dk), k=cut(offset + G * dk, G, dk), v=cut(offset + 2 * G * dk, H, dv),
                log_decay=ld, pool=(0.5 * torch.randn(slots, H, dv, dk, generator=g)).to(state))


def on_gpu(i):
    """The operands with their strides, and the pool."""
    wide = wide_copy(i["q"])
    base = wide.as_strided((wide.untyped_storage().nbytes() // wide.element_size(),), (1,), 0)
    out = {}
    for n in ("q", "k", "v"):
        t = i[n]
        if t.untyped_storage().data_ptr() == i["q"].untyped_storage().data_ptr():
            out[n] = base.as_strided(t.shape, t.stride(), t.storage_offset())
            out[n].copy_(t)
        else:
            out[n] = t.to(DEV)
    out["log_decay"] = None if i["log_decay"] is None else i["log_decay"].to(DEV)
    out["pool"] = None if i["pool"] is None else i["pool"].to(DEV)
    return out


def tensor_cores(i):
    """Whether a prompt call goes to the tensor cores."""
    return (i["v"].dtype in (BF16, F16) and i["q"].shape[2] in (64, 128) and i["v"].shape[2] in (64, 128)
            and all(t.storage_offset() % 8 == 0 and all(s % 8 == 0 for s in t.stride()[:2])
                    for t in (i["q"], i["k"], i["v"])))


def lin_check(i, got, held, label, scale=None, prompt=False, rel=None, eps=None, **seqs):
    chunks = prompt and tensor_cores(i)
    eps = eps or 2.0 ** (-18 if chunks else -20)
    scale = i["q"].shape[2] ** -0.5 if scale is None else scale
    o, bound, size, after, off, written = serving.linattn(
        i["q"], i["k"], i["v"], i["log_decay"], scale, prompt=prompt, eps=eps, **seqs)
    if chunks:
        far = 0.0
        if i["log_decay"] is not None:
            ld = i["log_decay"].double().clamp(min=-111.0).nan_to_num(0.0)
            if ld.dim() == 1:
                far = 64 * float(ld.abs().max())
            else:
                far = float(torch.nn.functional.pad(ld.abs(), (0, 0, 0, 63)).unfold(0, 64, 1)
                            .sum(-1).max())
        bound = bound + size * (2.0 ** -15 + 2.0 ** -23 * 1.45 * far)
    has = within(got, o, bound, f"{label}: out")
    if held is not None:
        w = sorted(written)
        within(held[w], after[w], off[w], f"{label}: state")
        rest = [s for s in range(held.shape[0]) if s not in written]
        same_bits(held[rest], i["pool"][rest])
    return has


def lin_prompt(i, lens, slots=None, init=None, idx=I32, **kw):
    d = on_gpu(i)
    got = ssu.linattn_fwd_varlen(d["q"], d["k"], d["v"], cu_of(lens, idx).to(DEV),
                                 log_decay=d["log_decay"], state=d["pool"],
                                 state_batch_indices=None if slots is None else slots.to(idx).to(DEV),
                                 has_initial_state=None if init is None else init.to(DEV), **kw)
    return got, d["pool"]


@pytest.mark.parametrize("io,state", [(BF16, F32), (BF16, BF16), (F16, F16), (F16, F32), (F32, F32),
                                      (F32, BF16)])
@pytest.mark.parametrize("H,G,dk,dv", [(3, 3, 16, 5), (4, 2, 32, 64), (4, 1, 64, 33), (2, 2, 128, 128),
                                       (6, 2, 128, 64), (2, 1, 256, 256)])
@pytest.mark.parametrize("batch", [1, 7])
def test_linattn_one_token(io, state, H, G, dk, dv, batch):
    i = lin_inputs(batch, H, G, dk, dv, batch + 3, io, state, seed=dk + dv)
    slots = torch.randperm(batch + 3, generator=gen(2))[:batch]
    if batch > 3:
        slots[2] = -1       # runs from zeros, writes nothing
    d = on_gpu(i)
    got = ssu.linattn_update(d["pool"], d["q"], d["k"], d["v"], log_decay=d["log_decay"],
                             state_batch_indices=slots.to(I32).to(DEV))
    lin_check(i, got, d["pool"], "token", pool=i["pool"], nseqs=batch, src=slots[:, None], steps=1)


@pytest.mark.parametrize("form", ["packed", "dense", "flat", "dst", "no_tables", "accepted", "disabled",
                                  "int64", "odd_offset", "head_decay", "no_decay"])
@pytest.mark.parametrize("io,dk,dv", [(BF16, 128, 64), (F32, 64, 24), (F16, 16, 128)])
def test_linattn_drafts(form, io, dk, dv):
    lens = [3] * 5 if form == "dense" else [1, 4, 0, 2, 3]
    S, W, T, slots = len(lens), 4, sum(lens), 40
    decay = {"head_decay": "head", "no_decay": None}.get(form, "token")
    i = lin_inputs(T, 4, 2, dk, dv, slots, io, BF16, decay, seed=5, offset=form == "odd_offset")
    idx = I64 if form == "int64" else I32
    g = gen(8)
    table = torch.randperm(slots, generator=g)[:S * W].view(S, W)
    kw, seqs = {}, dict(nseqs=S, cu=cu_of(lens), pool=i["pool"])
    if form == "no_tables":
        pass
    elif form == "flat":
        flat = torch.randperm(slots, generator=g)[:S + W].clone()
        # sequence s's steps share entries with its neighbours': one token each
        lens = [1] * S
        seqs["cu"] = cu_of(lens)
        kw["state_batch_indices"] = seqs["src"] = flat
    else:
        table[1, 2] = -1
        kw["state_batch_indices"] = seqs["src"] = table
    if form == "dst":
        kw["dst_state_batch_indices"] = seqs["dst"] = torch.randperm(slots, generator=gen(9))[:S * W].view(S, W)
        kw["state_batch_indices"] = seqs["src"] = kw["dst_state_batch_indices"].flip(1).clone()
    if form == "accepted":
        acc = torch.tensor([1, 4, 2, 9, 2])     # 9: outside the table, runs from zeros
        kw["num_accepted_tokens"] = seqs["accepted"] = acc
    if form == "disabled":
        kw["disable_state_update"], seqs["write"] = True, False
    d = on_gpu(i)
    kw = {k: v.to(idx).to(DEV) if torch.is_tensor(v) else v for k, v in kw.items()}
    args = [d["q"], d["k"], d["v"]]
    if form == "dense":
        args = [t.contiguous().unflatten(0, (S, 3)) for t in args]
        d["log_decay"] = d["log_decay"].unflatten(0, (S, 3))
        seqs["cu"], seqs["steps"] = None, 3
    else:
        kw["cu_seqlens"] = seqs["cu"].to(idx).to(DEV)
    out = torch.full_like(args[2], 7.0)
    got = ssu.linattn_update_varlen(d["pool"], *args, log_decay=d["log_decay"], scale=0.25, out=out, **kw)
    assert got.shape == args[2].shape
    got = got.reshape(T, 4, dv)
    has = lin_check(i, got, d["pool"], form, scale=0.25, **seqs)
    rest = ~torch.from_numpy(has[:, 0, 0])
    assert bool((got.cpu()[rest] == 7.0).all())      # rows of no sequence are left as they were


LENS = [1, 0, 63, 64, 2, 65, 150, 0, 300, 129]


@pytest.mark.parametrize("io,state", [(BF16, F32), (BF16, BF16), (F16, F16), (F16, F32), (BF16, F16)])
@pytest.mark.parametrize("dk", [64, 128])
@pytest.mark.parametrize("dv", [64, 128])
@pytest.mark.parametrize("decay", ["token", "head", None])
def test_linattn_prompts(io, state, dk, dv, decay):
    """Packed prompts of 0 to 300 rows, half continued; a fresh sequence's slot holds
    NaN; rows behind the last sequence hold NaN and keep what is in `out`."""
    S, T, more = len(LENS), sum(LENS), 5
    i = lin_inputs(T + more, 4, 2, dk, dv, S + 2, io, state, decay, seed=dk + dv)
    i["q"][T:], i["k"][T:], i["v"][T:] = math.nan, math.nan, math.nan
    slots = torch.randperm(S + 2, generator=gen(1))[:S]
    init = torch.tensor([s % 2 == 1 for s in range(S)])
    clean = i["pool"].clone()
    for s in range(S):
        if not init[s] and LENS[s]:
            i["pool"][slots[s]] = math.nan
    out = torch.full((T + more, 4, dv), 7.0, dtype=io, device=DEV)
    got, pool = lin_prompt(i, LENS, slots, init, out=out)
    i["pool"] = clean
    trimmed = dict(i, q=i["q"][:T], k=i["k"][:T], v=i["v"][:T])
    if decay == "token":
        trimmed["log_decay"] = i["log_decay"][:T]
    lin_check(trimmed, got[:T], pool, "prompts", pool=clean, init=init, nseqs=S, cu=cu_of(LENS),
              src=slots, prompt=True)
    assert bool((got[T:] == 7.0).all())


@pytest.mark.parametrize("io,dk,dv,offset", [(F32, 64, 64, 0), (BF16, 32, 64, 0), (F16, 256, 16, 0),
                                             (BF16, 64, 40, 0), (BF16, 64, 64, 1), (F16, 128, 128, 4)])
def test_linattn_prompts_row_by_row(io, dk, dv, offset):
    """What the tensor cores do not take: other types, sizes, and rows off their vectors."""
    lens = [70, 0, 1, 33]
    i = lin_inputs(sum(lens), 4, 2, dk, dv, 6, io, F32, seed=3, offset=offset)
    assert not tensor_cores(i)
    slots, init = torch.tensor([4, 0, 2, 1]), torch.tensor([True, False, True, False])
    got, pool = lin_prompt(i, lens, slots, init)
    lin_check(i, got, pool, "rows", pool=i["pool"], init=init, nseqs=4, cu=cu_of(lens), src=slots,
              prompt=True)


@pytest.mark.parametrize("variant", ["no_pool", "dst", "pads", "int64", "strided_out", "odd_out",
                                     "wide_groups", "one_head", "contiguous", "scale", "shared_k"])
def test_linattn_prompt_variants(variant):
    lens, H, G, dk, dv = [40, 1, 0, 197, 70], 4, 2, 64, 128
    if variant == "wide_groups":
        H, G = 6, 1
    if variant == "one_head":
        H = G = 1
    S, T = len(lens), sum(lens)
    i = lin_inputs(T, H, G, dk, dv, 9, BF16, F32, seed=4)
    if variant == "contiguous":
        i.update({n: i[n].contiguous() for n in ("q", "k", "v")})
    if variant == "shared_k":
        i["q"] = i["k"]
    slots, init = torch.tensor([8, 3, 0, 5, 1]), torch.tensor([True, False, True, True, False])
    kw, seqs = {}, dict(init=init, src=slots, nseqs=S, cu=cu_of(lens), pool=i["pool"], prompt=True)
    if variant == "pads":
        slots[3] = -1
    if variant == "dst":
        seqs["dst"] = torch.tensor([2, 3, 4, -1, 6])
        kw["dst_state_batch_indices"] = seqs["dst"].to(I32).to(DEV)
    if variant == "no_pool":
        slots, i["pool"], init = None, None, None
        seqs.update(src=None, pool=None, init=None)
    if variant == "scale":
        kw["scale"] = -3.0
    if variant == "strided_out":
        kw["out"] = torch.full((H, T, 2 * dv), 7.0, dtype=BF16, device=DEV)[:, :, dv:].transpose(0, 1)
    if variant == "odd_out":
        kw["out"] = torch.full((T, H * dv + 3), 7.0, dtype=BF16, device=DEV)[:, 3:].unflatten(1, (H, dv))
    got, pool = lin_prompt(i, lens, slots, init, idx=I64 if variant == "int64" else I32, **kw)
    lin_check(i, got, pool, variant, scale=kw.get("scale"), **seqs)
    if variant == "strided_out":
        assert bool((got._base[:, :, :dv] == 7.0).all())


@pytest.mark.parametrize("lens", [[1500], [2049, 3], [5, 1100, 0, 900]])
@pytest.mark.parametrize("io,dk,dv,decay", [(BF16, 128, 128, "token"), (F16, 64, 64, None),
                                            (F16, 128, 64, "token"), (BF16, 64, 128, "head")])
def test_linattn_long_prompts(lens, io, dk, dv, decay):
    """Few heads and long sequences, which are cut into pieces."""
    S = len(lens)
    i = lin_inputs(sum(lens), 2, 1, dk, dv, S + 1, io, F32, decay, seed=6)
    slots, init = torch.arange(S).flip(0), torch.tensor([s % 2 == 0 for s in range(S)])
    got, pool = lin_prompt(i, lens, slots, init)
    lin_check(i, got, pool, "long", pool=i["pool"], init=init, nseqs=S, cu=cu_of(lens), src=slots,
              prompt=True)


@pytest.mark.parametrize("prompt", [True, False])
@pytest.mark.parametrize("case", ["forget", "far", "tiny", "steep", "grow", "mixed"])
def test_linattn_decays_at_the_ends_of_the_range(case, prompt):
    lens, H = [200, 33], 4
    T = sum(lens)
    i = lin_inputs(T, H, H, 64, 64, 2, BF16, F32, seed=7)
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
    else:                           # slow heads beside ones that forget at once
        ld[:, 0], ld[:, 1], ld[::3, 2], ld[:, 3] = 0.0, -math.inf, -90.0, -1e-9
    d = on_gpu(i)
    cu = cu_of(lens).to(DEV)
    if prompt:
        got = ssu.linattn_fwd_varlen(d["q"], d["k"], d["v"], cu, log_decay=d["log_decay"],
                                     state=d["pool"])
    else:
        table = torch.tensor([[0] * 200, [1] * 200], dtype=I32, device=DEV)
        got = ssu.linattn_update_varlen(d["pool"], d["q"], d["k"], d["v"], log_decay=d["log_decay"],
                                        cu_seqlens=cu, state_batch_indices=table)
    seqs = dict(pool=i["pool"], nseqs=2, cu=cu_of(lens))
    if not prompt:
        seqs["src"] = torch.tensor([[0] * 200, [1] * 200])
    lin_check(i, got, d["pool"], case, prompt=prompt, **seqs)


@pytest.mark.parametrize("io", [BF16, F16])
@pytest.mark.parametrize("state", ["large", "small"])
def test_linattn_states_far_from_one(io, state):
    """A state beside which fp16 has no room, and values near its smallest."""
    by = 1e6 if state == "large" else 1e-5
    i = lin_inputs(150, 2, 2, 64, 128, 1, io, F32, "token", seed=11)
    i["pool"] = i["pool"] * by
    i["q"] = (i["q"].float() * (1e-6 if state == "large" else 1.0)).to(io)
    if state == "small":
        i["v"] = (i["v"].float() * 1e-3).to(io)
    got, pool = lin_prompt(i, [150])
    lin_check(i, got, pool, state, pool=i["pool"], nseqs=1, cu=cu_of([150]), prompt=True)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("name,at", [("q", 70), ("k", 70), ("v", 70), ("v", 5), ("v", 100), ("log_decay", 70)])
def test_linattn_bad_values_stay_where_they_belong(name, at, bad):
    """Rows before a value that is not finite, the other sequences, and the heads (of
    v: the channels) that it does not touch have the bits of a clean call."""
    if name == "log_decay" and bad == -math.inf:
        pytest.skip("a decay of zero")
    lens = [30, 100, 40]
    i = lin_inputs(sum(lens), 4, 2, 64, 64, 3, BF16, F32, seed=12)
    want, want_pool = lin_prompt(i, lens)
    j = dict(i)
    # a copy of the projection, so that `i` stays clean
    wide = i["q"].as_strided((sum(lens), 2 * 2 * 64 + 4 * 64), (i["q"].stride(0), 1), 0).clone()
    cut = lambda a, n: wide[:, a:a + n * 64].unflatten(1, (n, 64))  # noqa: E731
    j.update(q=cut(0, 2), k=cut(128, 2), v=cut(256, 4), log_decay=i["log_decay"].clone())
    if name == "log_decay":
        j["log_decay"][at, 1] = bad
        heads = [1]
    elif name == "v":
        j["v"][at, 1, 17] = bad
        heads = [1]
    else:
        j[name][at, 0, 17] = bad
        heads = [0, 1]
    got, pool = lin_prompt(j, lens)
    s = 0 if at < 30 else 1
    end = (30, 130)[s]
    clean = torch.ones(sum(lens), 4, 64, dtype=torch.bool)
    for h in heads:
        if name == "v":
            clean[at:end, h, 17] = False
        elif name == "q":
            clean[at, h] = False
        else:
            clean[at:end, h] = False
    if name == "log_decay":
        # the earlier rows of its chunk (rows 30 to 93) take their exponents one by one then:
        # either way half a unit in the last place and far less from the exact value
        clean[30:at, 1] = False
        a, b = got.cpu()[30:at, 1].float(), want.cpu()[30:at, 1].float()
        assert float((a - b).abs().max()) <= 2.0 ** -7 * float(b.abs().max())
    same_bits(got.cpu()[clean], want.cpu()[clean])
    assert not bool(torch.isfinite(got.cpu()[at:at + 1][~clean[at:at + 1]]).any())
    others = [x for x in range(3) if x != s]
    same_bits(pool[others], want_pool[others])
    rest = [h for h in range(4) if h not in heads]
    same_bits(pool[s][rest], want_pool[s][rest])
    if name == "q":
        same_bits(pool, want_pool)


@pytest.mark.parametrize("io,dv", [(BF16, 128), (F16, 64)])
def test_linattn_prompt_then_tokens_is_one_prompt(io, dv):
    """A prompt, a continued prompt and two tokens, through a slot in fp32."""
    T, H = 200, 4
    i = lin_inputs(T, H, 2, 128, dv, 3, io, F32, seed=13)
    d = on_gpu(i)
    pool, slot = d["pool"], torch.tensor([2], dtype=I32, device=DEV)
    fresh = torch.zeros(1, dtype=torch.bool, device=DEV)
    cut = lambda a, b: (d["q"][a:b], d["k"][a:b], d["v"][a:b])  # noqa: E731
    got = []
    for a, b in ((0, 130), (130, 198)):
        got.append(ssu.linattn_fwd_varlen(*cut(a, b), cu_of([b - a]).to(DEV),
                                          log_decay=d["log_decay"][a:b], state=pool,
                                          state_batch_indices=slot,
                                          has_initial_state=fresh if a == 0 else None))
    for t in (198, 199):
        got.append(ssu.linattn_update(pool, *cut(t, t + 1), log_decay=d["log_decay"][t:t + 1],
                                      state_batch_indices=slot))
    lin_check(i, torch.cat(got), pool, "pieces", pool=i["pool"], init=[False], src=torch.tensor([2]),
              nseqs=1, cu=cu_of([T]), prompt=True)


def test_linattn_results_do_not_depend_on_the_batch_or_the_run():
    """A prompt alone and in a batch of 40, twice: the same bits (sequences that are not
    cut); no sum depends on which SM comes first."""
    i = lin_inputs(40 * 130, 8, 8, 64, 64, 40, BF16, F32, seed=14)
    a, pa = lin_prompt(i, [130] * 40)
    b, pb = lin_prompt(i, [130] * 40)
    same_bits(a, b)
    same_bits(pa, pb)
    one = dict(i, q=i["q"][130:260], k=i["k"][130:260], v=i["v"][130:260],
               log_decay=i["log_decay"][130:260], pool=i["pool"][1:2])
    c, pc = lin_prompt(one, [130])
    same_bits(a[130:260], c)
    same_bits(pa[1:2], pc)
    long = lin_inputs(4000, 2, 2, 64, 64, 1, BF16, F32, seed=15)
    x, px = lin_prompt(long, [4000])
    y, py = lin_prompt(long, [4000])
    same_bits(x, y)
    same_bits(px, py)


def test_linattn_offsets_beyond_32_bits():
    """Slots and rows whose element offsets pass 2^31."""
    H, dk, dv, slots = 32, 128, 128, 4200           # 2.2e9 elements
    g = torch.Generator(device=DEV).manual_seed(1)
    pool = torch.zeros(slots, H, dv, dk, dtype=BF16, device=DEV)
    pool[-1].normal_(generator=g)
    x = torch.randn(3, H, dk, generator=gen(1)).to(BF16)
    d, last = x.to(DEV), torch.tensor([slots - 1], dtype=I32, device=DEV)
    small = pool[-1:].clone()
    want = [ssu.linattn_update(small, d[:1], d[1:2], d[2:]),
            ssu.linattn_fwd_varlen(d, d, d, cu_of([3]).to(DEV), state=small)]
    got = [ssu.linattn_update(pool, d[:1], d[1:2], d[2:], state_batch_indices=last),
           ssu.linattn_fwd_varlen(d, d, d, cu_of([3]).to(DEV), state=pool, state_batch_indices=last)]
    for a, b in zip(got, want):
        same_bits(a, b)
    same_bits(pool[-1:], small)
    assert not bool(pool[:2].any())
    del pool
    # rows far apart: a stride of 2^25 elements, 70 rows
    wide = torch.zeros(70, 1 << 25, dtype=F16, device=DEV)
    y = torch.randn(70, 1, 64, generator=gen(2)).to(F16).to(DEV)
    far = wide[:, :64].unflatten(1, (1, 64))
    far.copy_(y)
    cu = cu_of([70]).to(DEV)
    same_bits(ssu.linattn_fwd_varlen(far, far, far, cu), ssu.linattn_fwd_varlen(y, y, y, cu))


def test_linattn_launches_graphs_and_streams():
    i = lin_inputs(4 * 70, 4, 2, 64, 64, 4, BF16, F32, seed=16)
    d, cu = on_gpu(i), cu_of([70] * 4).to(DEV)
    out = torch.empty(280, 4, 64, dtype=BF16, device=DEV)
    ws = torch.empty(ssu.linattn_workspace_bytes(280, 4, 4, 64, 64, BF16), dtype=torch.uint8, device=DEV)
    args = (d["q"], d["k"], d["v"])
    fwd = lambda pool, ws=ws, out=out: ssu.linattn_fwd_varlen(  # noqa: E731
        *args, cu, log_decay=d["log_decay"], state=pool, out=out, workspace=ws)
    upd = lambda: ssu.linattn_update(d["pool"], *(t[:4] for t in args), out=out[:4])  # noqa: E731
    assert graph_kernel_nodes(upd) == 1
    start = d["pool"].clone()
    # two captured prompts, each with its own workspace, replayed twice; an eager one as reference
    want_pool = start.clone()
    want = [fwd(want_pool, out=torch.empty_like(out)) for _ in range(2)]
    graphs, pools = [], [start.clone(), start.clone()]
    outs = [torch.empty_like(out) for _ in range(2)]
    for pool, o in zip(pools, outs):
        own = torch.empty_like(ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fwd(pool, own, o)
        graphs.append((g, own))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for step in range(2):
        graphs[0][0].replay()
        with torch.cuda.stream(side):
            graphs[1][0].replay()
        torch.cuda.synchronize()
        for o in outs:
            same_bits(o, want[step])
    for pool in pools:
        same_bits(pool, want_pool)
    # behind work on a side stream, with stream= and the results from that stream's memory
    busy = torch.zeros(1 << 28, device=DEV)
    late = {n: torch.zeros_like(t) for n, t in zip("qkv", args)}
    pool = start.clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            busy.add_(1.0)
        for n, t in zip("qkv", args):
            late[n].copy_(t)
    got = ssu.linattn_fwd_varlen(late["q"], late["k"], late["v"], cu, log_decay=d["log_decay"],
                                 state=pool, stream=side)
    side.synchronize()
    same_bits(got, want[0])


@pytest.mark.parametrize("io,dv", [(BF16, 128), (F16, 64)])
def test_linattn_captured_prompts_in_pieces(io, dv):
    """Launches that are set up while the one before runs, replayed: four kernel nodes, the
    bits of the eager call, also when the inputs change and when two graphs run at once."""
    lens, H = [2500, 40], 2
    i = lin_inputs(sum(lens), H, H, 64, dv, 2, io, F32, seed=17)
    d, cu = on_gpu(i), cu_of(lens).to(DEV)
    size = ssu.linattn_workspace_bytes(sum(lens), 2, H, dv, 64, io)

    def call(pool, ws, out):
        ssu.linattn_fwd_varlen(d["q"], d["k"], d["v"], cu, log_decay=d["log_decay"], state=pool,
                               out=out, workspace=ws)

    sets = [(d["pool"].clone(), torch.empty(size, dtype=torch.uint8, device=DEV),
             torch.empty(sum(lens), H, dv, dtype=io, device=DEV)) for _ in range(3)]
    assert graph_kernel_nodes(lambda: call(*sets[0])) == 4
    sets[0][0].copy_(d["pool"])
    graphs = []
    for s in sets[1:]:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call(*s)
    side = torch.cuda.Stream()
    for step in range(3):
        call(*sets[0])
        side.wait_stream(torch.cuda.current_stream())
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
        torch.cuda.synchronize()
        for s in sets[1:]:
            same_bits(s[2], sets[0][2])
            same_bits(s[0], sets[0][0])
        d["v"].mul_(-0.5)


def test_linattn_empty_and_refused():
    i = lin_inputs(6, 4, 2, 64, 64, 3)
    d = on_gpu(i)
    q, k, v, pool = d["q"], d["k"], d["v"], d["pool"]
    cu = cu_of([2, 4]).to(DEV)
    for n in (0, 3):
        z = torch.zeros(n + 1, dtype=I32, device=DEV)
        assert ssu.linattn_fwd_varlen(q[:0], k[:0], v[:0], z).shape == (0, 4, 64)
    assert ssu.linattn_update(pool, q[:0], k[:0], v[:0]).shape == (0, 4, 64)
    before = pool.clone()
    with pytest.raises(ValueError, match="overlap"):
        ssu.linattn_fwd_varlen(q, k, v, cu, out=v)
    with pytest.raises(ValueError, match="exceed"):
        ssu.linattn_fwd_varlen(q, k, v, cu_of([1] * 6).to(DEV), state=pool)
    with pytest.raises(ValueError, match="slots need the state pool"):
        ssu.linattn_fwd_varlen(q, k, v, cu, state_batch_indices=cu[:2])
    with pytest.raises(ValueError, match="cu_seqlens"):
        ssu.linattn_fwd_varlen(q, k, v, None)
    with pytest.raises(ValueError, match="overlap state"):
        ssu.linattn_update(pool, q[:3], k[:3], v[:3], out=pool.view(BF16)[0, 0].view(-1)[:768].view(3, 4, 64))
    with pytest.raises(ValueError, match="workspace"):
        ssu.linattn_fwd_varlen(q, k, v, cu, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError, match="share the v dtype"):
        ssu.linattn_update(pool, q[:3].float(), k[:3], v[:3])
    with pytest.raises(ValueError, match="state must be"):
        ssu.linattn_update(pool[:, :, :32].contiguous(), q[:3], k[:3], v[:3])
    with pytest.raises(ValueError, match="contiguous"):
        ssu.linattn_update(pool.transpose(2, 3), q[:3], k[:3], v[:3])
    with pytest.raises(ValueError, match="log_decay must be"):
        ssu.linattn_update(pool, q[:3], k[:3], v[:3], log_decay=torch.zeros(3, device=DEV))
    with pytest.raises(NotImplementedError, match="log_decay must be fp32"):
        ssu.linattn_update(pool, q[:3], k[:3], v[:3], log_decay=torch.zeros(4, dtype=BF16, device=DEV))
    with pytest.raises(ValueError, match="multiple of the groups"):
        ssu.linattn_update(pool, *(t[:3].repeat(1, 3, 1) for t in (q, k)), v[:3])
    with pytest.raises(NotImplementedError, match="dk 48"):
        ssu.linattn_fwd_varlen(q[:, :, :48], k[:, :, :48], v, cu)
    with pytest.raises(ValueError, match="needs state_batch_indices"):
        ssu.linattn_update_varlen(pool, q, k, v, cu_seqlens=cu, num_accepted_tokens=cu[1:])
    with pytest.raises(ValueError):
        ssu.linattn_update(pool, q[:3], k[:3], v[:3].cpu())
    same_bits(pool, before)


# ---------------------------------------------------------------------------
# verification
# ---------------------------------------------------------------------------

def draft_inputs(S, K, V, probs=F32, q=True, ragged=True, seed=0, sharp=2.0):
    g = gen(seed)
    n = torch.randint(0, K + 1, (S,), generator=g).tolist() if ragged else [K] * S
    cu = cu_of([m + 1 for m in n])
    rows = int(cu[-1])
    p = torch.softmax(sharp * torch.randn(rows, V, generator=g), 1).to(probs)
    dq = torch.softmax(sharp * torch.randn(S, K, V, generator=g), 2)
    for s in range(S):      # a draft model that mostly agrees
        for j in range(min(n[s], K)):
            dq[s, j] = torch.softmax((p[int(cu[s]) + j].float() + 1e-9).log()
                                     + 0.5 * torch.randn(V, generator=g), 0)
    drafts = torch.stack([torch.multinomial(dq[s] + 1e-12, 1, generator=g)[:, 0] for s in range(S)]) \
        if K else torch.zeros(S, 0, dtype=I64)
    return dict(p=p, drafts=drafts, u=torch.rand(S, K + 1, generator=g),
                q=dq.to(probs) if q else None, cu=cu if ragged else None)


def verify_check(i, greedy=None, idx=I32, ints=I32, **kw):
    got, n = ssu.drafts_verify(
        i["p"] if i["p"].is_cuda else i["p"].to(DEV), i["drafts"].to(idx).to(DEV), i["u"].to(DEV),
        draft_probs=None if i["q"] is None else i["q"].to(DEV),
        cu_seqlens=None if i["cu"] is None else i["cu"].to(ints).to(DEV),
        greedy=None if greedy is None else greedy.to(DEV), **kw)
    want, counts = serving.verify(i["p"], i["drafts"], i["u"], i["q"], i["cu"], greedy)
    assert got.dtype == idx and n.tolist() == counts
    assert got.tolist() == want
    return got, n


@pytest.mark.parametrize("probs", [F32, BF16, F16])
@pytest.mark.parametrize("V", [1, 2, 37, 1024, 5003, 33333])
@pytest.mark.parametrize("q", [True, False])
@pytest.mark.parametrize("K", [1, 4])
def test_verify(probs, V, q, K):
    S = 40 if V < 2000 else 6
    i = draft_inputs(S, K, V, probs, q, seed=V + K)
    verify_check(i, torch.arange(S) % 4 == 3)


@pytest.mark.parametrize("V", [16384, 16385, 65537, 131073, 300001, 1 << 19])
def test_verify_vocabularies_of_every_split(V):
    i = draft_inputs(2, 1, V, seed=V % 97, ragged=False)
    i["u"][:, -1] = torch.tensor([0.25, 0.999])
    verify_check(i, torch.tensor([False, False]))
    verify_check(i, torch.tensor([True, False]))


@pytest.mark.parametrize("form", ["dense", "int64", "out", "strided", "odd_rows", "no_rows", "no_drafts",
                                  "many"])
def test_verify_forms(form):
    S, K, V = (3000 if form == "many" else 9), (0 if form == "no_drafts" else 3), 101
    i = draft_inputs(S, K, V if form != "many" else 17, ragged=form != "dense", seed=3)
    kw = {}
    if form == "no_drafts":
        i["q"] = None
    if form == "no_rows":           # a sequence without rows, and rows behind the last one
        i["cu"] = torch.cat([i["cu"][:4], i["cu"][3:-1]])
    if form == "int64":
        kw.update(idx=I64, ints=I64)
    if form == "out":
        kw["out"] = torch.full((S, 2 * K + 9), 7, dtype=I32, device=DEV)[:, 2:K + 3]
        kw["num_accepted"] = torch.empty(S, dtype=I64, device=DEV)
    if form in ("strided", "odd_rows"):
        wide = torch.zeros(i["p"].shape[0], V + (7 if form == "strided" else 6), device=DEV)
        view = wide[:, 3:3 + V] if form == "strided" else wide[:, 1:V + 1]
        view.copy_(i["p"])
        got, n = ssu.drafts_verify(view, i["drafts"].to(I32).to(DEV), i["u"].to(DEV),
                                   draft_probs=i["q"].to(DEV), cu_seqlens=i["cu"].to(DEV))
        want = serving.verify(i["p"], i["drafts"], i["u"], i["q"], i["cu"])
        assert (got.tolist(), n.tolist()) == want
        return
    got, _ = verify_check(i, torch.arange(S) % 3 == 2, **kw)
    if form == "out":
        assert bool((got._base[:, :2] == 7).all()) and bool((got._base[:, K + 3:] == 7).all())


def test_verify_edges():
    """Random numbers at their ends, nothing left, drafts outside, ties, values that are
    no probabilities."""
    p = torch.tensor([[0.5, 0.0, 0.5, 0.0, 0.0], [0.2] * 5])
    q = p[None, :1].repeat(12, 1, 1).clone()
    q[6:] = torch.tensor([0.0, 0.5, 0.5, 0.0, 0.0])
    S = 12
    u = torch.rand(S, 2, generator=gen(1))
    u[0], u[1], u[2] = torch.tensor([0.0, 0.0]), torch.tensor([1 - 2 ** -24, 1 - 2 ** -24]), 0.5
    u[3], u[9] = torch.tensor([math.nan, math.nan]), torch.tensor([2.0, 2.0])
    u[10] = torch.tensor([-1.0, -1.0])
    drafts = torch.tensor([[0], [1], [2], [0], [7], [-3], [1], [2], [0], [2], [1], [4]])
    i = dict(p=p.repeat(S, 1), drafts=drafts, u=u, q=q, cu=None)
    verify_check(i)
    verify_check(dict(i, q=None))
    bad = i["p"].clone()
    bad[0], bad[2, 0], bad[4] = math.nan, math.nan, -1.0
    bad[6], bad[8, 2], bad[11] = 0.0, math.inf, torch.tensor([math.nan, 3.0, 3.0, -math.inf, 1.0])
    verify_check(dict(i, p=bad))
    verify_check(dict(i, p=bad), torch.ones(S, dtype=torch.bool))
    logits = torch.randn(2 * S, 5, generator=gen(2))
    logits[3] = -math.inf
    verify_check(dict(i, p=logits, drafts=logits[::2].argmax(1)[:, None]), torch.ones(S, dtype=torch.bool))


def test_verify_draws_as_the_sum_of_integers():
    """A long flat row, where a sum in fp32 would drift: the drawn token is exact."""
    V = 200000
    p = torch.full((8, V), 1.0 / V)
    u = torch.linspace(0, 1 - 2.0 ** -24, 8)[:, None].contiguous()
    i = dict(p=p, drafts=torch.zeros(8, 0, dtype=I64), u=u, q=None, cu=None)
    got, _ = verify_check(i)
    assert got[:, 0].tolist() == sorted(got[:, 0].tolist()) and got[-1, 0] == V - 1


def test_verify_refused_and_captured():
    i = draft_inputs(5, 2, 64, ragged=False)
    p, drafts, u, q = (i[n].to(DEV) for n in ("p", "drafts", "u", "q"))
    with pytest.raises(ValueError, match="cannot be split"):
        ssu.drafts_verify(p[:-1], drafts, u)
    with pytest.raises(ValueError, match="draft_probs must be"):
        ssu.drafts_verify(p, drafts, u, draft_probs=q[:, :1])
    with pytest.raises(ValueError, match="share the target_probs dtype"):
        ssu.drafts_verify(p, drafts, u, draft_probs=q.half())
    with pytest.raises(ValueError, match="uniform must be"):
        ssu.drafts_verify(p, drafts, u[:, :2])
    with pytest.raises(NotImplementedError, match="uniform must be fp32"):
        ssu.drafts_verify(p, drafts, u.double())
    with pytest.raises(ValueError, match="contiguous along"):
        ssu.drafts_verify(p.t().contiguous().t(), drafts, u)
    with pytest.raises(ValueError, match="greedy"):
        ssu.drafts_verify(p, drafts, u, greedy=u[:, 0])
    with pytest.raises(ValueError, match="draft_tokens' dtype"):
        ssu.drafts_verify(p, drafts, u, out=torch.empty(5, 3, dtype=I32, device=DEV))
    with pytest.raises(NotImplementedError, match="2\\^19"):
        ssu.drafts_verify(torch.zeros(3, (1 << 19) + 1, device=DEV), drafts[:1], u[:1])
    want = ssu.drafts_verify(p, drafts, u, draft_probs=q)
    out, n = torch.empty_like(want[0]), torch.empty_like(want[1])
    call = lambda: ssu.drafts_verify(p, drafts, u, draft_probs=q, out=out, num_accepted=n)  # noqa: E731
    assert graph_kernel_nodes(call) == 1
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(n, want[1])
    assert ssu.drafts_verify(p[:0], drafts[:0], u[:0])[0].shape == (0, 3)


# ---------------------------------------------------------------------------
# maps
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("ints", [I32, I64])
@pytest.mark.parametrize("chunk", [1, 16, 100, 256])
@pytest.mark.parametrize("S,rows", [(0, 5), (1, 0), (1, 700), (9, 500), (513, 3000), (3000, 9000)])
def test_prompt_maps(ints, chunk, S, rows):
    r = np.random.default_rng(S + chunk)
    for fill in (0.5, 1.0, 1.5):     # padded, filled, cut off
        lens = [int(v) for v in r.multinomial(int(rows * fill), np.ones(S) / S)] if S else []
        if S > 4:
            lens[2], lens[3] = 0, -5
        for context in (None, [int(c) for c in r.integers(0, 1000, S) * r.integers(0, 2, S)]):
            got = ssu.prompt_maps(torch.tensor(lens, dtype=ints, device=DEV), chunk, rows,
                                  context_lens=None if context is None else
                                  torch.tensor(context, dtype=ints, device=DEV))
            want = serving.prompt_maps(lens, chunk, rows, context, got.seq_idx.numel())
            for name, a, b in zip(got._fields, got, want):
                assert a.tolist() == b, name
            assert got.has_initial_state.dtype == torch.bool and got.cu_seqlens.dtype == ints
            again = ssu.prompt_maps(torch.tensor(lens, dtype=ints, device=DEV), chunk, rows, out=got)
            assert again is got


def test_prompt_maps_many_rows_and_refused():
    S, rows = 16384, 1 << 20
    lens = torch.randint(0, 64, (S,), generator=gen(1))
    got = ssu.prompt_maps(lens.to(I32).to(DEV), 64, rows)
    cu = torch.cat([torch.zeros(1, dtype=I64), lens.cumsum(0)])
    assert torch.equal(got.cu_seqlens.cpu().long(), cu)
    owner = torch.full((rows,), -1, dtype=I64)
    owner[:int(cu[-1])] = torch.repeat_interleave(torch.arange(S), lens)
    assert torch.equal(got.row_seq.cpu().long(), owner)
    lens = torch.tensor([3, 4], dtype=I32, device=DEV)
    call = lambda: ssu.prompt_maps(lens, 16, 9, out=held)  # noqa: E731
    held = ssu.prompt_maps(lens, 16, 9)
    assert graph_kernel_nodes(call) == 1
    with pytest.raises(ValueError, match="room for 1"):
        ssu.prompt_maps(lens, 16, 9, max_chunks=1)
    with pytest.raises(ValueError, match="chunk_size"):
        ssu.prompt_maps(lens, 0, 9)
    with pytest.raises(ValueError, match="row_seq must"):
        ssu.prompt_maps(lens, 16, 8, out=held)
    with pytest.raises(ValueError, match="lens' dtype"):
        ssu.prompt_maps(lens, 16, 9, context_lens=lens.long())
    with pytest.raises(ValueError, match="int32 or int64"):
        ssu.prompt_maps(lens.float(), 16, 9)
    with pytest.raises(NotImplementedError, match="16384"):
        ssu.prompt_maps(torch.zeros(16385, dtype=I32, device=DEV), 16, 9)


def test_maps_drive_the_ssd_prefill():
    """The SSD prefill from maps made on the GPU, in two pieces through its initial states,
    is the prefill of the whole prompts."""
    g, H, P, N, cs = gen(3), 2, 64, 64, 64
    lens, first = [150, 70, 1], [100, 30, 0]
    T = sum(lens)
    x = torch.randn(T, H, P, generator=g).to(BF16).to(DEV)
    dt = torch.rand(T, H, generator=g).to(DEV) * 0.1
    A = -torch.rand(H, generator=g).to(DEV)
    B, C = (torch.randn(T, 1, N, generator=g).to(BF16).to(DEV) for _ in range(2))

    def run(rows, lens, context, init):
        n = len(rows)
        m = ssu.prompt_maps(torch.tensor(lens, dtype=I32, device=DEV), cs, n,
                            context_lens=torch.tensor(context, dtype=I32, device=DEV))
        y = torch.empty(n, H, P, dtype=BF16, device=DEV)
        st = ssu.ssd_combined_fwd_varlen(x[rows], dt[rows].contiguous(), A, B[rows], C[rows], cs,
                                         m.cu_seqlens, m.cu_chunk_seqlens,
                                         m.last_chunk_indices, m.seq_idx, out=y,
                                         initial_states=init, state_dtype=F32)
        return y, st

    starts = [0, 150, 220]
    y, st = run(list(range(T)), lens, [0, 0, 0], None)
    a = [starts[s] + t for s in range(3) for t in range(first[s])]
    b = [starts[s] + t for s in range(3) for t in range(first[s], lens[s])]
    ya, sa = run(a, first, [0, 0, 0], None)
    yb, sb = run(b, [n - f for n, f in zip(lens, first)], first, sa)
    # chunks end at the same places, but for the state that is handed over in fp32: a state's
    # relative error is below 2^-8 (bf16 operands) and its outputs' as well, rounded once more
    for got, want in ((ya, y[a]), (yb, y[b]), (sb, st)):
        size = want.float().abs().max()
        assert float((got.float() - want.float()).abs().max()) <= 2.0 ** -6 * float(size)


# ---------------------------------------------------------------------------
# assignment
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("ints", [I32, I64])
@pytest.mark.parametrize("S,T,slots", [(0, 4, 9), (5, 1, 3), (20, 1, 48), (300, 4, 900), (1500, 5, 9000),
                                       (7, 0, 4), (9, 3, 0), (64, 1, 64), (70, 300, 70000),
                                       (300, 4, 32768), (300, 4, 32769), (2, 2, 40000)])
@pytest.mark.parametrize("pad", [-1, 0, 5])
def test_slots_assign(ints, S, T, slots, pad):
    r = np.random.default_rng(S + T + pad)
    ids = r.permutation(slots).tolist()
    table, counts = [], []
    for _ in range(S):
        counts.append(int(r.choice([0, T, r.integers(0, T + 1), T + 3, -1])))
        row = [ids.pop() if ids and r.random() < 0.4 else int(r.choice([pad, -1, slots, slots + 7]))
               for _ in range(T)]
        table.append(row)
    t = torch.tensor(table, dtype=ints, device=DEV).view(S, T)
    c = torch.tensor(counts, dtype=ints, device=DEV)
    want = serving.assign(table, counts, slots, pad)
    out, fresh, missing = ssu.slots_assign(t, c, slots, pad_slot_id=pad)
    assert (out.tolist(), fresh.tolist(), int(missing)) == want
    assert t.tolist() == table
    same, fresh, missing = ssu.slots_assign(t, c, slots, pad_slot_id=pad, out=t)
    assert same is t and (t.tolist(), fresh.tolist(), int(missing)) == want


def test_slots_assign_large_pool_and_refused():
    slots = 1 << 20
    t = torch.full((1 << 18, 4), -1, dtype=I32, device=DEV)
    c = torch.full((1 << 18,), 4, dtype=I32, device=DEV)
    out, fresh, missing = ssu.slots_assign(t, c, slots)
    assert torch.equal(out.view(-1).cpu(), torch.arange(slots, dtype=I32)) and int(missing) == 0
    out, _, missing = ssu.slots_assign(t, c, slots - 5, pad_slot_id=3)
    assert int(missing) == 6 and out.view(-1)[:5].tolist() == [0, 1, 2, 4, 5]
    t, c = t[:3], c[:3]
    held = ssu.slots_assign(t, c, 99)
    assert graph_kernel_nodes(lambda: ssu.slots_assign(t, c, 99, out=held[0], fresh=held[1],
                                                       num_missing=held[2])) == 1
    with pytest.raises(ValueError, match="overlap"):
        ssu.slots_assign(t, c, 99, out=held[0], fresh=held[0])
    with pytest.raises(ValueError, match="table must be"):
        ssu.slots_assign(t[:, ::2], c, 99)
    with pytest.raises(ValueError, match="counts must have"):
        ssu.slots_assign(t, c.long(), 99)
    with pytest.raises(ValueError, match="one int32"):
        ssu.slots_assign(t, c, 99, num_missing=torch.empty(2, dtype=I32, device=DEV))
    with pytest.raises(NotImplementedError, match="2\\^20"):
        ssu.slots_assign(t, c, slots + 1)


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

def test_a_serving_step_on_the_gpu():
    """Lengths in, tokens out: slots are assigned and cleared, prompts run from maps, drafted
    tokens run through a slot each, are verified, and the next drafts read the slot that the
    count names -- the same states as running the accepted tokens one by one."""
    S, H, dk, dv, K, V, slots = 5, 4, 64, 64, 3, 50, 32
    lens = [70, 3, 129, 1, 40]
    T, W = sum(lens), K + 1
    i = lin_inputs(T + S * W + S, H, H, dk, dv, slots, BF16, F32, "head", seed=21)
    d = on_gpu(i)
    pool, ld = d["pool"], d["log_decay"]
    cut = lambda a, b: (d["q"][a:b], d["k"][a:b], d["v"][a:b])  # noqa: E731
    table = torch.full((S, W), -1, dtype=I32, device=DEV)
    counts = torch.full((S,), W, dtype=I32, device=DEV)
    table, fresh, missing = ssu.slots_assign(table, counts, slots, out=table)
    ssu.slots_clear([pool], fresh.view(-1))
    maps = ssu.prompt_maps(torch.tensor(lens, dtype=I32, device=DEV), 64, T)
    first = table[:, 0].contiguous()
    ssu.linattn_fwd_varlen(*cut(0, T), maps.cu_seqlens, log_decay=ld, state=pool,
                           state_batch_indices=first, has_initial_state=maps.has_initial_state)
    after_prompt = pool[first.long()].clone()
    draft_cu = torch.arange(0, S * W + 1, W, dtype=I32, device=DEV)
    accepted = torch.ones(S, dtype=I32, device=DEV)
    rows = cut(T, T + S * W)
    ssu.linattn_update_varlen(pool, *rows, log_decay=ld, cu_seqlens=draft_cu,
                              num_accepted_tokens=accepted, state_batch_indices=table)
    v = draft_inputs(S, K, V, ragged=False, seed=22)
    tokens, n = ssu.drafts_verify(v["p"].to(DEV), v["drafts"].to(I32).to(DEV), v["u"].to(DEV),
                                  draft_probs=v["q"].to(DEV), cu_seqlens=draft_cu)
    assert (tokens.tolist(), n.tolist()) == serving.verify(v["p"], v["drafts"], v["u"], v["q"])
    assert int(missing) == 0 and len(set(n.tolist())) > 1
    # the row after the accepted ones reads the slot that the count names
    nxt = cut(T + S * W, T + S * W + S)
    got = ssu.linattn_update_varlen(pool, *nxt, log_decay=ld,
                                    cu_seqlens=torch.arange(S + 1, dtype=I32, device=DEV),
                                    num_accepted_tokens=n, state_batch_indices=table)
    one = after_prompt.clone()
    for s in range(S):
        for t in range(int(n[s])):
            ssu.linattn_update(one[s:s + 1], *(x[s * W + t:s * W + t + 1] for x in rows), log_decay=ld)
    want = ssu.linattn_update(one, *nxt, log_decay=ld)
    same_bits(got, want)
    same_bits(pool[first.long()], one)


def test_tables_and_maps_feed_the_other_layers():
    """The slots, starts and flags made on the GPU in the convolution's and the scan's calls."""
    lens, C, N, slots = [40, 0, 7], 32, 16, 8
    T, g = sum(lens), gen(4)
    x = torch.randn(T, C, generator=g).to(BF16).to(DEV)
    w = torch.randn(C, 4, generator=g).to(BF16).to(DEV)
    A = -torch.rand(C, N, generator=g).to(DEV)
    B, Cm = (torch.randn(T, N, generator=g).to(BF16).to(DEV) for _ in range(2))
    cp, sp = torch.randn(slots, 3, C, generator=g).to(BF16).to(DEV), torch.zeros(slots, C, N, device=DEV)
    maps = ssu.prompt_maps(torch.tensor(lens, dtype=I32, device=DEV), 64, T,
                           context_lens=torch.tensor([0, 0, 9], dtype=I32, device=DEV))
    table, _, _ = ssu.slots_assign(torch.tensor([[-1], [-1], [1]], dtype=I32, device=DEV),
                                   torch.ones(3, dtype=I32, device=DEV), slots)
    assert table.view(-1).tolist() == [0, 2, 1]
    host = dict(state_batch_indices=torch.tensor([0, 2, 1], dtype=I32, device=DEV),
                has_initial_state=torch.tensor([False, False, True], device=DEV))
    made = dict(state_batch_indices=table.view(-1), has_initial_state=maps.has_initial_state)
    cu = cu_of(lens).to(DEV)
    pools = [(cp.clone(), sp.clone()) for _ in range(2)]
    got = [[ssu.conv_fwd_varlen(x, w, c, conv_state=a, **kw),
            ssu.scan_fwd_varlen(x, x, A, B, Cm, c, dt_softplus=True, state=b, **kw)]
           for (a, b), kw, c in zip(pools, (host, made), (cu, maps.cu_seqlens))]
    for a, b in zip(*got):
        same_bits(a, b)
    for a, b in zip(*pools):
        same_bits(a, b)
