"""Cases and plain forms of the operators around the state update: the short
causal convolution, the selective scan with a full A, and the moves of state
slots between and inside the pools.

`own` False: each operator in elementary torch operations, in fp32, rounded
once.  `own` True: the same call through the package's entry points.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BITS = {4: torch.int32, 2: torch.int16, 1: torch.uint8}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one user's short prompt, into a fresh slot; x is a column slice of the input projection
        dict(name="conv-prompt-one", op="conv_prompt", seqs=1, tokens=37, channels=5376, width=4,
             io="bf16", silu=True, sliced=True, steps=2048),
        # a packed batch of prompts, half of them continued from an earlier piece
        dict(name="conv-prompt-batch", op="conv_prompt", seqs=16, tokens=20634, channels=5376,
             width=4, io="bf16", silu=True, sliced=True, steps=2048),
        # one user's next token: a call that is all latency
        dict(name="conv-token-one", op="conv_token", seqs=1, steps=1, channels=5376, width=4,
             io="bf16", silu=True, sliced=True),
        # speculative decoding of a full batch: 1 to 4 drafted tokens a sequence, a slot for each
        dict(name="conv-token-drafts", op="conv_token", seqs=256, steps=4, channels=5376, width=4,
             io="bf16", silu=True, sliced=True),
        # one long document, of an odd length: few rows, a long axis
        dict(name="scan-prompt-long", op="scan_prompt", seqs=1, tokens=12289, channels=5120,
             dstate=16, groups=1, io="bf16", dt="bf16", state="f32", steps=12289),
        # a packed batch of prompts of 16 lengths, half of them continued
        dict(name="scan-prompt-batch", op="scan_prompt", seqs=16, tokens=9001, channels=4096,
             dstate=16, groups=1, io="bf16", dt="f32", state="bf16", steps=2048),
        # one user's next token
        dict(name="scan-token-one", op="scan_token", seqs=1, steps=1, channels=5120, dstate=16,
             groups=1, io="bf16", dt="bf16", state="f32"),
        # a large decode batch, fp32 state
        dict(name="scan-token-batch", op="scan_token", seqs=512, steps=1, channels=5120, dstate=16,
             groups=1, io="bf16", dt="bf16", state="f32"),
        # one sequence forked into three more samples, the pools of one layer
        dict(name="slots-fork", op="slots_copy", layers=1, slots=16, sources=1, copies=3,
             heads=80, headdim=64, dstate=128, state="f32"),
        # a beam step over eight sequences, the pools of four layers
        dict(name="slots-beams", op="slots_copy", layers=4, slots=64, sources=8, copies=3,
             heads=80, headdim=64, dstate=128, state="f32"),
        # a small pool closed up after some sequences ended
        dict(name="slots-compact-small", op="slots_compact", layers=2, slots=48, live=20, steps=1,
             heads=24, headdim=64, dstate=64, state="bf16"),
        # a serving pool, more than half empty, closed up; four slots a sequence
        dict(name="slots-compact-pool", op="slots_compact", layers=2, slots=1024, live=400, steps=4,
             heads=24, headdim=64, dstate=64, state="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv_prompt", "conv_token", "scan_prompt", "scan_token", "slots_copy",
                     "slots_compact"])
    io = rng.choice(["bf16", "f16", "bf16", "f32"])
    channels = _log(rng, 64, 8192)
    if rng.random() < 0.7:
        channels = max(8, channels // 8 * 8)
    if op == "conv_prompt":
        tokens = min(_log(rng, 1, 30000), int(1e8) // channels)
        return dict(op=op, seqs=min(tokens, _log(rng, 1, 32)), tokens=tokens, channels=channels,
                    width=rng.choice([2, 3, 4, 4]), io=io, silu=rng.random() < 0.8,
                    sliced=rng.random() < 0.5, steps=tokens)
    if op == "conv_token":
        return dict(op=op, seqs=_log(rng, 1, 1024), steps=rng.choice([1, 1, 2, 4, 7]),
                    channels=channels, width=rng.choice([2, 3, 4, 4]), io=io,
                    silu=rng.random() < 0.8, sliced=rng.random() < 0.5)
    if op in ("scan_prompt", "scan_token"):
        dstate = rng.choice([16, 16, 16, 32, 64, 128, 256])
        groups = rng.choice([g for g in (1, 1, 2, 4, 8) if channels % g == 0])
        more = dict(channels=channels, dstate=dstate, groups=groups, io=io,
                    dt=rng.choice([io, "f32"]), state=rng.choice(["f32", "bf16", "f16"]))
        if op == "scan_prompt":
            tokens = max(1, min(_log(rng, 1, 16384), int(6e8) // (channels * dstate),
                                int(2.8e7) // channels))
            return dict(op=op, seqs=min(tokens, _log(rng, 1, 32)), tokens=tokens, steps=tokens,
                        **more)
        return dict(op=op, seqs=max(1, min(_log(rng, 1, 1024), int(4e7) // (channels * dstate))),
                    steps=rng.choice([1, 1, 2, 4]), **more)
    dstate = rng.choice([16, 64, 128])
    state = rng.choice(["f32", "bf16"])
    layers = rng.choice([1, 2, 3, 4])
    heads, headdim = rng.randint(3, 80), 64
    sources, copies = _log(rng, 1, 8), rng.randint(1, 4)
    more = dict(layers=layers, heads=heads, headdim=headdim, dstate=dstate, state=state)
    if op == "slots_copy":
        return dict(op=op, slots=sources * (copies + 1) + _log(rng, 1, 32), sources=sources,
                    copies=copies, **more)
    slots = max(4, min(_log(rng, 4, 1024), int(8e8) // (heads * headdim * dstate * 4 * layers)))
    steps = rng.choice([1, 1, 2, 4])
    return dict(op=op, slots=slots, live=max(1, int(slots * rng.uniform(0.2, 0.9))), steps=steps,
                **more)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _cut(tokens, seqs, steps, r):
    """`seqs` lengths of 1 to `steps` tokens that sum to `tokens`."""
    lens = [1] * seqs
    left = tokens - seqs
    part = [r.uniform(0.25, 1.75) for _ in range(seqs)]
    for i in range(seqs):
        n = min(int(left * part[i] / sum(part[i:])) if i < seqs - 1 else left, steps - 1)
        lens[i] += n
        left -= n
    for i in range(seqs):
        n = min(left, steps - lens[i])
        lens[i] += n
        left -= n
    return lens


def _rows(case):
    """A prompt call's tokens; a decode call of up to k drafts has (k + 1) / 2 rows a sequence."""
    return case["tokens"] if "tokens" in case else case["seqs"] * (case["steps"] + 1) // 2


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _sequences(case, r, s):
    """Sequence starts, slots and what goes with them: a prompt has one slot, a
    decode call a table of a slot for each step and the accepted counts."""
    S = case["seqs"]
    prompt = case["op"].endswith("prompt")
    lens = _cut(_rows(case), S, case["steps"], r)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    width = 1 if prompt else case["steps"]
    slots = S * width + S // 4 + 2
    ids = list(range(slots))
    r.shuffle(ids)
    s["lens"], s["cu"], s["slots"], s["longest"] = lens, _ints(cu), slots, max(lens)
    if width == 1:
        s["table"] = _ints(ids[:S])
    else:
        s["table"] = _ints(ids[:S * width]).view(S, width)
        s["accepted"] = _ints([r.randint(1, width) for _ in range(S)])
    if prompt:
        s["init"] = torch.tensor([i % 2 == 1 for i in range(S)], dtype=torch.bool, device=DEV)
    return cu[-1]


def prepare(case, seed):
    r = random.Random(seed)
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        v = torch.empty(shape, dtype=torch.float32, device=DEV).normal_(0.0, std, generator=g)
        return v.to(dtype)

    def uniform(*shape, lo, hi):
        return torch.empty(shape, device=DEV).uniform_(lo, hi, generator=g)

    s = {"op": case["op"]}
    if case["op"].startswith("slots"):
        return _prepare_slots(case, r, s, normal)
    rows = _sequences(case, r, s)
    io, C = DT[case["io"]], case["channels"]
    if case["op"].startswith("conv"):
        W = case["width"]
        if case["sliced"]:  # x is a column slice of the input projection's output
            s["x"] = normal(rows, 2 * C, dtype=io)[:, C:]
        else:
            s["x"] = normal(rows, C, dtype=io)
        s["weight"] = normal(C, W, std=W ** -0.5, dtype=io)
        s["bias"] = normal(C, std=0.1, dtype=io)
        s["pool"] = normal(s["slots"], W - 1, C, dtype=io)
        s["silu"] = case["silu"]
        s["out"] = torch.empty((rows, C), dtype=io, device=DEV)
        return s
    N, G = case["dstate"], case["groups"]
    s["x"], s["z"] = normal(rows, C, dtype=io), normal(rows, C, dtype=io)
    s["dt"] = normal(rows, C, std=0.5, dtype=DT[case["dt"]])
    s["B"], s["C"] = normal(rows, G, N, dtype=io), normal(rows, G, N, dtype=io)
    # A starts training at -1 .. -N, dt_bias where softplus gives steps of 0.001 to 0.1
    s["A"] = -torch.arange(1, N + 1, device=DEV).float().repeat(C, 1) * uniform(C, N, lo=0.5, hi=1.5)
    s["D"] = uniform(C, lo=0.0, hi=1.0)
    step = torch.exp(uniform(C, lo=math.log(1e-3), hi=math.log(0.1)))
    s["bias"] = step + torch.log(-torch.expm1(-step))
    s["pool"] = normal(s["slots"], C, N, std=0.5, dtype=DT[case["state"]])
    s["out"] = torch.empty((rows, C), dtype=io, device=DEV)
    return s


def _prepare_slots(case, r, s, normal):
    """Per layer the state pool, the convolution's pool and, once, an integer tracker."""
    slots, H, P, N = case["slots"], case["heads"], case["headdim"], case["dstate"]
    s["pools"] = []
    for _ in range(case["layers"]):
        s["pools"].append(normal(slots, H, P, N, dtype=DT[case["state"]]))
        s["pools"].append(normal(slots, 3, H * P + 2 * N, dtype=torch.bfloat16))
    s["pools"].append(torch.arange(slots, dtype=torch.int32, device=DEV) * 7 + 1)
    ids = list(range(slots))
    r.shuffle(ids)
    if case["op"] == "slots_copy":
        n, k = case["sources"], case["copies"]
        s["src"] = _ints([ids[i] for i in range(n) for _ in range(k)])
        s["dst"] = _ints(ids[n:n + n * k])
        return s
    steps, live = case["steps"], case["live"]
    rows = -(-live // steps)
    held = ids[:live] + [-1] * (rows * steps - live)
    s["slots"] = slots
    s["table"] = _ints(held).view(rows, steps)
    s["moved"] = torch.empty_like(s["table"])
    s["count"] = torch.empty(1, dtype=torch.int32, device=DEV)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "slots_copy":
        src, dst = s["src"].long(), s["dst"].long()
        for p in s["pools"]:
            p[dst] = p[src]
        return [_whole(p) for p in s["pools"]]
    if s["op"] == "slots_compact":
        return _plain_compact(s)
    return _plain_conv(s) if s["op"].startswith("conv") else _plain_scan(s)


def _run_own(s):
    import mamba2_ssm_decode_gb300 as ssu
    op = s["op"]
    if op == "conv_prompt":
        ssu.conv_fwd_varlen(s["x"], s["weight"], s["cu"], bias=s["bias"],
                            activation="silu" if s["silu"] else None, conv_state=s["pool"],
                            state_batch_indices=s["table"], has_initial_state=s["init"],
                            out=s["out"])
        return s["out"], s["pool"]
    if op == "conv_token":
        act = "silu" if s["silu"] else None
        if "accepted" not in s:
            ssu.conv_update(s["pool"], s["x"], s["weight"], bias=s["bias"], activation=act,
                            state_batch_indices=s["table"], out=s["out"])
        else:
            ssu.conv_update_varlen(s["pool"], s["x"], s["weight"], bias=s["bias"], activation=act,
                                   cu_seqlens=s["cu"], num_accepted_tokens=s["accepted"],
                                   state_batch_indices=s["table"], out=s["out"])
        return s["out"], s["pool"]
    if op == "scan_prompt":
        ssu.scan_fwd_varlen(s["x"], s["dt"], s["A"], s["B"], s["C"], s["cu"], D=s["D"], z=s["z"],
                            dt_bias=s["bias"], dt_softplus=True, state=s["pool"],
                            state_batch_indices=s["table"], has_initial_state=s["init"],
                            out=s["out"])
        return s["out"], s["pool"]
    if op == "scan_token":
        kw = dict(D=s["D"], z=s["z"], dt_bias=s["bias"], dt_softplus=True,
                  state_batch_indices=s["table"], out=s["out"])
        if "accepted" not in s:
            ssu.scan_update(s["pool"], s["x"], s["dt"], s["A"], s["B"], s["C"], **kw)
        else:
            ssu.scan_update_varlen(s["pool"], s["x"], s["dt"], s["A"], s["B"], s["C"],
                                   cu_seqlens=s["cu"], num_accepted_tokens=s["accepted"], **kw)
        return s["out"], s["pool"]
    if op == "slots_copy":
        ssu.slots_copy(s["pools"], s["src"], s["dst"])
        return [_whole(p) for p in s["pools"]]
    ssu.slots_compact(s["pools"], s["table"], out=s["moved"], num_live=s["count"])
    return [s["moved"], s["count"]] + [_whole(p) for p in s["pools"]]


def _whole(p):
    """A pool's bits: what is copied has to be equal."""
    return p.view(BITS[p.element_size()])


def _places(s):
    """Per row its sequence and its position there; per sequence the slot read;
    the rows whose state is written, and the slots that take it."""
    cu = s["cu"].long()
    row = torch.arange(s["x"].shape[0], device=DEV)
    seq = torch.searchsorted(cu[1:], row, right=True)
    pos = row - cu[seq]
    table = s["table"].long()
    if "accepted" in s:
        read = table.gather(1, s["accepted"].long()[:, None] - 1)[:, 0]
        return cu, row, seq, pos, read, row, table[seq, pos]
    return cu, row, seq, pos, table, cu[1:] - 1, table


def _plain_conv(s):
    cu, row, seq, pos, read, kept, slot = _places(s)
    S, W = len(s["lens"]), s["weight"].shape[1]
    before = s["pool"][read]
    if "init" in s:
        before = torch.where(s["init"][:, None, None], before, torch.zeros_like(before))
    # the sequences' earlier rows, then the call's: what each of a row's W taps reads
    rows = torch.cat([before.reshape(S * (W - 1), -1), s["x"]])
    tap = torch.arange(W, device=DEV)
    at = torch.where(pos[:, None] + tap < W - 1, seq[:, None] * (W - 1) + pos[:, None] + tap,
                     S * (W - 1) + row[:, None] + tap - (W - 1))
    y = (rows[at].float() * s["weight"].float().t()).sum(1) + s["bias"].float()
    if s["silu"]:
        y = y / (1.0 + torch.exp(-y))
    s["pool"][slot] = rows[at[kept, 1:]]
    return y.to(s["x"].dtype), s["pool"]


def _plain_scan(s):
    cu, row, seq, pos, read, kept, slot = _places(s)
    T, C = s["x"].shape
    G, N = s["B"].shape[1:]
    h0 = s["pool"][read].float()
    if "init" in s:
        h0 = torch.where(s["init"][:, None, None], h0, torch.zeros_like(h0))
    x = s["x"].float()
    dt = s["dt"].float() + s["bias"]
    dt = torch.clamp(dt, min=0.0) + torch.log1p(torch.exp(-dt.abs()))
    a = torch.exp(dt[:, :, None] * s["A"])
    b = ((dt * x).view(T, G, C // G, 1) * s["B"].float()[:, :, None]).view(T, C, N)
    first = cu[:-1]
    b[first] += a[first] * h0
    a[first] = 0.0
    # h[t] = a[t] h[t-1] + b[t] over every sequence at once: spans of doubled length
    span = 1
    while span < s["longest"]:
        b[span:] += a[span:] * b[:-span].clone()
        a[span:] *= a[:-span].clone()
        span *= 2
    y = (b.view(T, G, C // G, N) * s["C"].float()[:, :, None]).sum(-1).view(T, C) + s["D"] * x
    z = s["z"].float()
    y = y * (z / (1.0 + torch.exp(-z)))
    s["pool"][slot] = b[kept].to(s["pool"].dtype)
    return y.to(s["x"].dtype), s["pool"]


def _plain_compact(s):
    table = s["table"].long()
    held = torch.zeros(s["slots"] + 1, dtype=torch.bool, device=DEV)
    held[torch.where(table < 0, s["slots"], table)] = True
    held = held[:-1]
    ids = torch.arange(s["slots"], device=DEV)
    live = held.sum()
    src = ids[held & (ids >= live)]
    dst = ids[~held & (ids < live)]
    to = ids.clone()
    to[src] = dst
    for p in s["pools"]:
        p[dst] = p[src]
    moved = torch.where(table < 0, table, to[table.clamp(min=0)]).int()
    return [moved, live.int().view(1)] + [_whole(p) for p in s["pools"]]


# ---------------------------------------------------------------------------
# 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    if case["op"].startswith("slots"):
        return None  # copies: whole values, equal or not
    s = prepare(case, seed)
    return _exact_conv(s) if case["op"].startswith("conv") else _exact_scan(s)


def _read_slot(s, i):
    return int(s["table"][i, int(s["accepted"][i]) - 1]) if "accepted" in s else int(s["table"][i])


def _exact_conv(s):
    """Sequence by sequence: the earlier rows and the call's side by side, tap by tap."""
    w, b, W = s["weight"].double(), s["bias"].double(), s["weight"].shape[1]
    pool = s["pool"].double()
    fresh = pool.clone()
    outs, at = [], 0
    for i, n in enumerate(s["lens"]):
        old = pool[_read_slot(s, i)]
        if "init" in s and not bool(s["init"][i]):
            old = old * 0.0
        line = torch.cat([old, s["x"][at:at + n].double()])
        y = b.expand(n, -1).clone()
        for j in range(W):
            y += w[:, j] * line[j:j + n]
        outs.append(y * torch.sigmoid(y) if s["silu"] else y)
        if "accepted" in s:
            for t in range(n):
                fresh[int(s["table"][i, t])] = line[t + 1:t + W]
        else:
            fresh[int(s["table"][i])] = line[n:]
        at += n
    return torch.cat(outs), fresh


def _exact_scan(s):
    """Token by token, every sequence that still has one."""
    S, (T, C), (G, N) = len(s["lens"]), s["x"].shape, s["B"].shape[1:]
    if s["longest"] * S * C * N > 2e10:
        return None
    A, D, bias = s["A"].double(), s["D"].double(), s["bias"].double()
    pool = s["pool"].double()
    fresh = pool.clone()
    h = torch.stack([pool[_read_slot(s, i)] for i in range(S)])
    if "init" in s:
        h[~s["init"]] = 0.0
    out = torch.empty((T, C), dtype=torch.float64, device=DEV)
    lens = torch.tensor(s["lens"], device=DEV)
    start = s["cu"][:-1].long()
    order = torch.argsort(lens, descending=True)
    many = [sum(n > t for n in s["lens"]) for t in range(s["longest"])]
    per = C // G
    for t in range(s["longest"]):
        q = order[:many[t]]
        r = start[q] + t
        x, z = s["x"][r].double(), s["z"][r].double()
        dt = torch.nn.functional.softplus(s["dt"][r].double() + bias, threshold=1e9)
        Bt = s["B"][r].double().repeat_interleave(per, dim=1)
        Ct = s["C"][r].double().repeat_interleave(per, dim=1)
        now = torch.exp(A * dt[:, :, None]) * h[q] + (dt * x)[:, :, None] * Bt
        h[q] = now
        out[r] = ((now * Ct).sum(-1) + D * x) * z * torch.sigmoid(z)
        if "accepted" in s:
            fresh[s["table"][q, t].long()] = now
    if "accepted" not in s:
        fresh[s["table"].long()] = h
    return out, fresh


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def _size(name):
    return DT[name].itemsize


def work(case):
    op = case["op"]
    if op.startswith("slots"):
        a_slot = case["layers"] * (case["heads"] * case["headdim"] * case["dstate"] *
                                   _size(case["state"]) +
                                   6 * (case["heads"] * case["headdim"] + 2 * case["dstate"])) + 4
        if op == "slots_copy":
            n, k = case["sources"], case["copies"]
            return {"bytes": n * (1 + k) * a_slot + 8 * n * k, "flops": 0}
        # of `live` slots spread over the pool, the share beyond the first `live` moves
        n = case["live"] * (1 - case["live"] / case["slots"])
        return {"bytes": int(2 * n * a_slot) + 8 * case["live"], "flops": 0}
    S, C = case["seqs"], case["channels"]
    prompt = op.endswith("prompt")
    rows = _rows(case)
    kept = S if prompt else rows  # a decode call keeps the state after each of its rows
    io = _size(case["io"])
    if op.startswith("conv"):
        W = case["width"]
        read = S // 2 if prompt else S
        return {"bytes": io * (2 * rows * C + (read + kept) * (W - 1) * C + (W + 1) * C),
                "flops": rows * C * (2 * W + (4 if case["silu"] else 0))}
    N = case["dstate"]
    read = S // 2 if prompt else S
    state = _size(case["state"]) * C * N
    moved = (rows * C * (3 * io + _size(case["dt"])) + 2 * rows * case["groups"] * N * io +
             (read + kept) * state + 4 * C * (N + 2))
    return {"bytes": moved, "flops": rows * C * (7 * N + 12)}
