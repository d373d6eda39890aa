"""Cases and plain forms of linear attention with a decay for each head, of the
verification of drafted tokens, and of the maps and slot tables that a batch's
lengths give.

`own` False: each operator in elementary torch operations, in fp32 (decays are
summed in 64 bits), rounded once.  `own` True: the same call through the
package's entry points.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
INT = {"i32": torch.int32, "i64": torch.int64}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one user's short prompt into a fresh slot, a fixed decay for each head
        dict(name="linattn-prompt-one", op="lin_prompt", seqs=1, tokens=300, steps=300, heads=32,
             groups=32, dk=128, dv=128, io="bf16", state="f32", decay="head"),
        # a packed batch of prompts of 16 lengths, half of them continued from an earlier piece
        dict(name="linattn-prompt-batch", op="lin_prompt", seqs=16, tokens=20634, steps=2048,
             heads=32, groups=32, dk=128, dv=128, io="bf16", state="f32", decay="token"),
        # one long document of an odd length; few heads, queries and keys shared by groups of them
        dict(name="linattn-prompt-long", op="lin_prompt", seqs=1, tokens=12289, steps=12289,
             heads=24, groups=8, dk=128, dv=64, io="f16", state="bf16", decay="token"),
        # one user's next token: a call that is all latency
        dict(name="linattn-token-one", op="lin_token", seqs=1, steps=1, heads=32, groups=32,
             dk=128, dv=128, io="bf16", state="f32", decay="head"),
        # a large decode batch
        dict(name="linattn-token-batch", op="lin_token", seqs=256, steps=1, heads=32, groups=32,
             dk=128, dv=128, io="bf16", state="f32", decay="token"),
        # speculative decoding: 1 to 4 drafted tokens a sequence, a slot for each, 16-bit state
        dict(name="linattn-token-drafts", op="lin_token", seqs=128, steps=4, heads=80, groups=8,
             dk=128, dv=64, io="bf16", state="bf16", decay="token"),
        # one user's four drafted tokens against the model's probabilities
        dict(name="verify-one", op="verify", seqs=1, drafts=4, vocab=50288, probs="f32", q=True,
             ragged=False),
        # a full batch, up to five drafts a sequence, a large vocabulary of an odd size
        dict(name="verify-batch", op="verify", seqs=256, drafts=5, vocab=128257, probs="f32",
             q=True, ragged=True),
        # the maps of a handful of prompts
        dict(name="maps-small", op="maps", seqs=16, tokens=20634, pad_rows=0, chunk=256,
             context=True, ints="i32"),
        # ... of a large batch, padded to a captured graph's size
        dict(name="maps-large", op="maps", seqs=2048, tokens=500001, pad_rows=24287, chunk=128,
             context=True, ints="i32"),
        # slots for new requests in a small pool
        dict(name="assign-small", op="assign", seqs=20, steps=1, slots=48, ints="i32", held=0.7),
        # a serving pool: one slot for each of four steps, some sequences ended, some grown
        dict(name="assign-pool", op="assign", seqs=2000, steps=4, slots=16384, ints="i32",
             held=0.8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lin_prompt", "lin_prompt", "lin_token", "lin_token", "verify", "maps",
                     "assign"])
    if op in ("lin_prompt", "lin_token"):
        groups = _log(rng, 1, 32)
        heads = groups * rng.choice([1, 1, 2, 3, 4])
        more = dict(heads=heads, groups=groups, state=rng.choice(["f32", "f32", "bf16", "f16"]),
                    decay=rng.choice(["head", "token", "token", "none"]))
        if op == "lin_prompt":
            dk, dv = rng.choice([64, 128, 128]), rng.choice([64, 128, 128])
            tokens = max(1, min(_log(rng, 1, 20000), int(660000 * 128 * 4) // (heads * (2 * dk + 2 * dv))))
            return dict(op=op, seqs=min(tokens, _log(rng, 1, 64)), tokens=tokens, steps=tokens,
                        dk=dk, dv=dv, io=rng.choice(["bf16", "bf16", "f16"]), **more)
        dk, dv = rng.choice([16, 32, 64, 128, 128, 256]), rng.choice([_log(rng, 1, 256), 64, 128])
        steps = rng.choice([1, 1, 2, 4, 6])
        most = int(1.2e8) // (heads * dk * dv * (steps + 1) // 2)
        return dict(op=op, seqs=max(1, min(_log(rng, 1, 512), most)), steps=steps, dk=dk, dv=dv,
                    io=rng.choice(["bf16", "bf16", "f16", "f32"]), **more)
    if op == "verify":
        vocab, drafts = _log(rng, 2, 160000), rng.randint(1, 8)
        most = int(1.5e8) // (vocab * (drafts + 1))
        return dict(op=op, seqs=max(1, min(_log(rng, 1, 512), most)), drafts=drafts, vocab=vocab,
                    probs=rng.choice(["f32", "f32", "bf16", "f16"]), q=rng.random() < 0.7,
                    ragged=rng.random() < 0.7)
    if op == "maps":
        seqs = _log(rng, 1, 4096)
        return dict(op=op, seqs=seqs, tokens=_log(rng, 1, 500000), pad_rows=rng.choice([0, 0, 1, 100, 5000]),
                    chunk=16 * _log(rng, 1, 16), context=rng.random() < 0.7,
                    ints=rng.choice(["i32", "i64"]))
    seqs, steps = _log(rng, 1, 2000), rng.choice([1, 1, 2, 4, 5])
    return dict(op=op, seqs=seqs, steps=steps, slots=max(2, int(seqs * steps * rng.uniform(0.5, 4.0))),
                ints=rng.choice(["i32", "i64"]), held=rng.uniform(0.0, 1.0))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _cut(tokens, seqs, steps, r):
    """`seqs` lengths of 1 to `steps` tokens that sum to `tokens`."""
    lens = [1] * seqs
    left = tokens - seqs
    part = [r.uniform(0.25, 1.75) for _ in range(seqs)]
    rest = sum(part)
    for i in range(seqs):
        n = min(int(left * part[i] / rest) if i < seqs - 1 else left, steps - 1)
        rest -= part[i]
        lens[i] += n
        left -= n
    for i in range(seqs):
        n = min(left, steps - lens[i])
        lens[i] += n
        left -= n
    return lens


def _sums(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device=DEV)


def _rows(case):
    """A prompt call's tokens; a decode call of up to k drafts has (k + 1) / 2 rows a sequence."""
    return case["tokens"] if "tokens" in case else case["seqs"] * (case["steps"] + 1) // 2


def prepare(case, seed):
    r = random.Random(seed)
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = {"op": case["op"]}
    if case["op"].startswith("lin"):
        return _prepare_lin(case, r, g, s)
    if case["op"] == "verify":
        return _prepare_verify(case, r, g, s)
    if case["op"] == "maps":
        return _prepare_maps(case, r, s)
    return _prepare_assign(case, r, s)


def _prepare_lin(case, r, g, s):
    def normal(*shape, std=1.0, dtype=torch.float32):
        v = torch.empty(shape, dtype=torch.float32, device=DEV).normal_(0.0, std, generator=g)
        return v.to(dtype)

    S, prompt = case["seqs"], case["op"] == "lin_prompt"
    H, G, dk, dv, io = case["heads"], case["groups"], case["dk"], case["dv"], DT[case["io"]]
    lens = _cut(_rows(case), S, case["steps"], r)
    rows = sum(lens)
    width = 1 if prompt else case["steps"]
    slots = S * width + S // 4 + 2
    ids = list(range(slots))
    r.shuffle(ids)
    s["lens"], s["cu"], s["longest"] = lens, _ints(_sums(lens)), max(lens)
    if width == 1:
        s["table"] = _ints(ids[:S])
    else:
        s["table"] = _ints(ids[:S * width]).view(S, width)
        s["accepted"] = _ints([r.randint(1, width) for _ in range(S)])
    if prompt:
        s["init"] = torch.tensor([i % 2 == 1 for i in range(S)], dtype=torch.bool, device=DEV)
    # q, k and v are column slices of one projection's output
    wide = normal(rows, 2 * G * dk + H * dv, dtype=io)
    s["q"] = wide[:, :G * dk].view(rows, G, dk)
    s["k"] = wide[:, G * dk:2 * G * dk].view(rows, G, dk)
    s["v"] = wide[:, 2 * G * dk:].view(rows, H, dv)
    s["decay"] = None
    if case["decay"] == "head":     # slopes that halve from head to head
        s["decay"] = -torch.exp2(-8.0 * torch.arange(1, H + 1, device=DEV).float() / H)
    elif case["decay"] == "token":  # the log of a gate, a sixteenth of it
        x = normal(rows, H, std=2.0)
        s["decay"] = -(torch.clamp(-x, min=0.0) + torch.log1p(torch.exp(-x.abs()))) / 16.0
    s["pool"] = normal(slots, H, dv, dk, std=0.5, dtype=DT[case["state"]])
    s["scale"] = dk ** -0.5
    s["out"] = torch.empty((rows, H, dv), dtype=io, device=DEV)
    return s


def _prepare_verify(case, r, g, s):
    S, K, V = case["seqs"], case["drafts"], case["vocab"]
    io = DT[case["probs"]]
    n = [r.randint(0, K) if case["ragged"] else K for _ in range(S)]
    cu = _sums([m + 1 for m in n])
    rows = cu[-1]
    s["cu"] = _ints(cu) if case["ragged"] else None
    s["lens"] = [m + 1 for m in n]
    logits = torch.empty((rows, V), device=DEV).normal_(0.0, 3.0, generator=g)
    e = torch.exp(logits - logits.amax(1, keepdim=True))
    s["p"] = (e / e.sum(1, keepdim=True)).to(io)
    # row of draft j of sequence i; places without a draft take any row
    at = torch.tensor([[min(cu[i] + j, rows - 1) for j in range(K)] for i in range(S)], device=DEV)
    # a draft model that mostly agrees; its drafts are drawn from its own probabilities
    noise = torch.empty((S, K, V), device=DEV).normal_(0.0, 0.7, generator=g)
    e = torch.exp(logits[at] + noise - 16.0)
    q = e / e.sum(2, keepdim=True)
    race = torch.empty((S, K, V), device=DEV).exponential_(generator=g)
    s["drafts"] = (q / race).argmax(2).int()
    s["q"] = q.to(io) if case["q"] else None
    s["u"] = torch.rand((S, K + 1), device=DEV, generator=g)
    s["greedy"] = torch.tensor([i % 4 == 3 for i in range(S)], dtype=torch.bool, device=DEV)
    s["tokens"] = torch.empty((S, K + 1), dtype=torch.int32, device=DEV)
    s["count"] = torch.empty(S, dtype=torch.int32, device=DEV)
    return s


def _prepare_maps(case, r, s):
    S, dtype = case["seqs"], INT[case["ints"]]
    weight = [r.uniform(0.0, 1.0) if r.random() < 0.9 else 0.0 for _ in range(S)]
    total = sum(weight) or 1.0
    lens = [int(case["tokens"] * w / total) for w in weight]
    s["lens"] = _ints(lens, dtype)
    s["rows"], s["chunk"] = case["tokens"] + case["pad_rows"], case["chunk"]
    s["context"] = None
    if case["context"]:
        s["context"] = _ints([r.choice([0, r.randint(1, 4000)]) for _ in range(S)], dtype)
    s["most"] = s["rows"] // case["chunk"] + (2 if case["context"] else 1) * S
    s["maps"] = None
    return s


def _prepare_assign(case, r, s):
    S, T, slots, dtype = case["seqs"], case["steps"], case["slots"], INT[case["ints"]]
    ids = list(range(slots))
    r.shuffle(ids)
    table, counts = [], []
    for _ in range(S):
        n = r.choice([0, T, T, r.randint(0, T)])
        have = min(len(ids), T if r.random() < case["held"] else 0)
        table.append([ids.pop() if t < have else -1 for t in range(T)])
        counts.append(n)
    s["table"], s["counts"], s["slots"] = _ints(table, dtype).view(S, T), _ints(counts, dtype), slots
    s["out"], s["fresh"] = torch.empty_like(s["table"]), torch.empty_like(s["table"])
    s["missing"] = torch.empty(1, dtype=torch.int32, device=DEV)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "lin_prompt":
        return _plain_prompt(s)
    if s["op"] == "lin_token":
        return _plain_token(s)
    return {"verify": _plain_verify, "maps": _plain_maps, "assign": _plain_assign}[s["op"]](s)


def _run_own(s):
    import mamba2_ssm_decode_gb300 as ssu
    op = s["op"]
    if op == "lin_prompt":
        ssu.linattn_fwd_varlen(s["q"], s["k"], s["v"], s["cu"], log_decay=s["decay"],
                               scale=s["scale"], state=s["pool"], state_batch_indices=s["table"],
                               has_initial_state=s["init"], out=s["out"])
        return s["out"], s["pool"]
    if op == "lin_token":
        kw = dict(log_decay=s["decay"], scale=s["scale"], state_batch_indices=s["table"],
                  out=s["out"])
        if "accepted" not in s:
            ssu.linattn_update(s["pool"], s["q"], s["k"], s["v"], **kw)
        else:
            ssu.linattn_update_varlen(s["pool"], s["q"], s["k"], s["v"], cu_seqlens=s["cu"],
                                      num_accepted_tokens=s["accepted"], **kw)
        return s["out"], s["pool"]
    if op == "verify":
        return ssu.drafts_verify(s["p"], s["drafts"], s["u"], draft_probs=s["q"],
                                 cu_seqlens=s["cu"], greedy=s["greedy"], out=s["tokens"],
                                 num_accepted=s["count"])
    if op == "maps":
        s["maps"] = m = ssu.prompt_maps(s["lens"], s["chunk"], s["rows"], context_lens=s["context"],
                                        out=s["maps"])
        return list(m)
    return ssu.slots_assign(s["table"], s["counts"], s["slots"], out=s["out"], fresh=s["fresh"],
                            num_missing=s["missing"])


def _places(s):
    """Per row its sequence and its position there."""
    cu = s["cu"].long()
    row = torch.arange(s["q"].shape[0], device=DEV)
    seq = torch.searchsorted(cu[1:], row, right=True)
    return cu, row, seq, row - cu[seq]


def _by_head(t, heads):
    """[rows, groups, d] as fp32 [rows, heads, d]: a group's vector for each of its heads."""
    return t.float().repeat_interleave(heads // t.shape[1], dim=1)


def _log_decay(s, rows, heads):
    if s["decay"] is None:
        return torch.zeros((rows, heads), device=DEV)
    return s["decay"].expand(rows, heads)


def _plain_token(s):
    """Every sequence's drafts side by side, padded to the longest: with the running sum a of the
    log decays, o_t = e^a_t S0 q_t + sum over j <= t of e^(a_t - a_j) (q_t . k_j) v_j."""
    cu, row, seq, pos = _places(s)
    (T, H, dv), S, L = s["v"].shape, len(s["lens"]), s["longest"]
    table = s["table"].long().view(S, -1)
    first = s["accepted"].long() - 1 if "accepted" in s else torch.zeros_like(table[:, 0])
    h0 = s["pool"][table.gather(1, first[:, None])[:, 0]].float()

    def padded(t):
        out = torch.zeros((S, L) + t.shape[1:], dtype=t.dtype, device=DEV)
        out[seq, pos] = t
        return out.transpose(1, 2)                                  # [S, H, L, ...]

    q, k, v = padded(_by_head(s["q"], H)), padded(_by_head(s["k"], H)), padded(s["v"].float())
    a = padded(_log_decay(s, T, H).double()).cumsum(2)
    gap = a[..., :, None] - a[..., None, :]
    before = torch.ones((L, L), dtype=torch.bool, device=DEV).tril()
    e = torch.exp(torch.where(before, gap, torch.full_like(gap, -math.inf))).float()
    ea = torch.exp(a).float()
    o = torch.matmul(torch.matmul(q, k.transpose(2, 3)) * e, v)
    o = s["scale"] * (o + ea[..., None] * torch.matmul(q, h0.transpose(2, 3)))
    out = o.transpose(1, 2)[seq, pos].to(s["v"].dtype)
    # the state after each step, into that step's slot
    h = ea[..., None, None] * h0[:, :, None]
    w = e[..., None] * v[:, :, None]                                # [S, H, L, L, dv]
    h = h + torch.matmul(w.transpose(3, 4), k[:, :, None])
    s["pool"][table[seq, pos]] = h.transpose(1, 2)[seq, pos].to(s["pool"].dtype)
    return out, s["pool"]


def _plain_prompt(s):
    """Chunks of 64 tokens of every sequence side by side; the states that enter them from spans of
    doubled length."""
    Q = 64
    cu, row, seq, pos = _places(s)
    (T, H, dv), S, dk = s["v"].shape, len(s["lens"]), s["q"].shape[2]
    many = (cu[1:] - cu[:-1] + Q - 1) // Q
    end = many.cumsum(0)
    N = (s["longest"] + Q - 1) // Q
    total = sum((n + Q - 1) // Q for n in s["lens"])
    chunk, at = (end - many)[seq] + pos // Q, pos % Q

    def chunks(t):
        out = torch.zeros((total, Q) + t.shape[1:], dtype=t.dtype, device=DEV)
        out[chunk, at] = t
        return out.transpose(1, 2)                                  # [chunks, H, Q, ...]

    q, k, v = chunks(_by_head(s["q"], H)), chunks(_by_head(s["k"], H)), chunks(s["v"].float())
    a = chunks(_log_decay(s, T, H).double()).cumsum(2)
    gap = a[..., :, None] - a[..., None, :]
    before = torch.ones((Q, Q), dtype=torch.bool, device=DEV).tril()
    e = torch.exp(torch.where(before, gap, torch.full_like(gap, -math.inf))).float()
    o = torch.matmul(torch.matmul(q, k.transpose(2, 3)) * e, v)
    # b: the state that a chunk leaves (its sequence's initial one counts into the first)
    b = torch.matmul((v * e[:, :, -1, :, None]).transpose(2, 3), k)
    d = torch.exp(a[:, :, -1]).float()[..., None, None]
    h0 = s["pool"][s["table"].long()].float()
    h0 = torch.where(s["init"][:, None, None, None], h0, torch.zeros_like(h0))
    first = end - many
    b[first] += d[first] * h0
    d[first] = 0.0
    span = 1
    while span < N:
        b[span:] += d[span:] * b[:-span].clone()
        d[span:] *= d[:-span].clone()
        span *= 2
    enter = torch.empty_like(b)
    enter[1:] = b[:-1]
    enter[first] = h0
    o = s["scale"] * (o + torch.exp(a).float()[..., None] * torch.matmul(q, enter.transpose(2, 3)))
    s["pool"][s["table"].long()] = b[end - 1].to(s["pool"].dtype)
    return o.transpose(1, 2)[chunk, at].to(s["v"].dtype), s["pool"]


def _plain_verify(s):
    p, q, u, drafts = s["p"].float(), s["q"], s["u"], s["drafts"].long()
    S, K = drafts.shape
    V = p.shape[1]
    if s["cu"] is None:
        start = torch.arange(S, device=DEV) * (K + 1)
        n = torch.full_like(start, K)
    else:
        start = s["cu"][:-1].long()
        n = s["cu"][1:].long() - start - 1
    j = torch.arange(K, device=DEV)
    there = j < n[:, None]
    row = torch.where(there, start[:, None] + j, start[:, None])
    pd = p[row, drafts]
    qd = torch.ones_like(pd) if q is None else q.gather(2, drafts[..., None])[..., 0].float()
    # products of two fp32 numbers are whole in 64 bits: no draft is decided by a rounding
    taken = u[:, :K].double() * qd.double() < pd.double()
    top = p.argmax(1)
    taken = torch.where(s["greedy"][:, None], top[row] == drafts, taken) & there
    count = taken.long().cumprod(1).sum(1)
    last = start + count
    left = p[last]
    rejected = (count < n)[:, None]
    place = count.clamp(max=K - 1)
    if q is None:
        other = torch.arange(V, device=DEV) == drafts.gather(1, place[:, None])
        less = torch.where(other, torch.zeros_like(left), left)
    else:
        less = torch.clamp(left - q[torch.arange(S, device=DEV), place].float(), min=0.0)
    left = torch.where(rejected, less, left)
    # weights in units of 2^-44, summed as integers
    cum = torch.round(left.double() * 2.0 ** 44).long().cumsum(1)
    total = cum[:, -1]
    mark = torch.floor(u[:, K].double() * total.double()).long()
    mark = torch.minimum(mark, total - 1)
    token = (cum <= mark[:, None]).sum(1)
    token = torch.where(s["greedy"], top[last], token)
    step = torch.arange(K + 1, device=DEV)
    wide = torch.cat([drafts, drafts[:, :1]], 1)
    tokens = torch.where(step < count[:, None], wide,
                         torch.where(step == count[:, None], token[:, None],
                                     torch.full_like(wide, -1)))
    return tokens.int(), (count + 1).int()


def _plain_maps(s):
    lens, rows, cs, most = s["lens"].long(), s["rows"], s["chunk"], s["most"]
    S, dtype = lens.shape[0], s["lens"].dtype
    context = s["context"].long() if s["context"] is not None else torch.zeros_like(lens)
    zero = torch.zeros(1, dtype=torch.long, device=DEV)
    cu = torch.cat([zero, lens.cumsum(0)])
    off = context % cs
    many = torch.clamp((off + lens + cs - 1) // cs, min=1)
    end = many.cumsum(0)
    chunk = torch.arange(most, device=DEV)
    seq = torch.searchsorted(end, chunk, right=True).clamp(max=S - 1)
    nth = chunk - (end - many)[seq]
    start = torch.where(nth == 0, cu[seq], cu[seq] + nth * cs - off[seq])
    start = torch.minimum(start, cu[seq + 1])
    start = torch.cat([torch.where(chunk < end[-1], start, cu[-1]), cu[-1:]])
    row = torch.arange(rows, device=DEV)
    owner = torch.searchsorted(cu[1:], row, right=True)
    inside = owner < S
    o = owner.clamp(max=S - 1)
    pos = context[o] + row - cu[o]
    none = torch.full_like(row, -1)
    return [cu.to(dtype), start.to(dtype), seq.to(dtype), (end - 1).to(dtype), context > 0,
            end[-1:].to(dtype), torch.where(inside, owner, none).to(dtype),
            torch.where(inside, pos, none).to(dtype)]


def _plain_assign(s):
    table, slots = s["table"].long(), s["slots"]
    T = table.shape[1]
    wanted = torch.arange(T, device=DEV) < s["counts"].long()[:, None]
    kept = wanted & (table >= 0) & (table < slots)
    held = torch.zeros(slots + 1, dtype=torch.bool, device=DEV)
    held[torch.where(kept, table, slots)] = True
    free = torch.nonzero(~held[:-1])[:, 0]
    need = wanted & ~kept
    rank = need.view(-1).long().cumsum(0).view(table.shape) - 1
    got = need & (rank < free.shape[0])
    some = torch.cat([free, free.new_zeros(1)])
    none = torch.full_like(table, -1)
    fresh = torch.where(got, some[torch.where(got, rank, 0)], none)
    out = torch.where(kept, table, fresh)
    return out.to(s["table"].dtype), fresh.to(s["table"].dtype), (need & ~got).sum().int().view(1)


# ---------------------------------------------------------------------------
# 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] in ("maps", "assign"):
        return None  # whole values, equal or not
    s = prepare(case, seed)
    return _exact_lin(s) if case["op"].startswith("lin") else _exact_verify(s)


def _exact_lin(s):
    """Token by token, every sequence that still has one."""
    S, (T, H, dv), (G, dk) = len(s["lens"]), s["v"].shape, s["q"].shape[1:]
    if s["longest"] * S * H * dv * dk > 4e10:
        return None
    pool = s["pool"].double()
    fresh = pool.clone()
    table = s["table"].long().view(S, -1)
    pick = [int(s["accepted"][i]) - 1 if "accepted" in s else 0 for i in range(S)]
    h = torch.stack([pool[int(table[i, pick[i]])] for i in range(S)])
    if "init" in s:
        h[~s["init"]] = 0.0
    out = torch.empty((T, H, dv), dtype=torch.float64, device=DEV)
    order = torch.argsort(torch.tensor(s["lens"], device=DEV), descending=True)
    many = [sum(n > t for n in s["lens"]) for t in range(s["longest"])]
    start, per = s["cu"][:-1].long(), H // G
    for t in range(s["longest"]):
        i = order[:many[t]]
        r = start[i] + t
        q = s["q"][r].double().repeat_interleave(per, dim=1)
        k = s["k"][r].double().repeat_interleave(per, dim=1)
        now = h[i]
        if s["decay"] is not None:
            d = s["decay"] if s["decay"].dim() == 1 else s["decay"][r]
            now = now * torch.exp(d.double())[..., None, None]
        now = now + s["v"][r].double()[..., None] * k[:, :, None]
        h[i] = now
        out[r] = s["scale"] * (now * q[:, :, None]).sum(-1)
        if "accepted" in s:
            fresh[table[i, t]] = now
    if "accepted" not in s:
        fresh[table[:, 0]] = h
    return out, fresh


def _exact_verify(s):
    """Sequence by sequence, draft by draft."""
    S, K = s["drafts"].shape
    drafts, u, greedy = s["drafts"].tolist(), s["u"].double(), s["greedy"].tolist()
    tokens = torch.full((S, K + 1), -1, dtype=torch.int32, device=DEV)
    counts, at = [], 0
    for i in range(S):
        n, k = s["lens"][i] - 1, 0
        token = None
        while token is None:
            p = s["p"][at + k].double()
            q = s["q"][i, min(k, K - 1)].double() if s["q"] is not None else None
            if greedy[i]:
                best = int(p.argmax())
                if k == n or best != drafts[i][k]:
                    token = best
            elif k == n or not float(u[i, k]) * (1.0 if q is None else float(q[drafts[i][k]])) < float(p[drafts[i][k]]):
                if k < n and q is None:
                    p[drafts[i][k]] = 0.0
                elif k < n:
                    p = torch.clamp(p - q, min=0.0)
                c = torch.round(p.float().double() * 2.0 ** 44).cumsum(0)
                token = int((c <= float(torch.floor(u[i, K] * c[-1]))).sum())
            if token is None:
                tokens[i, k] = drafts[i][k]
                k += 1
        tokens[i, k] = token
        counts.append(k + 1)
        at += n + 1
    return tokens, _ints(counts)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op.startswith("lin"):
        S, H, G, dk, dv = (case[n] for n in ("seqs", "heads", "groups", "dk", "dv"))
        rows, prompt = _rows(case), op == "lin_prompt"
        io, state = DT[case["io"]].itemsize, DT[case["state"]].itemsize * H * dv * dk
        read = S // 2 if prompt else S
        kept = S if prompt else rows  # a decode call keeps the state after each of its rows
        decay = {"none": 0, "head": 4 * H, "token": 4 * rows * H}[case["decay"]]
        return {"bytes": io * rows * (2 * G * dk + 2 * H * dv) + decay + (read + kept) * state,
                "flops": rows * H * dk * dv * 5}
    if op == "verify":
        # the probabilities of the row that decides, and the draft's where one was turned down
        S, V, io = case["seqs"], case["vocab"], DT[case["probs"]].itemsize
        return {"bytes": int(S * V * io * (1.75 if case["q"] else 1.0)) + 12 * S * (case["drafts"] + 1),
                "flops": 3 * S * V}
    i = INT[case["ints"]].itemsize
    if op == "maps":
        rows, S = case["tokens"] + case["pad_rows"], case["seqs"]
        most = rows // case["chunk"] + (2 if case["context"] else 1) * S
        return {"bytes": i * (2 * rows + 2 * most + (5 if case["context"] else 3) * S), "flops": 0}
    return {"bytes": i * (3 * case["seqs"] * case["steps"] + case["seqs"]), "flops": 0}
