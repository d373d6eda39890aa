"""A two-layer state-space language model served through the library: packed
prompts, a forked sequence, decode steps replayed from a CUDA graph, and a pool
closed up after a sequence ends.

Layer 1 is of the first Mamba form (A varies along dstate: conv_*, scan_*),
layer 2 of the second (A per head: conv_*, ssd_combined_fwd_varlen for prompts,
ssu_update for tokens).  Both keep a convolution pool and a state pool that the
same slot ids index, so one slots_copy forks a sequence and one slots_compact
moves it.  Weights are random; the projections are torch matrix products.

    python examples/serve_layers.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mamba2_ssm_decode_gb300 as ssu  # noqa: E402

BF16 = torch.bfloat16


def _param(g, *shape, scale):
    return (torch.randn(shape, generator=g) * scale).to("cuda", BF16)


def _dt_bias(g, n):
    """Where softplus gives steps of 0.001 to 0.1."""
    step = torch.exp(torch.rand(n, generator=g) * 4.6 - 6.9)
    return (step + torch.log(-torch.expm1(-step))).cuda()


class ScanLayer:
    """x -> x + W_out scan(conv(W_in x)): A [dim, dstate]."""

    def __init__(self, g, width, slots, dim=512, dstate=16, rank=32):
        self.dim, self.dstate, self.rank = dim, dstate, rank
        self.w_in = _param(g, width, 2 * dim, scale=width ** -0.5)
        self.w_x = _param(g, dim, rank + 2 * dstate, scale=dim ** -0.5)
        self.w_dt = _param(g, rank, dim, scale=rank ** -0.5)
        self.w_out = _param(g, dim, width, scale=dim ** -0.5)
        self.conv_w, self.conv_b = _param(g, dim, 4, scale=0.5), _param(g, dim, scale=0.1)
        self.A = -torch.arange(1, dstate + 1).float().repeat(dim, 1).cuda()
        self.D, self.dt_bias = torch.ones(dim, device="cuda"), _dt_bias(g, dim)
        self.conv = torch.zeros(slots, 3, dim, dtype=BF16, device="cuda")
        self.state = torch.zeros(slots, dim, dstate, device="cuda")
        self.pools = [self.conv, self.state]

    def _rows(self, x):
        """What the scan takes of the convolution's output."""
        r, n = self.rank, self.dstate
        p = x @ self.w_x
        return x, p[:, :r] @ self.w_dt, self.A, p[:, None, r:r + n], p[:, None, r + n:]

    def prompt(self, h, batch):
        xz = h @ self.w_in
        x = ssu.conv_fwd_varlen(xz[:, :self.dim], self.conv_w, batch.cu, bias=self.conv_b,
                                conv_state=self.conv, state_batch_indices=batch.slots,
                                has_initial_state=batch.fresh)
        y = ssu.scan_fwd_varlen(*self._rows(x), batch.cu, D=self.D, z=xz[:, self.dim:],
                                dt_bias=self.dt_bias, dt_softplus=True, state=self.state,
                                state_batch_indices=batch.slots, has_initial_state=batch.fresh)
        return h + y @ self.w_out

    def token(self, h, slots):
        xz = h @ self.w_in
        x = ssu.conv_update(self.conv, xz[:, :self.dim], self.conv_w, bias=self.conv_b,
                            state_batch_indices=slots)
        y = ssu.scan_update(self.state, *self._rows(x), D=self.D, z=xz[:, self.dim:],
                            dt_bias=self.dt_bias, dt_softplus=True, state_batch_indices=slots)
        return h + y @ self.w_out


class HeadLayer:
    """x -> x + W_out ssd(conv(W_in x)): A per head."""

    def __init__(self, g, width, slots, heads=8, headdim=64, dstate=64):
        self.h, self.p, self.n = heads, headdim, dstate
        self.inner, self.conv_dim = heads * headdim, heads * headdim + 2 * dstate
        self.w_in = _param(g, width, self.inner + self.conv_dim + heads, scale=width ** -0.5)
        self.w_out = _param(g, self.inner, width, scale=self.inner ** -0.5)
        self.conv_w, self.conv_b = (_param(g, self.conv_dim, 4, scale=0.5),
                                    _param(g, self.conv_dim, scale=0.1))
        self.A = -(1.0 + 15.0 * torch.rand(heads, generator=g)).cuda()
        self.D, self.dt_bias = torch.ones(heads, device="cuda"), _dt_bias(g, heads)
        self.conv = torch.zeros(slots, 3, self.conv_dim, dtype=BF16, device="cuda")
        self.state = torch.zeros(slots, heads, headdim, dstate, device="cuda")
        self.pools = [self.conv, self.state]

    def _split(self, x):
        rows, n = x.shape[0], self.n
        return (x[:, :self.inner].reshape(rows, self.h, self.p),
                x[:, None, self.inner:self.inner + n], x[:, None, self.inner + n:])

    def prompt(self, h, batch):
        zxd = h @ self.w_in
        x = ssu.conv_fwd_varlen(zxd[:, self.inner:self.inner + self.conv_dim], self.conv_w,
                                batch.cu, bias=self.conv_b, conv_state=self.conv,
                                state_batch_indices=batch.slots, has_initial_state=batch.fresh)
        x, B, C = (v.contiguous() for v in self._split(x))
        z = zxd[:, :self.inner].reshape(x.shape).contiguous()
        dt = zxd[:, -self.h:].float().contiguous()
        y = torch.empty_like(x)
        states = ssu.ssd_combined_fwd_varlen(
            x, dt, self.A, B, C, 64, batch.cu, batch.chunks, batch.last,
            batch.chunk_seq, out=y, D=self.D, z=z, dt_bias=self.dt_bias, dt_softplus=True,
            state_dtype=torch.float32)
        self.state[batch.slots.long()] = states
        return h + y.view(h.shape[0], self.inner) @ self.w_out

    def token(self, h, slots):
        zxd = h @ self.w_in
        x = ssu.conv_update(self.conv, zxd[:, self.inner:self.inner + self.conv_dim], self.conv_w,
                            bias=self.conv_b, state_batch_indices=slots)
        x, B, C = self._split(x)
        y = ssu.ssu_update(self.state, x, zxd[:, -self.h:].float(), self.A, B, C, D=self.D,
                           z=zxd[:, :self.inner].view(x.shape), dt_bias=self.dt_bias,
                           dt_softplus=True, state_batch_indices=slots)
        return h + y.reshape(h.shape[0], self.inner) @ self.w_out


class Prompts:
    """A packed batch of fresh prompts: starts, slots, and the SSD's chunks."""

    def __init__(self, lengths, slots):
        cu, chunks, seq, last = [0], [0], [], []
        for b, n in enumerate(lengths):
            for at in range(0, n, 64):
                chunks.append(cu[-1] + min(at + 64, n))
                seq.append(b)
            last.append(len(seq) - 1)
            cu.append(cu[-1] + n)
        ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        self.cu, self.chunks, self.chunk_seq, self.last = ints(cu), ints(chunks), ints(seq), ints(last)
        self.slots, self.fresh = ints(slots), torch.zeros(len(lengths), dtype=torch.bool, device="cuda")


class Server:
    """Sequences by name in slots; `batch` decode rows, unused ones padded with -1."""

    def __init__(self, vocab=512, width=256, slots=12, batch=6, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.embed = _param(g, vocab, width, scale=1.0)
        self.layers = [ScanLayer(g, width, slots), HeadLayer(g, width, slots)]
        self.pools = [p for layer in self.layers for p in layer.pools]
        self.nslots, self.slot = slots, {}
        self.table = torch.full((batch,), -1, dtype=torch.int32, device="cuda")
        self.tokens = torch.zeros(batch, dtype=torch.int64, device="cuda")
        self.logits, self.graph = None, None

    def _free(self):
        return next(i for i in range(self.nslots) if i not in self.slot.values())

    def prefill(self, prompts):
        """{name: tokens} -> {name: logits after the last token}."""
        for name in prompts:
            self.slot[name] = self._free()
        batch = Prompts([len(t) for t in prompts.values()], [self.slot[n] for n in prompts])
        h = self.embed[torch.cat([t.cuda() for t in prompts.values()])]
        for layer in self.layers:
            h = layer.prompt(h, batch)
        return dict(zip(prompts, (h[batch.cu[1:].long() - 1] @ self.embed.t()).float()))

    def fork(self, name, new):
        """Copies of a sequence under the names `new`, in every pool, in one launch."""
        ids = []
        for n in new:
            self.slot[n] = self._free()
            ids.append(self.slot[n])
        src = torch.full((len(ids),), self.slot[name], dtype=torch.int32, device="cuda")
        ssu.slots_copy(self.pools, src, torch.tensor(ids, dtype=torch.int32, device="cuda"))

    def end(self, name):
        """Free a sequence and clear what it leaves."""
        ssu.slots_clear(self.pools, torch.tensor([self.slot.pop(name)], dtype=torch.int32, device="cuda"))

    def compact(self):
        """Move the live sequences to the front of every pool; their number."""
        names = list(self.slot)
        table = torch.tensor([self.slot[n] for n in names], dtype=torch.int32, device="cuda")
        moved, live = ssu.slots_compact(self.pools, table)
        self.slot = dict(zip(names, moved.tolist()))
        return int(live)

    def _forward(self):
        h = self.embed[self.tokens]
        for layer in self.layers:
            h = layer.token(h, self.table)
        self.logits = (h @ self.embed.t()).float()

    def step(self, tokens):
        """{name: next token} -> {name: logits}: one replay of the captured step."""
        names = list(tokens)
        pad = len(self.table) - len(names)
        self.table.copy_(torch.tensor([self.slot[n] for n in names] + [-1] * pad, dtype=torch.int32))
        self.tokens.copy_(torch.tensor([int(tokens[n]) for n in names] + [0] * pad))
        if self.graph is None:
            kept = [p.clone() for p in self.pools]
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):   # set-up outside the capture
                self._forward()
            torch.cuda.current_stream().wait_stream(side)
            for p, k in zip(self.pools, kept):
                p.copy_(k)
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                self._forward()
        self.graph.replay()
        return dict(zip(names, self.logits[:len(names)].clone()))


def main():
    g = torch.Generator().manual_seed(1)
    text = {n: torch.randint(0, 512, (k,), generator=g) for n, k in (("a", 37), ("b", 200), ("c", 5))}
    server = Server()
    logits = server.prefill(text)
    server.fork("b", ["b1", "b2"])              # two more continuations of b
    logits.update(b1=logits["b"], b2=logits["b"])
    text.update(b1=text["b"], b2=text["b"])
    for t in range(8):
        # greedy, except that each continuation of b begins with another token
        best = {n: v.topk(3).indices[{"b1": 1, "b2": 2}.get(n, 0) if t == 0 else 0]
                for n, v in logits.items()}
        text = {n: torch.cat([text[n], best[n].cpu()[None]]) for n in best}
        logits = server.step(best)
        if t == 3:
            server.end("a")
            server.end("b")
            for n in ("a", "b"):
                del logits[n]
                del text[n]
            print("live sequences after compaction:", server.compact(), server.slot)
    # a server that has seen none of it, given the whole texts as prompts
    whole = Server().prefill(text)
    worst = 0.0
    for n in text:
        d = float((whole[n] - logits[n]).norm() / whole[n].norm())
        worst = max(worst, d)
        print(f"{n}: {len(text[n])} tokens, step by step against at once: relative difference {d:.2e}")
    return worst


if __name__ == "__main__":
    if main() > 0.03:
        sys.exit("the two ways disagree")
