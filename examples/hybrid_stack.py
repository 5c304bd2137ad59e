"""A hybrid stack served with this library: KDA layers, layers of linear
attention with one decay per head, and full-attention layers over a paged cache,
between projections that carry their epilogue.

Prompts go through the chunked forms, new tokens through the recurrent ones; both
leave their states in the same pools and pages.  ``main`` runs a few ragged
prompts, then some tokens one by one, and compares them with the same tokens run
as part of longer prompts.

    python examples/hybrid_stack.py
"""
import os
import sys
from dataclasses import dataclass, field

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_delta_rule_46_gb300 as kda  # noqa: E402

D = 128                                     # channels per head


def _norm(x):
    """RMS norm without a weight."""
    f = x.float()
    return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)


def _unit(x):
    return torch.nn.functional.normalize(x.float(), dim=-1).to(x.dtype).contiguous()


@dataclass
class Batch:
    """Sequences of a serving engine: pool slots, pages, and how many tokens each has so far."""
    slots: torch.Tensor                     # [N] int32
    table: torch.Tensor                     # [N, max_pages] int32
    have: torch.Tensor                      # [N] int32, tokens so far
    host: list = field(default_factory=list)     # the same on the host


class HybridStack:
    """`kinds`: "kda", "decay" or "attention" per layer.  H heads of 128 channels; the attention layers
    share each key-value head between `group` query heads."""

    def __init__(self, kinds, H, group, slots, pages, page_size, device, seed=0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.kinds, self.H, self.Hkv, self.ps, self.dev = kinds, H, H // group, page_size, device
        dm = H * D
        w = lambda n, k: (torch.randn(n, k, generator=g, device=device) / k ** 0.5).to(torch.bfloat16)  # noqa: E731
        self.layers = []
        for kind in kinds:
            p = {"out": w(dm, dm)}
            if kind == "kda":
                p.update(qkvz=w(4 * dm, dm), beta=w(H, dm), beta_bias=torch.zeros(H, device=device),
                         A=2 * torch.rand(H, D, generator=g, device=device) - 1,
                         pool=torch.zeros(slots, H, D, D, device=device))
            elif kind == "decay":
                p.update(qkv=w(3 * dm, dm), log_decay=-torch.exp2(-8 * torch.arange(1, H + 1, device=device) / H),
                         pool=torch.zeros(slots, H, D, D, device=device))
            else:
                kv = (pages, self.Hkv, page_size, D)
                p.update(qkv=w(dm + 2 * self.Hkv * D, dm), k=torch.empty(kv, dtype=torch.bfloat16, device=device),
                         v=torch.empty(kv, dtype=torch.bfloat16, device=device))
            self.layers.append(p)

    def _attention(self, p, y, batch, rows, start, cu, lens):
        """Appends this call's keys and values, then one row of attention per token."""
        a = kda.linear(y, p["qkv"])
        n, kv = self.H * D, self.Hkv * D
        q, k, v = (a[:, o:o + c].unflatten(1, (-1, D)) for o, c in ((0, n), (n, kv), (n + kv, kv)))
        kda.paged_append(k, v, p["k"], p["v"], batch.table, start, cu)
        return kda.paged_decode(q, p["k"], p["v"], rows, lens)

    def prefill(self, x, lens, batch):
        """x [T, H D], packed prompts of `lens` tokens; the states and caches of their slots start here."""
        T, H, dev = x.shape[0], self.H, self.dev
        cu = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device=dev)
        seq = torch.repeat_interleave(torch.arange(len(lens), device=dev), torch.tensor(lens, device=dev))
        pos = (torch.arange(T, device=dev) - cu[seq]).to(torch.int32)
        rows, upto, zero = batch.table[seq].contiguous(), pos + 1, torch.zeros_like(batch.have)
        for kind, p in zip(self.kinds, self.layers):
            y = _norm(x)
            if kind == "kda":
                a = kda.linear(y, p["qkvz"]).unflatten(1, (4, H, D))
                beta = kda.linear(y, p["beta"], p["beta_bias"], act="sigmoid", out_dtype=torch.float32)
                o, state = kda.chunk_prefill(_unit(a[:, 0]), _unit(a[:, 1]), a[:, 2].contiguous(), a[:, 3].contiguous(),
                                             p["A"], beta, cu)
                kda.state_slots_copy(p["pool"], batch.slots, state)
            elif kind == "decay":
                a = kda.linear(y, p["qkv"]).unflatten(1, (3, H, D))
                o, state = kda.decay_prefill(a[:, 0], a[:, 1], a[:, 2], p["log_decay"], cu, scale=1 / D)
                kda.state_slots_copy(p["pool"], batch.slots, state)
            else:
                o = self._attention(p, y, batch, rows, zero, cu, upto)
            x = kda.linear(o.reshape(T, -1), p["out"], residual=x)
        batch.have.copy_(cu[1:] - cu[:-1])
        return x

    def decode(self, x, batch):
        """x [N, H D], one new token per sequence."""
        N, H = x.shape[0], self.H
        upto = batch.have + 1
        for kind, p in zip(self.kinds, self.layers):
            y = _norm(x)
            if kind == "kda":
                a = kda.linear(y, p["qkvz"]).unflatten(1, (4, H, D))
                beta = kda.linear(y, p["beta"], p["beta_bias"], act="sigmoid", out_dtype=torch.float32)
                q, k, v, z = (t.unsqueeze(1).contiguous() for t in (_unit(a[:, 0]), _unit(a[:, 1]), a[:, 2], a[:, 3]))
                o = kda.decode_tokens(q, k, v, z, p["A"], beta.unsqueeze(1), p["pool"], batch.slots)
            elif kind == "decay":
                a = kda.linear(y, p["qkv"]).unflatten(1, (3, H, D))
                o = kda.decay_decode(a[:, 0], a[:, 1], a[:, 2], p["log_decay"], p["pool"], batch.slots, scale=1 / D)
            else:
                o = self._attention(p, y, batch, batch.table, batch.have, None, upto)
            x = kda.linear(o.reshape(N, -1), p["out"], residual=x)
        batch.have.copy_(upto)
        return x


def make_batch(stack, lens, new, first_slot=0, first_page=0):
    """Slots and pages, in no particular order, for prompts of `lens` tokens and `new` more each."""
    need = [-(-(n + new) // stack.ps) for n in lens]
    ids = (torch.randperm(sum(need), generator=torch.Generator().manual_seed(1)) + first_page).tolist()
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32)
    for i, n in enumerate(need):
        table[i, :n] = torch.tensor([ids.pop() for _ in range(n)], dtype=torch.int32)
    slots = torch.arange(first_slot, first_slot + len(lens), dtype=torch.int32).flip(0)
    return Batch(slots.to(stack.dev), table.to(stack.dev), torch.zeros(len(lens), dtype=torch.int32, device=stack.dev), lens)


def run(lens, new, kinds=("kda", "decay", "attention", "decay"), H=4, group=2, device="cuda:0"):
    """Prompts of `lens` tokens and `new` tokens after them, twice: token by token, and as longer
    prompts.  Returns the two hidden states of the new tokens, [len(lens), new, H 128] each."""
    dev = torch.device(device)
    pages = 2 * sum(-(-(n + new) // 16) for n in lens)
    stack = HybridStack(kinds, H, group, slots=2 * len(lens), pages=pages, page_size=16, device=dev)
    g = torch.Generator(device=dev)
    g.manual_seed(2)
    tokens = [torch.randn(n + new, H * D, generator=g, device=dev).to(torch.bfloat16) for n in lens]
    batch = make_batch(stack, lens, new)
    stack.prefill(torch.cat([t[:n] for t, n in zip(tokens, lens)]), lens, batch)
    steps = [stack.decode(torch.stack([t[n + s] for t, n in zip(tokens, lens)]), batch) for s in range(new)]
    whole = make_batch(stack, lens, new, first_slot=len(lens), first_page=pages // 2)
    longer = [n + new for n in lens]
    y = stack.prefill(torch.cat(tokens), longer, whole)
    ends = torch.tensor(longer).cumsum(0).tolist()
    return torch.stack(steps, 1), torch.stack([y[e - new:e] for e in ends])


def main():
    lens, new = [37, 1, 300, 64], 8
    one, all_ = run(lens, new)
    d = (one.float() - all_.float()).norm() / all_.float().norm()
    print(f"{len(lens)} prompts of {lens} tokens, {new} tokens each one by one: "
          f"relative difference from longer prompts {float(d):.1e}")


if __name__ == "__main__":
    main()
