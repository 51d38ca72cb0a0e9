"""A small hybrid decoder served end to end: packed prompts, single-token steps on a state cache, parallel
samples by forking, requests that end, compaction.

    python -m gated_delta_rule_sm_gb300.serve --prompts 37 200 5 --samples 3 --steps 16

Layers alternate between the delta rule (``short_conv_prompt``, ``forward``, ``gated_norm``; then
``short_conv_step``, ``decode_step``) and the state space scan (``short_conv_prompt``, ``ssm_scan``,
``gated_norm``; then ``short_conv_step``, ``ssm_step``).  Weights are random; the dense projections are
plain matrix products.  Every sequence owns one page of the cache, which holds all layers' recurrent states
and convolution histories; a page's index is its slot in the steps' pools.
"""
from __future__ import annotations

import argparse
import math
import time

import torch

from . import (decode_step, device_status, forward, gated_norm, pages_compact, pages_copy, pages_extend, pages_fork,
               pages_free, short_conv_prompt, short_conv_step, ssm_scan, ssm_step)

WHOLE = 1 << 30   # tokens of a page: more than any sequence, so that a page never fills


class Decoder:
    """Weights of a decoder with ``layers`` layers of ``heads`` heads."""

    def __init__(self, layers=4, heads=4, groups=2, dim=128, head_dim=64, state_dim=64, width=4, vocab=512, seed=0,
                 device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.heads, self.groups, self.dim, self.head_dim, self.state_dim, self.width = (heads, groups, dim, head_dim,
                                                                                       state_dim, width)
        H, P, N, G = heads, head_dim, state_dim, groups

        def normal(*shape, std=None):
            std = 1.0 / math.sqrt(shape[0]) if std is None else std
            return (std * torch.randn(*shape, generator=g)).to(device)

        self.embed = normal(vocab, dim, std=1.0).bfloat16()
        self.head = normal(dim, vocab).bfloat16()
        self.layers = []
        for i in range(layers):
            delta = i % 2 == 0
            conv = 3 * H * P if delta else H * P + 2 * G * N          # channels that pass the convolution
            rest = H * P + (H * P + H if delta else H)                # output gate; g_raw and beta, or dt
            step = torch.exp(math.log(1e-3) + torch.rand(H, generator=g) * math.log(1e2))
            self.layers.append(dict(
                # (the projection's width is rounded up: the convolution reads it in vectors of eight channels)
                delta=delta, conv=conv, rest=rest, w_in=normal(dim, -(-(conv + rest) // 8) * 8).bfloat16(),
                w_out=normal(H * P, dim).bfloat16(), taps=normal(conv, width, std=0.5), taps_bias=torch.zeros(conv, device=device),
                a_log=torch.log(1.0 + 15.0 * torch.rand(H, generator=g)).to(device),
                dt_bias=(normal(H * P, std=0.1) if delta else (step + torch.log(-torch.expm1(-step))).to(device)),
                d_skip=torch.ones(H, device=device), norm=torch.ones(P, device=device)))

    def state_shape(self, layer):
        return ((self.heads, self.head_dim, self.head_dim) if layer["delta"]
                else (self.heads, self.state_dim, self.head_dim))


class StateCache:
    """Pools of recurrent states and convolution histories, one page (slot) per sequence."""

    def __init__(self, model: Decoder, slots: int, sequences: int, device="cuda"):
        self.pools = []
        for layer in model.layers:
            self.pools.append(dict(
                state=torch.zeros(1, slots, *model.state_shape(layer), device=device),
                history=torch.zeros(1, slots, model.width - 1, layer["conv"], device=device, dtype=torch.bfloat16)))
        self.table = torch.full((sequences, 1), -1, dtype=torch.int32, device=device)
        self.lengths = torch.zeros(sequences, dtype=torch.int32, device=device)
        self.refs = torch.zeros(slots, dtype=torch.int32, device=device)
        self.ids = torch.arange(slots, dtype=torch.int32, device=device)

    def every_pool(self):
        for pool in self.pools:
            yield from pool.values()

    def admit(self, rows, tokens):
        """Pages for sequences of the given lengths."""
        return pages_extend(self.table, self.lengths, self.refs, rows, tokens, page_tokens=WHOLE)

    def slots(self, rows):
        return self.table[rows.long(), 0].contiguous()

    def fork(self, parents, children):
        """children go on from copies of the parents' states.  Returns ok: 0 where nothing was done (no free page, or
        the child holds one)."""
        first, *others = self.every_pool()
        ok = pages_fork(first, self.table, self.lengths, self.refs, parents, children, page_tokens=WHOLE)
        src, dst = self.slots(parents), self.slots(children)
        dst = torch.where(ok > 0, dst, -1)       # pairs out of range are skipped
        for pool in others:
            pages_copy(pool, src, dst)
        return ok

    def release(self, rows):
        pages_free(self.table, self.lengths, self.refs, rows)

    def compact(self):
        first, *others = self.every_pool()
        to = pages_compact(first, self.table, self.refs)
        src = torch.where((to >= 0) & (to != self.ids), self.ids, -1)     # pairs out of range are skipped
        for pool in others:
            pages_copy(pool, src, to)


def _rms(x):
    x = x.float()
    return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).bfloat16()


def _split(model, layer, z):
    """The convolution's channels, the output gate and the mixer's own inputs of a projection."""
    H, P = model.heads, model.head_dim
    conv, both = layer["conv"], layer["conv"] + layer["rest"]
    return z[..., :conv], z[..., conv:conv + H * P], z[..., conv + H * P:both]


def _mix_out(model, layer, h, y, gate):
    y = gated_norm(y.contiguous(), gate.unflatten(-1, (model.heads, model.head_dim)).contiguous(), layer["norm"])
    return h + y.flatten(-2) @ layer["w_out"]


def prompt(model: Decoder, cache: StateCache, tokens, cu_seqlens, rows):
    """Packed prompts [1, T] from empty states; their states go to the rows' pages.  Returns the logits [1, T, vocab]."""
    H, P, N, G = model.heads, model.head_dim, model.state_dim, model.groups
    h = model.embed[tokens]
    slots = cache.slots(rows)
    docs = torch.arange(rows.numel(), dtype=torch.int32, device=rows.device)
    for layer, pool in zip(model.layers, cache.pools):
        conv, gate, rest = _split(model, layer, _rms(h) @ layer["w_in"])
        conv, history = short_conv_prompt(conv, layer["taps"], layer["taps_bias"], cu_seqlens=cu_seqlens)
        if layer["delta"]:
            q, k, v = (t.unflatten(-1, (H, P)).contiguous() for t in conv.chunk(3, dim=-1))
            g_raw, beta = rest.split([H * P, H], dim=-1)
            y, state = forward(q, k, v, g_raw.unflatten(-1, (H, P)).contiguous(), beta.contiguous(), layer["a_log"],
                               layer["dt_bias"], scale=P ** -0.5, cu_seqlens=cu_seqlens, output_final_state=True)
        else:
            x, b, c = conv.split([H * P, G * N, G * N], dim=-1)
            y, state = ssm_scan(x.unflatten(-1, (H, P)), rest, b.unflatten(-1, (G, N)), c.unflatten(-1, (G, N)),
                                layer["a_log"], layer["dt_bias"], layer["d_skip"], cu_seqlens=cu_seqlens,
                                output_final_state=True)
        pages_copy(pool["state"], docs, slots, src_pool=state[None])
        pages_copy(pool["history"], docs, slots, src_pool=history[None])
        h = _mix_out(model, layer, h, y, gate)
    return (_rms(h) @ model.head).float()


def step(model: Decoder, cache: StateCache, tokens, rows):
    """The next token [B] of each row.  Returns the logits [B, vocab]."""
    H, P, N, G = model.heads, model.head_dim, model.state_dim, model.groups
    h = model.embed[tokens]
    slots = cache.slots(rows)
    for layer, pool in zip(model.layers, cache.pools):
        conv, gate, rest = _split(model, layer, _rms(h) @ layer["w_in"])
        conv, _ = short_conv_step(conv, layer["taps"], layer["taps_bias"], history=pool["history"][0], slots=slots)
        if layer["delta"]:
            q, k, v = (t.unflatten(-1, (H, P)).contiguous() for t in conv.chunk(3, dim=-1))
            g_raw, beta = rest.split([H * P, H], dim=-1)
            y, _ = decode_step(q, k, v, g_raw.unflatten(-1, (H, P)).contiguous(), beta.contiguous(), layer["a_log"],
                               layer["dt_bias"], scale=P ** -0.5, state=pool["state"][0], slots=slots)
        else:
            x, b, c = conv.split([H * P, G * N, G * N], dim=-1)
            y, _ = ssm_step(x.unflatten(-1, (H, P)), rest, b.unflatten(-1, (G, N)), c.unflatten(-1, (G, N)),
                            layer["a_log"], layer["dt_bias"], layer["d_skip"], state=pool["state"][0], slots=slots)
        h = _mix_out(model, layer, h, y, gate)
    return (_rms(h) @ model.head).float()


def offsets(lengths, device="cuda"):
    ends = torch.tensor([0, *lengths]).cumsum(0)
    return ends.to(torch.int32).to(device)


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--prompts", type=int, nargs="+", default=[37, 200, 5], help="prompt lengths")
    ap.add_argument("--samples", type=int, default=3, help="samples that go on from the first prompt")
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--heads", type=int, default=4)
    a = ap.parse_args()
    model = Decoder(layers=a.layers, heads=a.heads)
    n = len(a.prompts)
    total = n + a.samples - 1
    cache = StateCache(model, slots=total + 4, sequences=total)
    ids = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    rows = ids(*range(n))
    cache.admit(rows, ids(*a.prompts))
    g = torch.Generator().manual_seed(1)
    tokens = torch.randint(0, model.embed.shape[0], (1, sum(a.prompts)), generator=g).cuda()
    cu = offsets(a.prompts)
    logits = prompt(model, cache, tokens, cu, rows)
    last = logits[0, cu[1:].long() - 1]
    # the first prompt's samples start from its best few tokens
    children = ids(*range(n, total))
    cache.fork(torch.zeros_like(children), children)
    rows = ids(*range(total))
    best = last.topk(a.samples, dim=-1).indices
    nxt = torch.cat([best[:, 0], best[0, 1:]])
    made = [nxt]
    for i in range(a.steps):
        if i == 1:                      # (the first step loads kernels)
            torch.cuda.synchronize()
            t0 = time.perf_counter()
        nxt = step(model, cache, nxt, rows).argmax(-1)
        made.append(nxt)
    torch.cuda.synchronize()
    dt = (time.perf_counter() - t0) / max(1, a.steps - 1) if a.steps > 1 else float("nan")
    cache.release(rows[1:2])            # the second request ends
    cache.compact()
    rows = torch.cat([rows[:1], rows[2:]])
    step(model, cache, torch.cat([nxt[:1], nxt[2:]]), rows)
    torch.cuda.synchronize()
    assert device_status() == 0
    print(f"{n} prompts of {a.prompts} tokens, {total} sequences, {a.steps} steps: {dt * 1e6:.0f} us a step")
    for r, seq in enumerate(torch.stack(made, 1).tolist()):
        print(f"  sequence {r}: {seq}")


if __name__ == "__main__":
    main()
