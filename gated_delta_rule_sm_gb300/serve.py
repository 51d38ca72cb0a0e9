"""A small hybrid decoder served end to end: packed prompts, single-token steps on a state cache, parallel
samples by forking, requests that end, compaction.

    python -m gated_delta_rule_sm_gb300.serve --prompts 37 200 5 --samples 3 --steps 16 --pattern dsga

Layers go through a pattern of mixers: the delta rule d (``short_conv_prompt``, ``forward``, ``gated_norm``; then
``short_conv_step``, ``decode_step``), the state space scan s (``ssm_scan``; then ``ssm_step``), the gated linear
recurrence g (``gated_scan``; then ``gated_step``), both between the same convolution and norm, and attention a
(``pages_append``, ``pages_attention``, ``gated_norm``).  Weights are random; the dense projections are
plain matrix products.  Every sequence owns one page of the cache, which holds all layers' recurrent states
and convolution histories; a page's index is its slot in the steps' pools.  Its keys and values are in pages of a
few tokens of a second cache.
"""
from __future__ import annotations

import argparse
import math
import time

import torch

from . import (decode_step, device_status, forward, gated_norm, gated_scan, gated_step, pages_append, pages_attention,
               pages_compact, pages_copy, pages_extend, pages_fork, pages_free, short_conv_prompt, short_conv_step,
               ssm_scan, ssm_step)

WHOLE = 1 << 30   # tokens of a page: more than any sequence, so that a page never fills


class Decoder:
    """Weights of a decoder with ``layers`` layers of ``heads`` heads, their mixers by the letters of ``pattern`` in turn."""

    def __init__(self, layers=4, heads=4, groups=2, dim=128, head_dim=64, state_dim=64, width=4, vocab=512, seed=0,
                 device="cuda", pattern="ds"):
        if not pattern or set(pattern) - set("dsga") or not set(pattern[:layers]) & set("dsg"):
            raise ValueError("pattern must be letters of d, s, g and a, a recurrent one (d, s, g) among the layers'")
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
            kind = pattern[i % len(pattern)]
            delta = kind == "d"
            # channels that pass the convolution; and the output gate with g_raw and beta, dt, both gates, or q, k and v
            conv = {"d": 3 * H * P, "s": H * P + 2 * G * N, "g": H * P, "a": 0}[kind]
            rest = H * P + {"d": H * P + H, "s": H, "g": 2 * H * P, "a": (H + 2 * G) * P}[kind]
            step = torch.exp(math.log(1e-3) + torch.rand(H, generator=g) * math.log(1e2))
            self.layers.append(dict(
                # (the projection's width is rounded up: the convolution reads it in vectors of eight channels)
                kind=kind, delta=delta, conv=conv, rest=rest, w_in=normal(dim, -(-(conv + rest) // 8) * 8).bfloat16(),
                w_out=normal(H * P, dim).bfloat16(), taps=normal(conv, width, std=0.5), taps_bias=torch.zeros(conv, device=device),
                a_log=(torch.log(-torch.log(0.9 + 0.099 * torch.rand(H * P, generator=g))) if kind == "g"
                       else torch.log(1.0 + 15.0 * torch.rand(H, generator=g))).to(device),
                dt_bias=(normal(H * P, std=0.1) if delta else (step + torch.log(-torch.expm1(-step))).to(device)),
                d_skip=torch.ones(H, device=device), norm=torch.ones(P, device=device)))

    def state_shape(self, layer):
        return {"d": (self.heads, self.head_dim, self.head_dim), "s": (self.heads, self.state_dim, self.head_dim),
                "g": (self.heads * self.head_dim,)}[layer["kind"]]


class StateCache:
    """Pools of recurrent states and convolution histories, one page (slot) per sequence, and the attention layers' keys
    and values in ``kv_pages`` pages of ``page_tokens`` tokens."""

    def __init__(self, model: Decoder, slots: int, sequences: int, device="cuda", kv_pages: int = 0, kv_row: int = 64,
                 page_tokens: int = 16):
        ints = lambda *shape, fill=0: torch.full(shape, fill, dtype=torch.int32, device=device)  # noqa: E731
        self.pools = []
        attention = sum(layer["kind"] == "a" for layer in model.layers)
        kv_pages = kv_pages or sequences * kv_row
        self.page_tokens = page_tokens
        self.kv = torch.zeros(attention, kv_pages, 2, model.groups, page_tokens, model.head_dim, device=device,
                              dtype=torch.bfloat16) if attention else None
        self.kv_table, self.kv_lengths, self.kv_refs = ints(sequences, kv_row, fill=-1), ints(sequences), ints(kv_pages)
        for layer in model.layers:
            if layer["kind"] == "a":
                self.pools.append(dict(kv=self.kv[sum("kv" in pool for pool in self.pools)]))
                continue
            self.pools.append(dict(
                state=torch.zeros(1, slots, *model.state_shape(layer), device=device),
                history=torch.zeros(1, slots, model.width - 1, layer["conv"], device=device, dtype=torch.bfloat16)))
        self.table = ints(sequences, 1, fill=-1)
        self.lengths = ints(sequences)
        self.refs = ints(slots)
        self.ids = torch.arange(slots, dtype=torch.int32, device=device)

    def every_pool(self):
        for pool in self.pools:
            if "kv" not in pool:
                yield from pool.values()

    def admit(self, rows, tokens):
        """Pages for sequences of the given lengths.  Returns ok: 0 where there were not enough (the row then stays as it was)."""
        before = self.lengths[rows.long().clamp(0, self.lengths.numel() - 1)]      # (rows that are none are refused below)
        ok = pages_extend(self.table, self.lengths, self.refs, rows, tokens, page_tokens=WHOLE)
        if self.kv is not None:
            both = pages_extend(self.kv_table, self.kv_lengths, self.kv_refs, torch.where(ok > 0, rows, -1), tokens,
                                page_tokens=self.page_tokens)
            back = (ok > 0) & (both == 0)
            # (a page that the row had before this call holds its states)
            pages_free(self.table, self.lengths, self.refs, torch.where(back & (before == 0), rows, -1))
            self.lengths[rows[back].long()] = before[back]
            ok = both
        return ok

    def grow(self, rows, tokens):
        """Room for that many more keys and values of each row.  Returns ok."""
        if self.kv is None:
            return torch.ones_like(rows)
        return pages_extend(self.kv_table, self.kv_lengths, self.kv_refs, rows, self.kv_lengths[rows.long()] + tokens,
                            page_tokens=self.page_tokens)

    def slots(self, rows):
        return self.table[rows.long(), 0].contiguous()

    def fork(self, parents, children):
        """children go on from copies of the parents' states.  Returns ok: 0 where nothing was done (no free page, or
        the child holds one)."""
        first, *others = self.every_pool()
        ok = pages_fork(first, self.table, self.lengths, self.refs, parents, children, page_tokens=WHOLE)
        if self.kv is not None:
            both = pages_fork(self.kv, self.kv_table, self.kv_lengths, self.kv_refs, torch.where(ok > 0, parents, -1), children,
                              page_tokens=self.page_tokens)
            pages_free(self.table, self.lengths, self.refs, torch.where((ok > 0) & (both == 0), children, -1))
            ok = both
        src, dst = self.slots(parents), self.slots(children)
        dst = torch.where(ok > 0, dst, -1)       # pairs out of range are skipped
        for pool in others:
            pages_copy(pool, src, dst)
        return ok

    def release(self, rows):
        pages_free(self.table, self.lengths, self.refs, rows)
        pages_free(self.kv_table, self.kv_lengths, self.kv_refs, rows)

    def compact(self):
        first, *others = self.every_pool()
        to = pages_compact(first, self.table, self.refs)
        src = torch.where((to >= 0) & (to != self.ids), self.ids, -1)     # pairs out of range are skipped
        for pool in others:
            pages_copy(pool, src, to)
        if self.kv is not None:
            pages_compact(self.kv, self.kv_table, self.kv_refs)


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


def _attend(model, cache, pool, z, rows, cu_seqlens):
    """The new tokens' keys and values into the pages, and their attention: z [B, n, channels] or packed."""
    H, G, P = model.heads, model.groups, model.head_dim
    q, k, v = (t.unflatten(-1, (n, P)) for t, n in zip(z.split([H * P, G * P, G * P], dim=-1), (H, G, G)))
    pages_append(pool["kv"], cache.kv_table, cache.kv_lengths, k, v, seqs=rows, cu_seqlens=cu_seqlens)
    return pages_attention(q, pool["kv"], cache.kv_table, cache.kv_lengths, scale=P ** -0.5, seqs=rows, cu_seqlens=cu_seqlens)


def prompt(model: Decoder, cache: StateCache, tokens, cu_seqlens, rows, more: bool = False):
    """Packed prompts [1, T], counted in the cache already; their states go to the rows' pages.  From empty states, or, with
    ``more``, from what the rows' earlier chunks left.  Returns the logits [1, T, vocab]."""
    H, P, N, G = model.heads, model.head_dim, model.state_dim, model.groups
    h = model.embed[tokens]
    slots = cache.slots(rows)
    docs = torch.arange(rows.numel(), dtype=torch.int32, device=rows.device)
    for layer, pool in zip(model.layers, cache.pools):
        conv, gate, rest = _split(model, layer, _rms(h) @ layer["w_in"])
        if layer["kind"] == "a":
            h = _mix_out(model, layer, h, _attend(model, cache, pool, rest, rows, cu_seqlens), gate)
            continue
        state, history = (pool[n][0][slots.long()] if more else None for n in ("state", "history"))
        conv, history = short_conv_prompt(conv, layer["taps"], layer["taps_bias"], cu_seqlens=cu_seqlens, initial_history=history)
        if layer["kind"] == "d":
            q, k, v = (t.unflatten(-1, (H, P)).contiguous() for t in conv.chunk(3, dim=-1))
            g_raw, beta = rest.split([H * P, H], dim=-1)
            y, state = forward(q, k, v, g_raw.unflatten(-1, (H, P)).contiguous(), beta.contiguous(), layer["a_log"],
                               layer["dt_bias"], scale=P ** -0.5, cu_seqlens=cu_seqlens, initial_state=state,
                               output_final_state=True)
        elif layer["kind"] == "s":
            x, b, c = conv.split([H * P, G * N, G * N], dim=-1)
            y, state = ssm_scan(x.unflatten(-1, (H, P)), rest, b.unflatten(-1, (G, N)), c.unflatten(-1, (G, N)),
                                layer["a_log"], layer["dt_bias"], layer["d_skip"], cu_seqlens=cu_seqlens, initial_state=state,
                                output_final_state=True)
        else:
            g_raw, i_raw = rest.chunk(2, dim=-1)
            y, state = gated_scan(conv, g_raw, i_raw, layer["a_log"], cu_seqlens=cu_seqlens, initial_state=state,
                                  output_final_state=True)
            y = y.unflatten(-1, (H, P))
        pages_copy(pool["state"], docs, slots, src_pool=state[None])
        pages_copy(pool["history"], docs, slots, src_pool=history[None])
        h = _mix_out(model, layer, h, y, gate)
    return (_rms(h) @ model.head).float()


def step(model: Decoder, cache: StateCache, tokens, rows):
    """The next token [B] of each row.  Returns the logits [B, vocab]; a row whose keys and values find no free page stays as
    it is and gets NaN."""
    H, P, N, G = model.heads, model.head_dim, model.state_dim, model.groups
    h = model.embed[tokens]
    slots = cache.slots(rows)
    if cache.kv is not None:
        refused = cache.grow(rows, 1) == 0
        rows, slots = (t.masked_fill(refused, -1) for t in (rows, slots))
    for layer, pool in zip(model.layers, cache.pools):
        conv, gate, rest = _split(model, layer, _rms(h) @ layer["w_in"])
        if layer["kind"] == "a":
            h = _mix_out(model, layer, h, _attend(model, cache, pool, rest[:, None], rows, None)[:, 0], gate)
            continue
        conv, _ = short_conv_step(conv, layer["taps"], layer["taps_bias"], history=pool["history"][0], slots=slots)
        if layer["kind"] == "d":
            q, k, v = (t.unflatten(-1, (H, P)).contiguous() for t in conv.chunk(3, dim=-1))
            g_raw, beta = rest.split([H * P, H], dim=-1)
            y, _ = decode_step(q, k, v, g_raw.unflatten(-1, (H, P)).contiguous(), beta.contiguous(), layer["a_log"],
                               layer["dt_bias"], scale=P ** -0.5, state=pool["state"][0], slots=slots)
        elif layer["kind"] == "s":
            x, b, c = conv.split([H * P, G * N, G * N], dim=-1)
            y, _ = ssm_step(x.unflatten(-1, (H, P)), rest, b.unflatten(-1, (G, N)), c.unflatten(-1, (G, N)),
                            layer["a_log"], layer["dt_bias"], layer["d_skip"], state=pool["state"][0], slots=slots)
        else:
            g_raw, i_raw = rest.chunk(2, dim=-1)
            y, _ = gated_step(conv, g_raw, i_raw, layer["a_log"], state=pool["state"][0], slots=slots)
            y = y.unflatten(-1, (H, P))
        h = _mix_out(model, layer, h, y, gate)
    logits = (_rms(h) @ model.head).float()
    return logits if cache.kv is None else logits.masked_fill(refused[:, None], math.nan)


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
    ap.add_argument("--pattern", default="ds", help="mixers of the layers in turn: d, s, g, a")
    a = ap.parse_args()
    model = Decoder(layers=a.layers, heads=a.heads, pattern=a.pattern)
    n = len(a.prompts)
    total = n + a.samples - 1
    most = max(a.prompts) + a.steps + 1
    cache = StateCache(model, slots=total + 4, sequences=total, kv_row=-(-most // 16))
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
