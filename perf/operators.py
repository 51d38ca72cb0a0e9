"""Cases of the serving operators: the state space scan over prompts, the single-token steps, the short
convolution with a carried history, and the page operators of the state and key/value caches.

``run`` computes a case in its plain form (elementary torch operations in 32 bits) while ``own`` is false,
and through the package's entry points while it is true.  ``exact`` gives the same outputs in 64 bits,
computed token by token from the definitions.
"""
from __future__ import annotations

import math

import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
NORM_EPS = 1e-6
STATE_PAGE = 1 << 30   # tokens of a page that never fills: a recurrent state


def listed():
    return [
        # a chat turn's short prompt on a small hybrid layer: latency
        dict(name="scan short", kind="scan", B=1, T=37, H=8, G=1, N=64, P=64, docs=0, dtype="bf16", init=True),
        # a packed prefill batch of continued conversations: documents of any length, each from its own state
        dict(name="scan packed", kind="scan", B=1, T=16384, H=32, G=4, N=128, P=64, docs=12, dtype="bf16", init=True),
        # one long prompt: few heads' chains over many tokens
        dict(name="scan long", kind="scan", B=1, T=65536, H=32, G=1, N=128, P=64, docs=0, dtype="bf16", init=False),
        # the fp32 evaluation path at odd sizes, an odd number of heads to a group
        dict(name="scan fp32 odd", kind="scan", B=2, T=1021, H=6, G=2, N=48, P=40, docs=0, dtype="fp32", init=True),
        # one user's next token
        dict(name="ssm step one", kind="ssm_step", B=1, H=8, G=1, N=64, P=64, slots=16, dtype="bf16"),
        # a serving batch's next token, rows scattered over the pool, some rows idle
        dict(name="ssm step batch", kind="ssm_step", B=128, H=32, G=1, N=128, P=64, slots=160, dtype="bf16"),
        # the same two for the delta rule's own state
        dict(name="decode one", kind="decode", B=1, H=16, Hk=16, K=128, V=128, slots=16, gate="lower_bounded",
             dtype="bf16"),
        dict(name="decode batch", kind="decode", B=64, H=32, Hk=16, K=128, V=128, slots=96, gate="softplus",
             dtype="bf16"),
        # the projections of a packed prefill through the convolution, histories in and out
        dict(name="conv packed", kind="conv", B=1, T=16384, C=4096, W=4, docs=12, dtype="bf16"),
        # the same for a batch's next token
        dict(name="conv step batch", kind="conv_step", B=128, C=12288, W=4, slots=160, dtype="bf16"),
        # parallel samples from one prompt: 24 forks of recurrent states, 1 MB a layer each
        dict(name="fork states", kind="fork", seqs=64, forks=24, pages=96, row=1, page_tokens=STATE_PAGE, layers=8,
             words=1 << 18),
        # finished requests leave a paged cache, the rest moves together: 16-token pages of 16 KB a layer
        dict(name="compact pages", kind="compact", seqs=256, gone=128, pages=16384, row=64, page_tokens=16, layers=4,
             words=4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["scan", "scan", "scan", "ssm_step", "decode", "conv", "conv_step", "fork", "compact"])
    if kind == "scan":
        dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
        G = rng.choice([1, 1, 2, 4])
        H = G * rng.choice([2, 3, 4, 6, 8])
        T = _log(rng, 1, 32768 if dtype == "bf16" else 4096)
        docs = rng.choice([0, 0, rng.randint(1, 24)])
        B = 1 if docs else rng.choice([1, 1, 2, 3])
        return dict(kind=kind, B=B, T=T, H=H, G=G, N=16 * rng.randint(1, 8), P=rng.choice([32, 64, 64, 80, 128]),
                    docs=docs, dtype=dtype, init=rng.random() < 0.5)
    if kind in ("ssm_step", "conv_step"):
        B = _log(rng, 1, 128)
        slots = B + rng.randint(0, 40)
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        if kind == "conv_step":
            return dict(kind=kind, B=B, C=8 * (2 * _log(rng, 4, 768) + 1), W=rng.randint(2, 8), slots=slots, dtype=dtype)
        G = rng.choice([1, 2, 4])
        return dict(kind=kind, B=B, H=G * rng.choice([2, 3, 8]), G=G, N=16 * rng.randint(1, 16),
                    P=16 * rng.randint(1, 8), slots=slots, dtype=dtype)
    if kind == "decode":
        B = _log(rng, 1, 64)
        Hk = rng.choice([2, 5, 8, 16])
        return dict(kind=kind, B=B, H=Hk * rng.choice([1, 2]), Hk=Hk, K=16 * rng.randint(1, 8),
                    V=16 * rng.randint(1, 8), slots=B + rng.randint(0, 40),
                    gate=rng.choice(["lower_bounded", "softplus"]), dtype=rng.choice(["bf16", "bf16", "fp32"]))
    if kind == "conv":
        docs = rng.choice([0, rng.randint(1, 24)])
        return dict(kind=kind, B=1 if docs else rng.choice([1, 2]), T=_log(rng, 1, 8192), C=8 * (2 * _log(rng, 4, 256) + 1),
                    W=rng.randint(2, 8), docs=docs, dtype=rng.choice(["bf16", "bf16", "fp32"]))
    if kind == "fork":
        seqs = _log(rng, 4, 256)
        row = _log(rng, 1, 64)
        pages = seqs * row + rng.randint(0, seqs)
        return dict(kind=kind, seqs=seqs, forks=rng.randint(1, max(1, seqs // 2)), pages=pages, row=row,
                    page_tokens=rng.choice([1, 16, 64]), layers=rng.randint(1, 4), words=4 * _log(rng, 1, 1024))
    seqs = _log(rng, 4, 256)
    row = _log(rng, 1, 64)
    return dict(kind=kind, seqs=seqs, gone=rng.randint(0, seqs), pages=seqs * row + rng.randint(0, 64), row=row,
                page_tokens=rng.choice([1, 16, 64]), layers=rng.randint(1, 4), words=4 * _log(rng, 1, 512))


# ---------------------------------------------------------------------------------------------- inputs


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEVICE, dtype=torch.float32)


def _rand(gen, *shape):
    return torch.rand(shape, generator=gen, device=DEVICE, dtype=torch.float32)


def _silu(x):
    return x / (1.0 + torch.exp(-x))


def _lengths(gen, tokens, docs):
    """Offsets of `docs` documents of random lengths (empty ones among them) that cover the tokens."""
    cuts = torch.randint(0, tokens + 1, (docs - 1,), generator=gen, device=DEVICE).sort().values
    ends = torch.tensor([0], device=DEVICE), cuts, torch.tensor([tokens], device=DEVICE)
    return torch.cat(ends).to(torch.int32)


def _pool_rows(gen, B, slots):
    """Every row's slot of the pool, in no order; every seventh row is idle (-1) where there are several."""
    rows = torch.randperm(slots, generator=gen, device=DEVICE)[:B].to(torch.int32)
    rows[6::7] = -1
    return rows


def _dt_params(gen, H):
    step = torch.exp(math.log(1e-3) + _rand(gen, H) * math.log(1e2))   # steps of 0.001 to 0.1
    dt_bias = step + torch.log(-torch.expm1(-step))                    # softplus gives the step back
    return dict(a_log=torch.log(1.0 + 15.0 * _rand(gen, H)), dt_bias=dt_bias, d_skip=1.0 + 0.1 * _randn(gen, H))


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    return dict(globals()["_prepare_" + case["kind"]](case, gen), case=case)


def _prepare_scan(c, gen):
    B, T, H, G, N, P = (c[k] for k in ("B", "T", "H", "G", "N", "P"))
    # x, b and c come as one projection's output after the convolution and SiLU
    xbc = _silu(_randn(gen, B, T, H * P + 2 * G * N)).to(DTYPES[c["dtype"]])
    x, b, cc = xbc.split([H * P, G * N, G * N], dim=-1)
    s = dict(x=x.unflatten(-1, (H, P)), b=b.unflatten(-1, (G, N)), c=cc.unflatten(-1, (G, N)),
             dt_raw=(0.5 * _randn(gen, B, T, H)).to(DTYPES[c["dtype"]]), **_dt_params(gen, H))
    s["cu_seqlens"] = _lengths(gen, T, c["docs"]) if c["docs"] else None
    rows = c["docs"] or B
    s["longest"] = int((s["cu_seqlens"][1:] - s["cu_seqlens"][:-1]).max()) if c["docs"] else T
    s["initial_state"] = 0.5 * _randn(gen, rows, H, N, P) if c["init"] else None
    return s


def _prepare_ssm_step(c, gen):
    B, H, G, N, P = (c[k] for k in ("B", "H", "G", "N", "P"))
    xbc = _silu(_randn(gen, B, H * P + 2 * G * N)).to(DTYPES[c["dtype"]])
    x, b, cc = xbc.split([H * P, G * N, G * N], dim=-1)
    s = dict(x=x.unflatten(-1, (H, P)), b=b.unflatten(-1, (G, N)), c=cc.unflatten(-1, (G, N)),
             dt_raw=(0.5 * _randn(gen, B, H)).to(DTYPES[c["dtype"]]), **_dt_params(gen, H))
    s["slots"] = _pool_rows(gen, B, c["slots"])
    s["state"] = 0.5 * _randn(gen, c["slots"], H, N, P)
    s["state_out"] = s["state"].clone()
    return s


def _prepare_decode(c, gen):
    B, H, Hk, K, V = (c[k] for k in ("B", "H", "Hk", "K", "V"))
    act = lambda *shape: _randn(gen, *shape).to(DTYPES[c["dtype"]])  # noqa: E731
    s = dict(q=act(B, Hk, K), k=act(B, Hk, K), v=act(B, H, V), g_raw=act(B, H, K), beta_raw=act(B, H),
             a_log=math.log(16.0) * _rand(gen, H), dt_bias=0.1 * _randn(gen, H * K))
    s["slots"] = _pool_rows(gen, B, c["slots"])
    s["state"] = 0.1 * _randn(gen, c["slots"], H, K, V)
    s["state_out"] = s["state"].clone()
    return s


def _prepare_conv(c, gen):
    B, T, C, W = (c[k] for k in ("B", "T", "C", "W"))
    s = dict(x=_randn(gen, B, T, C).to(DTYPES[c["dtype"]]), weight=_randn(gen, C, W) / math.sqrt(W),
             bias=0.1 * _randn(gen, C), cu_seqlens=_lengths(gen, T, c["docs"]) if c["docs"] else None)
    s["initial_history"] = _randn(gen, c["docs"] or B, W - 1, C).to(DTYPES[c["dtype"]])
    return s


def _prepare_conv_step(c, gen):
    B, C, W = (c[k] for k in ("B", "C", "W"))
    s = dict(x=_randn(gen, B, C).to(DTYPES[c["dtype"]]), weight=_randn(gen, C, W) / math.sqrt(W),
             bias=0.1 * _randn(gen, C), slots=_pool_rows(gen, B, c["slots"]))
    s["history"] = _randn(gen, c["slots"], W - 1, C).to(DTYPES[c["dtype"]])
    s["history_out"] = s["history"].clone()
    return s


def _cache(c, gen, seqs, lengths):
    """A pool and the table of its sequences' pages, in no order."""
    M, pt = c["row"], c["page_tokens"]
    held = (lengths + pt - 1) // pt
    col = torch.arange(M, device=DEVICE)
    used = col[None] < held[:, None]
    order = torch.randperm(c["pages"], generator=gen, device=DEVICE)
    table = torch.full((seqs, M), -1, dtype=torch.int64, device=DEVICE)
    table[used] = order[:int(used.sum())]
    refs = torch.zeros(c["pages"], dtype=torch.int32, device=DEVICE)
    refs[table[used]] = 1
    pool = torch.randint(-(1 << 31), 1 << 31, (c["layers"], c["pages"], c["words"]), generator=gen, device=DEVICE,
                         dtype=torch.int32)
    table = table.to(torch.int32)
    return dict(pool=pool, table=table, lengths=lengths.to(torch.int32), refs=refs, table_out=table.clone(),
                lengths_out=lengths.to(torch.int32), refs_out=refs.clone())


def _row_lengths(c, gen, seqs):
    span = c["row"] * min(c["page_tokens"], 4096)
    return torch.randint(1, span + 1, (seqs,), generator=gen, device=DEVICE)


def _prepare_fork(c, gen):
    lengths = _row_lengths(c, gen, c["seqs"])
    rows = torch.randperm(c["seqs"], generator=gen, device=DEVICE)
    children = rows[:c["forks"]]          # empty rows that take the forks
    lengths[children] = 0
    pick = torch.randint(0, c["seqs"] - c["forks"], (c["forks"],), generator=gen, device=DEVICE)
    s = _cache(c, gen, c["seqs"], lengths)
    return dict(s, parents=rows[c["forks"]:][pick].to(torch.int32), children=children.to(torch.int32))


def _prepare_compact(c, gen):
    s = _cache(c, gen, c["seqs"], _row_lengths(c, gen, c["seqs"]))
    s["gone"] = torch.randperm(c["seqs"], generator=gen, device=DEVICE)[:c["gone"]].to(torch.int32)
    return s


# ------------------------------------------------------------------------------------------------ runs


def run(state):
    return globals()[("_own_" if own else "_plain_") + state["case"]["kind"]](state, state["case"])


def _own_scan(s, c):
    import gated_delta_rule_sm_gb300 as kda
    return kda.ssm_scan(s["x"], s["dt_raw"], s["b"], s["c"], s["a_log"], s["dt_bias"], s["d_skip"],
                        cu_seqlens=s["cu_seqlens"], initial_state=s["initial_state"], output_final_state=True)


def _own_ssm_step(s, c):
    import gated_delta_rule_sm_gb300 as kda
    return kda.ssm_step(s["x"], s["dt_raw"], s["b"], s["c"], s["a_log"], s["dt_bias"], s["d_skip"],
                        state=s["state"], slots=s["slots"], state_out=s["state_out"])


def _own_decode(s, c):
    import gated_delta_rule_sm_gb300 as kda
    return kda.decode_step(s["q"], s["k"], s["v"], s["g_raw"], s["beta_raw"], s["a_log"], s["dt_bias"],
                           scale=c["K"] ** -0.5, lower_bound=-5.0, gate=c["gate"], state=s["state"],
                           slots=s["slots"], state_out=s["state_out"])


def _own_conv(s, c):
    import gated_delta_rule_sm_gb300 as kda
    return kda.short_conv_prompt(s["x"], s["weight"], s["bias"], cu_seqlens=s["cu_seqlens"],
                                 initial_history=s["initial_history"])


def _own_conv_step(s, c):
    import gated_delta_rule_sm_gb300 as kda
    return kda.short_conv_step(s["x"], s["weight"], s["bias"], history=s["history"], slots=s["slots"],
                               history_out=s["history_out"])


def _own_fork(s, c):
    import gated_delta_rule_sm_gb300 as kda
    ok = kda.pages_fork(s["pool"], s["table"], s["lengths"], s["refs"], s["parents"], s["children"],
                        page_tokens=c["page_tokens"], table_out=s["table_out"], lengths_out=s["lengths_out"],
                        refs_out=s["refs_out"])
    return ok, s["table_out"], s["lengths_out"], s["refs_out"], s["pool"]


def _own_compact(s, c):
    import gated_delta_rule_sm_gb300 as kda
    kda.pages_free(s["table"], s["lengths"], s["refs"], s["gone"], table_out=s["table_out"],
                   lengths_out=s["lengths_out"], refs_out=s["refs_out"])
    moved = kda.pages_compact(s["pool"], s["table_out"], s["refs_out"])
    return moved, s["table_out"], s["lengths_out"], s["refs_out"], s["pool"]


def _softplus(z):
    return z.clamp(min=0) + torch.log1p(torch.exp(-z.abs()))


def _plain_scan(s, c, Q=64):
    """Chunks of Q tokens: products inside a chunk, the chunks' states joined by a doubling scan."""
    H, G, N, P = c["H"], c["G"], c["N"], c["P"]
    dtype = s["x"].dtype
    x, b, cc, dt = s["x"], s["b"], s["c"], s["dt_raw"]
    L = max(Q, -(-s["longest"] // Q) * Q)
    at = torch.arange(L, device=x.device)
    if s["cu_seqlens"] is not None:
        cu = s["cu_seqlens"].long()
        live = at[None] < (cu[1:] - cu[:-1])[:, None]                      # [rows, L]
        src = (cu[:-1, None] + at[None]).clamp(max=c["T"] - 1)
        x, b, cc, dt = x[0][src], b[0][src], cc[0][src], dt[0][src]
    else:
        live = (at < c["T"])[None].expand(c["B"], L)
        src = at.clamp(max=c["T"] - 1)
        x, b, cc, dt = x[:, src], b[:, src], cc[:, src], dt[:, src]
    rows, nc = x.shape[0], L // Q
    delta = _softplus(dt.float() + s["dt_bias"]) * live[..., None]
    la = (delta * -torch.exp(s["a_log"])).view(rows, nc, Q, H).transpose(2, 3)          # [rows, nc, H, Q]
    delta = delta.view(rows, nc, Q, H).transpose(2, 3)
    x = (x.float() * live[..., None, None]).view(rows, nc, Q, H, P).transpose(2, 3)     # [rows, nc, H, Q, P]
    b = (b.float() * live[..., None, None]).view(rows, nc, Q, G, N).transpose(2, 3)
    cc = (cc.float() * live[..., None, None]).view(rows, nc, Q, G, N).transpose(2, 3)
    cum = la.cumsum(-1)
    after = torch.cat([la.flip(-1).cumsum(-1).flip(-1)[..., 1:], torch.zeros_like(la[..., :1])], -1)
    lower = at[:Q, None] >= at[None, :Q]
    decay = torch.exp((cum[..., :, None] - cum[..., None, :]).masked_fill(~lower, -math.inf))
    m = (cc @ b.transpose(-1, -2)).repeat_interleave(H // G, 2) * decay * delta[..., None, :]
    y = m @ x
    del m, decay
    bw = b.repeat_interleave(H // G, 2) * (delta * torch.exp(after))[..., None]
    first = torch.zeros_like(s["x"], dtype=torch.float32).new_zeros(rows, 1, H, N, P)
    if s["initial_state"] is not None:
        first = s["initial_state"][:, None]
    st = torch.cat([first, bw.transpose(-1, -2) @ x], 1)                                # [rows, nc + 1, H, N, P]
    dec = torch.cat([torch.ones_like(la[:, :1, :, 0]), torch.exp(la.sum(-1))], 1)
    step = 1
    while step <= nc:
        st = torch.cat([st[:, :step], st[:, step:] + dec[:, step:, :, None, None] * st[:, :-step]], 1)
        dec = torch.cat([dec[:, :step], dec[:, step:] * dec[:, :-step]], 1)
        step *= 2
    y = y + torch.exp(cum)[..., None] * (cc.repeat_interleave(H // G, 2) @ st[:, :-1])
    y = y + s["d_skip"][:, None, None] * x
    y = y.transpose(2, 3).reshape(rows, L, H, P)
    y = y[live][None] if s["cu_seqlens"] is not None else y[:, :c["T"]]
    return y.to(dtype).contiguous(), st[:, -1].contiguous()


def _plain_ssm_step(s, c):
    rep = c["H"] // c["G"]
    on = s["slots"] >= 0
    old = s["state"][s["slots"].clamp(min=0).long()]
    delta = _softplus(s["dt_raw"].float() + s["dt_bias"])
    b = s["b"].float().repeat_interleave(rep, 1)
    cc = s["c"].float().repeat_interleave(rep, 1)
    x = s["x"].float()
    new = torch.exp(delta * -torch.exp(s["a_log"]))[..., None, None] * old
    new = new + (delta[..., None] * b)[..., None] * x[:, :, None, :]
    y = (cc[..., None] * new).sum(2) + s["d_skip"][:, None] * x
    s["state_out"][s["slots"][on].long()] = new[on]
    return (y * on[:, None, None]).to(s["x"].dtype), s["state_out"]


def _plain_decode(s, c):
    rep = c["H"] // c["Hk"]
    on = s["slots"] >= 0
    old = s["state"][s["slots"].clamp(min=0).long()]
    unit = lambda t: t / torch.sqrt((t * t).sum(-1, keepdim=True) + NORM_EPS)  # noqa: E731
    q = unit(s["q"].float()).repeat_interleave(rep, 1)
    k = unit(s["k"].float()).repeat_interleave(rep, 1)
    z = s["g_raw"].float() + s["dt_bias"].view(c["H"], c["K"])
    ea = torch.exp(s["a_log"])[:, None]
    g = -ea * _softplus(z) if c["gate"] == "softplus" else -5.0 / (1.0 + torch.exp(-ea * z))
    beta = 1.0 / (1.0 + torch.exp(-s["beta_raw"].float()))
    new = torch.exp(g)[..., None] * old
    u = beta[..., None] * (s["v"].float() - (k[..., None] * new).sum(2))
    new = new + k[..., None] * u[:, :, None, :]
    out = c["K"] ** -0.5 * (q[..., None] * new).sum(2)
    s["state_out"][s["slots"][on].long()] = new[on]
    return (out * on[:, None, None]).to(s["q"].dtype), s["state_out"]


def _plain_conv(s, c):
    B, T, C, W = (c[k] for k in ("B", "T", "C", "W"))
    x, hist = s["x"].reshape(B * T, C), s["initial_history"]
    t = torch.arange(B * T, device=x.device)
    if s["cu_seqlens"] is not None:
        cu = s["cu_seqlens"].long()
    else:
        cu = torch.arange(B + 1, device=x.device) * T
    row = (t[:, None] >= cu[None, 1:]).sum(1)                               # the token's segment
    tap = t[:, None] - (W - 1) + torch.arange(W, device=x.device)           # [tokens, W]
    before = tap - cu[row][:, None]                                         # below 0: in the history
    old = hist[row[:, None], (before + W - 1).clamp(0, W - 2)]              # [tokens, W, C]
    win = torch.where((before >= 0)[..., None], x[tap.clamp(min=0)], old).float()
    a = (win * s["weight"].t()[None]).sum(1) + s["bias"]
    y = _silu(a).to(x.dtype).view(B, T, C)
    back = cu[1:, None] - (W - 1) + torch.arange(W - 1, device=x.device)    # the last W - 1 inputs of each segment
    rel = back - cu[:-1, None]
    seg = torch.arange(hist.shape[0], device=x.device)[:, None]
    last = torch.where((rel >= 0)[..., None], x[back.clamp(min=0)], hist[seg, (rel + W - 1).clamp(0, W - 2)])
    return y, last


def _plain_conv_step(s, c):
    on = s["slots"] >= 0
    win = torch.cat([s["history"][s["slots"].clamp(min=0).long()], s["x"][:, None]], 1)     # [B, W, C]
    a = (win.float() * s["weight"].t()[None]).sum(1) + s["bias"]
    s["history_out"][s["slots"][on].long()] = win[on][:, 1:]
    return (_silu(a) * on[:, None]).to(s["x"].dtype), s["history_out"]


def _plain_fork(s, c):
    pt = c["page_tokens"]
    p, ch = s["parents"].long(), s["children"].long()
    n = s["lengths"][p].long()
    full, need = n // pt, n % pt != 0
    free = (s["refs"] <= 0).nonzero()[:, 0]
    rank = need.long().cumsum(0) - need.long()
    ok = ~need | (rank < free.numel())
    page = free[rank.clamp(max=max(0, free.numel() - 1))] if free.numel() else rank
    rows = s["table"][p]
    col = torch.arange(c["row"], device=p.device)[None]
    shared = (col < full[:, None]) & ok[:, None]
    fresh = (col == full[:, None]) & (need & ok)[:, None]
    child = torch.where(shared, rows, torch.where(fresh, page[:, None].to(torch.int32), -1))
    s["table_out"].copy_(s["table"])
    s["lengths_out"].copy_(s["lengths"])
    s["refs_out"].copy_(s["refs"])
    s["table_out"][ch[ok]] = child[ok]
    s["lengths_out"][ch[ok]] = s["lengths"][p][ok]
    s["refs_out"].index_add_(0, rows[shared].long(), torch.ones_like(rows[shared]))
    took = need & ok
    s["refs_out"][page[took]] = 1
    src = rows.gather(1, full.clamp(max=c["row"] - 1)[:, None])[:, 0].long()[took]
    s["pool"][:, page[took]] = s["pool"][:, src]
    return ok.to(torch.int32), s["table_out"], s["lengths_out"], s["refs_out"], s["pool"]


def _plain_compact(s, c):
    gone = s["gone"].long()
    rows = s["table"][gone]
    s["table_out"].copy_(s["table"])
    s["lengths_out"].copy_(s["lengths"])
    s["refs_out"].copy_(s["refs"])
    s["refs_out"].index_add_(0, rows[rows >= 0].long(), -torch.ones_like(rows[rows >= 0]))
    s["table_out"][gone] = -1
    s["lengths_out"][gone] = 0
    refs = s["refs_out"].clone()
    live = (refs > 0).nonzero()[:, 0]
    held = live.numel()
    src = live[live >= held].flip(0)
    dst = (refs[:held] <= 0).nonzero()[:, 0]
    moved = torch.where(refs > 0, torch.arange(c["pages"], device=refs.device), -1)
    moved[src] = dst
    s["pool"][:, dst] = s["pool"][:, src]
    s["refs_out"].zero_()
    s["refs_out"][:held] = refs[:held]
    s["refs_out"][dst] = refs[src]
    table = s["table_out"]
    s["table_out"].copy_(torch.where(table >= 0, moved[table.clamp(min=0).long()].to(torch.int32), -1))
    return moved.to(torch.int32), s["table_out"], s["lengths_out"], s["refs_out"], s["pool"]


# ------------------------------------------------------------------------------------------------ work


def work(case):
    c = case
    es = 2 if c.get("dtype") == "bf16" else 4
    if c["kind"] == "scan":
        tokens, rows = c["B"] * c["T"], c["docs"] or c["B"]
        state = rows * c["H"] * c["N"] * c["P"] * 4
        return {"bytes": tokens * (2 * c["H"] * c["P"] + 2 * c["G"] * c["N"] + c["H"]) * es + state * (1 + c["init"]),
                "flops": 5.0 * tokens * c["H"] * c["N"] * c["P"]}
    if c["kind"] in ("ssm_step", "conv_step", "decode"):
        on = c["B"] - (c["B"] + 0) // 7
        if c["kind"] == "ssm_step":
            cell, io, per = c["H"] * c["N"] * c["P"], 2 * c["H"] * c["P"] + 2 * c["G"] * c["N"] + c["H"], 5
            return {"bytes": on * (8 * cell + io * es), "flops": float(per * on * cell)}
        if c["kind"] == "decode":
            cell = c["H"] * c["K"] * c["V"]
            io = 2 * c["Hk"] * c["K"] + 2 * c["H"] * c["V"] + c["H"] * c["K"] + c["H"]
            return {"bytes": on * (8 * cell + io * es), "flops": 7.0 * on * cell}
        return {"bytes": on * c["C"] * (2 + 2 * (c["W"] - 1)) * es + 4 * c["C"] * (c["W"] + 1),
                "flops": 2.0 * on * c["C"] * (c["W"] + 2)}
    if c["kind"] == "conv":
        tokens, rows = c["B"] * c["T"], c["docs"] or c["B"]
        return {"bytes": (2 * tokens + 2 * rows * (c["W"] - 1)) * c["C"] * es + 4 * c["C"] * (c["W"] + 1),
                "flops": 2.0 * tokens * c["C"] * (c["W"] + 2)}
    page, tables = 4 * c["layers"] * c["words"], 8 * (c["seqs"] * (c["row"] + 1) + c["pages"])
    if c["kind"] == "fork":
        partial = 1.0 - 1.0 / c["page_tokens"]           # share of lengths that end inside a page
        return {"bytes": 2 * page * c["forks"] * partial + tables, "flops": 0}
    held = c["seqs"] * (c["row"] + 1) / 2 * (1 - c["gone"] / c["seqs"])
    return {"bytes": 2 * page * held * (1 - held / c["pages"]) + tables, "flops": 0}


# ----------------------------------------------------------------------------------------------- exact


def exact(case, seed):
    make = globals().get("_exact_" + case["kind"])
    return make(prepare(case, seed), case) if make else None


def _d(t):
    return t.double()


def _exact_scan(s, c):
    """The recurrence token by token, all rows at once."""
    G, R, N, P, H = c["G"], c["H"] // c["G"], c["N"], c["P"], c["H"]
    if s["cu_seqlens"] is None:
        starts, sizes = [i * c["T"] for i in range(c["B"])], [c["T"]] * c["B"]
    else:
        cu = s["cu_seqlens"].tolist()
        starts, sizes = cu[:-1], [e - a for a, e in zip(cu, cu[1:])]
    rows, tokens = len(starts), c["B"] * c["T"]
    z = _d(s["dt_raw"]).reshape(tokens, G, R) + _d(s["dt_bias"]).view(G, R)
    delta = torch.logaddexp(z, torch.zeros_like(z))
    alpha = torch.exp(-torch.exp(_d(s["a_log"])).view(G, R) * delta)[..., None, None]
    x = _d(s["x"]).reshape(tokens, G, R, 1, P)
    dx = delta[..., None, None] * x
    b, cc = _d(s["b"]).reshape(tokens, G, 1, N, 1), _d(s["c"]).reshape(tokens, G, 1, N, 1)
    y = torch.empty(tokens, G, R, P, dtype=torch.float64, device=x.device)
    S = torch.zeros(rows, G, R, N, P, dtype=torch.float64, device=x.device)
    if s["initial_state"] is not None:
        S += _d(s["initial_state"]).view(rows, G, R, N, P)
    # rows by falling length: at step t the first `live` of them go on
    order = sorted(range(rows), key=lambda i: -sizes[i])
    S = S[order]
    first = torch.tensor([starts[i] for i in order], device=x.device)
    live = rows
    for t in range(max(sizes)):
        while sizes[order[live - 1]] <= t:
            live -= 1
        at = slice(starts[order[0]] + t, starts[order[0]] + t + 1) if live == 1 else first[:live] + t
        now = S[:live]
        now.mul_(alpha[at]).addcmul_(b[at], dx[at])
        y[at] = (cc[at] * now).sum(-2)
    y += _d(s["d_skip"]).view(G, R, 1) * x[..., 0, :]
    back = torch.empty(rows, dtype=torch.long, device=x.device)
    back[torch.tensor(order, device=x.device)] = torch.arange(rows, device=x.device)
    return y.view(c["B"], c["T"], H, P), S[back].view(rows, H, N, P)


def _exact_ssm_step(s, c):
    out, pool = torch.zeros(c["B"], c["H"], c["P"], dtype=torch.float64, device=s["x"].device), _d(s["state"])
    head = torch.arange(c["H"], device=out.device) // (c["H"] // c["G"])
    z = _d(s["dt_raw"]) + _d(s["dt_bias"])
    delta = torch.logaddexp(z, torch.zeros_like(z))
    for r, slot in enumerate(s["slots"].tolist()):
        if slot >= 0:
            grow = torch.einsum("h,hn,hp->hnp", delta[r], _d(s["b"])[r][head], _d(s["x"])[r])
            pool[slot] = torch.exp(-delta[r] * torch.exp(_d(s["a_log"])))[:, None, None] * pool[slot] + grow
            out[r] = torch.einsum("hn,hnp->hp", _d(s["c"])[r][head], pool[slot])
            out[r] += _d(s["d_skip"])[:, None] * _d(s["x"])[r]
    return out, pool


def _exact_decode(s, c):
    out, pool = torch.zeros(c["B"], c["H"], c["V"], dtype=torch.float64, device=s["q"].device), _d(s["state"])
    head = torch.arange(c["H"], device=out.device) // (c["H"] // c["Hk"])
    z = _d(s["g_raw"]) + _d(s["dt_bias"]).view(c["H"], c["K"])
    ea = torch.exp(_d(s["a_log"]))[:, None]
    if c["gate"] == "softplus":
        g = -ea * torch.logaddexp(z, torch.zeros_like(z))
    else:
        g = -5.0 * torch.sigmoid(ea * z)
    for r, slot in enumerate(s["slots"].tolist()):
        if slot >= 0:
            q, k = _d(s["q"])[r], _d(s["k"])[r]
            q = (q / (q.square().sum(-1, keepdim=True) + NORM_EPS).sqrt())[head]
            k = (k / (k.square().sum(-1, keepdim=True) + NORM_EPS).sqrt())[head]
            kept = torch.exp(g[r])[..., None] * pool[slot]
            miss = _d(s["v"])[r] - torch.einsum("hk,hkv->hv", k, kept)
            pool[slot] = kept + torch.einsum("h,hk,hv->hkv", torch.sigmoid(_d(s["beta_raw"])[r]), k, miss)
            out[r] = torch.einsum("hk,hkv->hv", q, pool[slot]) / math.sqrt(c["K"])
    return out, pool


def _exact_conv(s, c):
    W = c["W"]
    flat = s["x"].reshape(-1, c["C"])
    if s["cu_seqlens"] is None:
        cu = [i * c["T"] for i in range(c["B"] + 1)]
    else:
        cu = s["cu_seqlens"].tolist()
    ys, last = [], []
    for r in range(len(cu) - 1):
        seq = torch.cat([s["initial_history"][r], flat[cu[r]:cu[r + 1]]])
        n = cu[r + 1] - cu[r]
        a = _d(s["bias"]).expand(n, -1)
        for i in range(W):
            a = a + _d(s["weight"])[:, i] * _d(seq[i:i + n])
        ys.append(a * torch.sigmoid(a))
        last.append(_d(seq[n:]))
    return torch.cat(ys).view(c["B"], c["T"], c["C"]), torch.stack(last)


def _exact_conv_step(s, c):
    out, pool = torch.zeros(c["B"], c["C"], dtype=torch.float64, device=s["x"].device), _d(s["history"])
    for r, slot in enumerate(s["slots"].tolist()):
        if slot >= 0:
            seq = torch.cat([pool[slot], _d(s["x"])[r][None]])
            a = (seq * _d(s["weight"]).t()).sum(0) + _d(s["bias"])
            out[r], pool[slot] = a * torch.sigmoid(a), seq[1:]
    return out, pool
