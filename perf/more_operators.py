"""Cases of the gated linear recurrence (its scan over prompts, the scan's gradients, single tokens on a pool of
states) and of attention over the pages of a key/value cache (new keys and values into their pages, a chunk of new
tokens or a single token attending to everything before it).

``run`` computes a case in its plain form (elementary torch operations in 32 bits) while ``own`` is false,
and through the package's entry points while it is true.  ``exact`` gives the same outputs in 64 bits,
computed token by token (the recurrence) or query head by query head (attention) from the definitions.

The gated linear recurrence, per channel:
    log a_t = -exp(a_log) sigmoid(g_t),   h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t,   y_t = h_t

Pages hold [2, Hkv, page_tokens, D]: keys, then values, head by head.  The n new tokens of a row are the last n of its
``lengths`` tokens; the one at position p attends to the positions 0 .. p, with a window to the last ``window`` of them.
"""
from __future__ import annotations

import math

import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # a chat turn's short prompt on a small layer: latency
        dict(name="scan short", kind="scan", B=1, T=37, C=512, docs=0, dtype="bf16", init=True),
        # a packed prefill batch of continued conversations: documents of any length, each from its own state
        dict(name="scan packed", kind="scan", B=1, T=16384, C=4096, docs=12, dtype="bf16", init=True),
        # a training step's mixer, forward and backward, at the training benchmark's tokens
        dict(name="train", kind="train", B=4, T=4096, C=4096, docs=0, dtype="bf16", init=False),
        # the same in fp32 on packed documents, an odd number of channels: the evaluation path
        dict(name="train fp32 odd", kind="train", B=1, T=1021, C=515, docs=5, dtype="fp32", init=True),
        # one user's next token
        dict(name="step one", kind="step", B=1, C=4096, slots=16, dtype="bf16"),
        # a serving batch's next token, rows scattered over the pool, some rows idle
        dict(name="step batch", kind="step", B=128, C=4096, slots=160, dtype="bf16"),
        # the keys and values of a packed prefill chunk into their pages
        dict(name="append chunk", kind="append", rows=8, T=8192, past=4096, Hkv=8, D=128, page_tokens=16, dtype="bf16"),
        # a batch's next token into its pages
        dict(name="append batch", kind="append", rows=128, T=0, past=2000, Hkv=8, D=128, page_tokens=16, dtype="bf16"),
        # one user's next token over a long conversation
        dict(name="attention one", kind="attention", rows=1, T=0, past=32768, Hq=32, Hkv=8, D=128, page_tokens=16,
             window=0, dtype="bf16"),
        # a serving batch's next token: ragged contexts, rows in no order, some idle, one without a token yet
        dict(name="attention batch", kind="attention", rows=64, T=0, past=8192, Hq=32, Hkv=8, D=128, page_tokens=16,
             window=0, dtype="bf16"),
        # chunked prefill: chunks of new tokens over what each request has in the cache already
        dict(name="attention chunk", kind="attention", rows=8, T=8192, past=16384, Hq=32, Hkv=8, D=128, page_tokens=16,
             window=0, dtype="bf16"),
        # the fp32 evaluation path at odd sizes with a sliding window
        dict(name="attention fp32 odd", kind="attention", rows=3, T=301, past=700, Hq=6, Hkv=2, D=40, page_tokens=24,
             window=257, dtype="fp32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["scan", "scan", "train", "train", "step", "append", "attention", "attention", "attention"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    if kind in ("scan", "train"):
        C = rng.choice([_log(rng, 1, 600), 8 * _log(rng, 8, 512)])
        docs = rng.choice([0, 0, rng.randint(1, 24)])
        return dict(kind=kind, B=1 if docs else rng.choice([1, 1, 2, 3]), T=_log(rng, 1, 8192), C=C, docs=docs, dtype=dtype,
                    init=rng.random() < 0.5)
    if kind == "step":
        B = _log(rng, 1, 128)
        return dict(kind=kind, B=B, C=rng.choice([_log(rng, 1, 600), 8 * _log(rng, 8, 1024)]), slots=B + rng.randint(0, 40),
                    dtype=dtype)
    Hkv = rng.choice([1, 2, 3, 4, 8])
    D = rng.choice([64, 128, 128, 8 * rng.randint(2, 16), 8 * rng.randint(17, 32)])
    page_tokens = rng.choice([1, 16, 16, 24, 64, 128])
    one = rng.random() < 0.5                     # a token a row, or packed chunks
    if kind == "append":
        rows = _log(rng, 1, 128) if one else rng.randint(1, 12)
        return dict(kind=kind, rows=rows, T=0 if one else _log(rng, 1, 8192), past=_log(rng, 1, 4096), Hkv=Hkv, D=D,
                    page_tokens=page_tokens, dtype=dtype)
    cost = 1 if dtype == "bf16" and D <= 128 else 8
    return dict(kind=kind, rows=_log(rng, 1, 64) if one else rng.randint(1, 8), T=0 if one else _log(rng, 1, 4096 // cost),
                past=_log(rng, 1, 8192 // cost), Hq=Hkv * rng.choice([1, 2, 3, 4, 8]), Hkv=Hkv, D=D, page_tokens=page_tokens,
                window=rng.choice([0, 0, _log(rng, 1, 4096)]), dtype=dtype)


# ---------------------------------------------------------------------------------------------- inputs


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEVICE, dtype=torch.float32)


def _rand(gen, *shape):
    return torch.rand(shape, generator=gen, device=DEVICE, dtype=torch.float32)


def _sigmoid(z):
    return 1.0 / (1.0 + torch.exp(-z))


def _lengths(gen, tokens, docs):
    """Lengths of `docs` documents (empty ones among them) that cover the tokens."""
    cuts = torch.randint(0, tokens + 1, (docs - 1,), generator=gen, device=DEVICE).sort().values.tolist()
    return [b - a for a, b in zip([0, *cuts], [*cuts, tokens])]


def _offsets(lengths):
    return torch.tensor([0, *lengths], device=DEVICE).cumsum(0).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    return dict(globals()["_prepare_" + case["kind"]](case, gen), case=case)


def _decay(gen, C):
    # with an open gate a token keeps 0.9 to 0.999 of the state
    return torch.log(-torch.log(0.9 + 0.099 * _rand(gen, C)))


def _prepare_scan(c, gen):
    B, T, C, dt = c["B"], c["T"], c["C"], DTYPES[c["dtype"]]
    x = _randn(gen, B, T, C)
    # x comes out of the convolution and its SiLU, the two gates are halves of one projection
    gates = _randn(gen, B, T, 2 * C).to(dt)
    g_raw, i_raw = gates.chunk(2, dim=-1)
    lengths = _lengths(gen, T, c["docs"]) if c["docs"] else None
    return dict(x=(x * _sigmoid(x)).to(dt), g_raw=g_raw, i_raw=i_raw, a_log=_decay(gen, C),
                initial_state=_randn(gen, c["docs"] or B, C) if c["init"] else None,
                cu_seqlens=_offsets(lengths) if lengths else None)


def _prepare_train(c, gen):
    s = _prepare_scan(c, gen)
    return dict(s, dy=_randn(gen, c["B"], c["T"], c["C"]).to(DTYPES[c["dtype"]]),
                dfinal_state=_randn(gen, c["docs"] or c["B"], c["C"]) if c["init"] else None)


def _prepare_step(c, gen):
    B, C, dt = c["B"], c["C"], DTYPES[c["dtype"]]
    x = _randn(gen, B, C)
    g_raw, i_raw = _randn(gen, B, 2 * C).to(dt).chunk(2, dim=-1)
    slots = torch.randperm(c["slots"], generator=gen, device=DEVICE)[:B].to(torch.int32)
    slots[6::7] = -1
    state = _randn(gen, c["slots"], C)
    return dict(x=(x * _sigmoid(x)).to(dt), g_raw=g_raw, i_raw=i_raw, a_log=_decay(gen, C), slots=slots, state=state,
                state_out=state.clone())


def _prepare_cache(c, gen):
    """The pages, table and lengths of `rows` requests whose new tokens are counted in the lengths already; table rows
    in no order, a few rows idle where there are many (their tokens, if any, are nobody's)."""
    rows, pt = c["rows"], c["page_tokens"]
    new = [1] * rows if c["T"] == 0 else _lengths(gen, c["T"], rows)
    past = torch.randint(0, c["past"] + 1, (rows,), generator=gen, device=DEVICE).tolist()
    if rows == 1:
        past = [c["past"] - new[0] if c["past"] > new[0] else c["past"]]
    held = [p + n for p, n in zip(past, new)]
    if c["T"] == 0 and rows >= 16:
        held[3] = 0                       # a request whose first token is not in the cache: nothing to write or attend to
    spare = 2
    order = torch.randperm(rows + spare, generator=gen, device=DEVICE)[:rows]
    where = order.tolist()
    M = -(-(c["past"] + max(1, c["T"])) // pt) + 1
    pages = rows * (c["past"] // pt + 2) + c["T"] // pt + spare          # (room for any lengths)
    perm = torch.randperm(pages, generator=gen, device=DEVICE).to(torch.int32)
    table = torch.full((rows + spare, M), -1, dtype=torch.int32, device=DEVICE)
    lengths = torch.zeros(rows + spare, dtype=torch.int32, device=DEVICE)
    at = 0
    for r, n in enumerate(held):
        k = -(-n // pt)
        table[where[r], :k] = perm[at:at + k]
        lengths[where[r]] = n
        at += k
    seqs = order.to(torch.int32)
    idle = [r for r in range(rows) if rows >= 16 and r % 13 == 6]
    for r in idle:
        seqs[r] = -1
    pool = torch.randn((pages, 2, c["Hkv"], pt, c["D"]), generator=gen, device=DEVICE, dtype=DTYPES[c["dtype"]])
    cu = None if c["T"] == 0 else _offsets(new)
    return dict(pool=pool, table=table, lengths=lengths, seqs=seqs, cu_seqlens=cu,
                host=[(where[r], new[r], held[r]) if r not in idle else (-1, new[r], 0) for r in range(rows)])


def _prepare_append(c, gen):
    s = _prepare_cache(c, gen)
    lead = (c["rows"], 1) if c["T"] == 0 else (1, c["T"])
    kv = _randn(gen, *lead, 2 * c["Hkv"] * c["D"]).to(DTYPES[c["dtype"]])       # one projection's output
    k, v = kv.chunk(2, dim=-1)
    return dict(s, k=k.unflatten(-1, (c["Hkv"], c["D"])), v=v.unflatten(-1, (c["Hkv"], c["D"])))


def _prepare_attention(c, gen):
    s = _prepare_cache(c, gen)
    lead = (c["rows"], 1) if c["T"] == 0 else (1, c["T"])
    return dict(s, q=_randn(gen, *lead, c["Hq"], c["D"]).to(DTYPES[c["dtype"]]))


# ------------------------------------------------------------------------------------------------ runs


def run(state):
    return globals()[("_own_" if own else "_plain_") + state["case"]["kind"]](state, state["case"])


def _own_scan(s, c):
    import gated_delta_rule_sm_gb300 as kda
    return kda.gated_scan(s["x"], s["g_raw"], s["i_raw"], s["a_log"], cu_seqlens=s["cu_seqlens"],
                          initial_state=s["initial_state"], output_final_state=True)


def _own_train(s, c):
    import gated_delta_rule_sm_gb300 as kda
    saved = torch.empty(kda.gated_scan_saved_size(s["x"]), dtype=torch.uint8, device=s["x"].device)
    y, last = kda.gated_scan(s["x"], s["g_raw"], s["i_raw"], s["a_log"], cu_seqlens=s["cu_seqlens"],
                             initial_state=s["initial_state"], output_final_state=True, saved=saved)
    grads = kda.gated_scan_backward(s["x"], s["g_raw"], s["i_raw"], s["a_log"], s["dy"], cu_seqlens=s["cu_seqlens"],
                                    initial_state=s["initial_state"], dfinal_state=s["dfinal_state"], saved=saved)
    return y, last, grads["dx"], grads["dg_raw"], grads["di_raw"], grads["da_log"], grads["dinitial_state"]


def _own_step(s, c):
    import gated_delta_rule_sm_gb300 as kda
    return kda.gated_step(s["x"], s["g_raw"], s["i_raw"], s["a_log"], state=s["state"], slots=s["slots"],
                          state_out=s["state_out"])


def _own_append(s, c):
    import gated_delta_rule_sm_gb300 as kda
    return kda.pages_append(s["pool"], s["table"], s["lengths"], s["k"], s["v"], seqs=s["seqs"], cu_seqlens=s["cu_seqlens"])


def _own_attention(s, c):
    import gated_delta_rule_sm_gb300 as kda
    return kda.pages_attention(s["q"], s["pool"], s["table"], s["lengths"], scale=c["D"] ** -0.5, seqs=s["seqs"],
                               cu_seqlens=s["cu_seqlens"], window=c["window"])


def _gates(s):
    """Log-decays, decays, input factors and scaled inputs.  (The decays in 64 bits and rounded once: they are close to 1,
    and a long row multiplies thousands of them.)"""
    log_a = -torch.exp(s["a_log"].double()) * _sigmoid(s["g_raw"].double())
    beta = torch.sqrt(-torch.expm1(2.0 * log_a))
    return log_a.float(), torch.exp(log_a).float(), beta.float(), _sigmoid(s["i_raw"].float()) * s["x"].float()


def _doubling(a, b):
    """h_t = a_t h_{t-1} + b_t along axis 1, from zero."""
    step = 1
    while step < a.shape[1]:
        b = torch.cat([b[:, :step], b[:, step:] + a[:, step:] * b[:, :-step]], 1)
        a = torch.cat([a[:, :step], a[:, step:] * a[:, :-step]], 1)
        step *= 2
    return b


def _edges(s, c):
    """(row of the batch, first token, last token) of the segments that hold tokens, and which they are."""
    if s["cu_seqlens"] is None:
        n = torch.arange(c["B"], device=s["x"].device)
        return n, torch.zeros_like(n), torch.full_like(n, c["T"] - 1), n
    cu = s["cu_seqlens"].long()
    n = (cu[1:] > cu[:-1]).nonzero()[:, 0]
    return torch.zeros_like(n), cu[:-1][n], cu[1:][n] - 1, n


def _plain_states(s, c, a, b):
    """The states after every token, and those before."""
    row, first, _, n = _edges(s, c)
    b, carry = b.clone(), a.clone()
    if s["initial_state"] is not None:
        b[row, first] += a[row, first] * s["initial_state"][n]
    carry[row, first] = 0.0
    h = _doubling(carry, b)
    before = torch.cat([torch.zeros_like(h[:, :1]), h[:, :-1]], 1)
    before[row, first] = s["initial_state"][n] if s["initial_state"] is not None else 0.0
    return h, before


def _plain_last(s, c, h):
    row, _, last, n = _edges(s, c)
    rows = c["docs"] or c["B"]
    out = s["initial_state"].clone() if s["initial_state"] is not None else torch.zeros(rows, c["C"], device=h.device)
    out[n] = h[row, last]
    return out


def _plain_scan(s, c):
    _, a, beta, u = _gates(s)
    h, _ = _plain_states(s, c, a, beta * u)
    return h.to(s["x"].dtype), _plain_last(s, c, h)


def _plain_train(s, c):
    log_a, a, beta, u = _gates(s)
    h, before = _plain_states(s, c, a, beta * u)
    row, first, last, n = _edges(s, c)
    # the gradient of h_t: dy_t + a_{t+1} times that of h_{t+1}, from the end of every segment
    after = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    after[row, last] = 0.0
    dh = s["dy"].float().clone()
    if s["dfinal_state"] is not None:
        dh[row, last] += s["dfinal_state"][n]
    dh = _doubling(after.flip(1), dh.flip(1)).flip(1)
    dlog = dh * (a * before - u * a * a / beta)
    sg, si, du = _sigmoid(s["g_raw"].float()), _sigmoid(s["i_raw"].float()), dh * beta
    rows = c["docs"] or c["B"]
    dinit = torch.zeros(rows, c["C"], device=a.device) if s["dfinal_state"] is None else s["dfinal_state"].clone()
    dinit[n] = (a * dh)[row, first]
    return (h.to(s["x"].dtype), _plain_last(s, c, h), du * si, dlog * log_a * (1.0 - sg), du * s["x"].float() * si * (1.0 - si),
            (dlog * log_a).sum((0, 1), dtype=torch.float64).float(), dinit)


def _plain_step(s, c):
    on = s["slots"] >= 0
    old = s["state"][s["slots"].clamp(min=0).long()]
    _, a, beta, u = _gates(s)
    h = a * old + beta * u
    s["state_out"][s["slots"][on].long()] = h[on]
    return (h * on[:, None]).to(s["x"].dtype), s["state_out"]


def _row_tokens(s, c):
    """(table row, its tokens, the new ones' slice of the flattened tokens, their positions) of every row that has some."""
    start = 0
    for seq, n, total in s["host"]:
        if seq >= 0 and total > 0 and n > 0:
            yield seq, total, slice(start, start + n), torch.arange(total - n, total, device=s["pool"].device)
        start += n


def _plain_append(s, c):
    k, v = s["k"].flatten(0, 1), s["v"].flatten(0, 1)
    page, within, token = [], [], []
    for seq, _, at, pos in _row_tokens(s, c):
        page.append(s["table"][seq].long()[pos // c["page_tokens"]])
        within.append(pos % c["page_tokens"])
        token.append(torch.arange(at.start, at.stop, device=pos.device))
    if page:
        page, within, token = torch.cat(page), torch.cat(within), torch.cat(token)
        s["pool"][page, 0, :, within] = k[token]
        s["pool"][page, 1, :, within] = v[token]
    return s["pool"]


def _plain_attention(s, c):
    q = s["q"].flatten(0, 1)
    out = torch.zeros_like(q)
    pt, R = c["page_tokens"], c["Hq"] // c["Hkv"]
    for seq, total, at, pos in _row_tokens(s, c):
        n = pos.numel()
        pages = s["table"][seq, :-(-total // pt)].long()
        kv = s["pool"][pages].float()                                             # [pages, 2, Hkv, pt, D]
        kv = kv.permute(1, 2, 0, 3, 4).reshape(2, c["Hkv"], -1, c["D"])[:, :, :total]
        qs = q[at].float().view(n, c["Hkv"], R, c["D"]).permute(1, 2, 0, 3).reshape(c["Hkv"], R * n, c["D"])
        score = (qs @ kv[0].transpose(1, 2)).view(c["Hkv"], R, n, total) * c["D"] ** -0.5
        key = torch.arange(total, device=pos.device)
        hide = key[None] > pos[:, None]
        if c["window"]:
            hide |= key[None] <= pos[:, None] - c["window"]
        score = score.masked_fill(hide, -math.inf)
        w = torch.exp(score - score.amax(-1, keepdim=True))
        w = w / w.sum(-1, keepdim=True)
        o = (w.view(c["Hkv"], R * n, total) @ kv[1]).view(c["Hkv"], R, n, c["D"])
        out[at] = o.permute(2, 0, 1, 3).reshape(n, c["Hq"], c["D"]).to(out.dtype)
    return out.view(s["q"].shape)


# ------------------------------------------------------------------------------------------------ work


def work(case):
    c = case
    es = 2 if c["dtype"] == "bf16" else 4
    if c["kind"] in ("scan", "train"):
        n, rows = c["B"] * c["T"] * c["C"], c["docs"] or c["B"]
        state = 4 * rows * c["C"]
        if c["kind"] == "scan":
            return {"bytes": 4 * n * es + state * (1 + c["init"]), "flops": 20.0 * n}
        # x, both gates and dy once, y and three gradients once; states and their gradients
        return {"bytes": n * (5 * es + 12) + state * (2 + 2 * c["init"]) + 8 * c["C"], "flops": 60.0 * n}
    if c["kind"] == "step":
        on = c["B"] - c["B"] // 7
        return {"bytes": on * c["C"] * (4 * es + 8), "flops": 20.0 * on * c["C"]}
    rows, new = c["rows"], c["T"] or c["rows"]
    past = c["past"] / 2 if rows > 1 else c["past"]          # on average
    if rows >= 16:
        on = rows - sum(r % 13 == 6 for r in range(rows))
        rows, new = on, new * on / rows
    token = 2 * c["Hkv"] * c["D"] * es
    if c["kind"] == "append":
        return {"bytes": 2 * new * token, "flops": 0}
    per = new / rows                                         # new tokens of a row
    seen = past + (per + 1) / 2                              # keys of a query
    read = past + per
    if c["window"]:
        seen, read = min(seen, c["window"]), min(read, c["window"] + per)
    return {"bytes": rows * read * token + 2 * new * c["Hq"] * c["D"] * es, "flops": 4.0 * new * seen * c["Hq"] * c["D"]}


# ----------------------------------------------------------------------------------------------- exact


def exact(case, seed):
    make = globals().get("_exact_" + case["kind"])
    return make(prepare(case, seed), case) if make else None


def _d(t):
    return t.double()


def _segments(s, c):
    """(first flattened token, tokens) of every segment."""
    if s["cu_seqlens"] is None:
        return [(r * c["T"], c["T"]) for r in range(c["B"])]
    cu = s["cu_seqlens"].tolist()
    return [(a, b - a) for a, b in zip(cu, cu[1:])]


def _exact_recurrence(s, c):
    """Token by token, segment by segment.  Returns the per-token factors, all states and the end states."""
    TT, C = c["B"] * c["T"], c["C"]
    rate = torch.exp(_d(s["a_log"]))
    open_ = torch.sigmoid(_d(s["g_raw"]).reshape(TT, C))
    a = torch.exp(-rate * open_)
    root = torch.sqrt((1.0 - a) * (1.0 + a)) if bool((a < 0.999).all()) else torch.sqrt(-torch.expm1(-2.0 * rate * open_))
    put = root * torch.sigmoid(_d(s["i_raw"]).reshape(TT, C)) * _d(s["x"]).reshape(TT, C)
    h = torch.empty(TT, C, dtype=torch.float64, device=a.device)
    ends = []
    for n, (first, size) in enumerate(_segments(s, c)):
        now = torch.zeros(C, dtype=torch.float64, device=a.device) if s["initial_state"] is None else _d(s["initial_state"][n])
        for t in range(first, first + size):
            now = torch.addcmul(put[t], a[t], now)
            h[t] = now
        ends.append(now)
    return open_, a, root, h, torch.stack(ends)


def _exact_scan(s, c):
    h, last = _exact_recurrence(s, c)[3:]
    return h.view(c["B"], c["T"], c["C"]), last


def _exact_train(s, c):
    """The chain rule backwards through h_t = a_t h_{t-1} + r_t k_t x_t with r_t^2 = 1 - a_t^2."""
    TT, C = c["B"] * c["T"], c["C"]
    open_, a, root, h, last = _exact_recurrence(s, c)
    keep, x = torch.sigmoid(_d(s["i_raw"]).reshape(TT, C)), _d(s["x"]).reshape(TT, C)
    grad = _d(s["dy"]).reshape(TT, C).clone()
    old = torch.empty_like(h)
    dinit = []
    for n, (first, size) in enumerate(_segments(s, c)):
        back = torch.zeros(C, dtype=torch.float64, device=a.device) if s["dfinal_state"] is None else _d(s["dfinal_state"][n])
        for t in range(first + size - 1, first - 1, -1):
            grad[t] += back
            back = a[t] * grad[t]
        dinit.append(back)
        if size:
            old[first] = 0.0 if s["initial_state"] is None else _d(s["initial_state"][n])
            old[first + 1:first + size] = h[first:first + size - 1]
    da = grad * (old - keep * x * a / root)                   # dr/da = -a / r
    drate = -da * a * open_                                   # a = exp(-rate open)
    dg = -da * a * torch.exp(_d(s["a_log"])) * open_ * (1.0 - open_)
    dput = grad * root
    shape = (c["B"], c["T"], C)
    return (h.view(shape), last, (dput * keep).view(shape), dg.view(shape), (dput * x * keep * (1.0 - keep)).view(shape),
            drate.sum(0) * torch.exp(_d(s["a_log"])), torch.stack(dinit))


def _exact_step(s, c):
    pool, y = _d(s["state"]), torch.zeros(c["B"], c["C"], dtype=torch.float64, device=s["x"].device)
    for r, slot in enumerate(s["slots"].tolist()):
        if slot >= 0:
            a = torch.exp(-torch.exp(_d(s["a_log"])) * torch.sigmoid(_d(s["g_raw"][r])))
            pool[slot] = a * pool[slot] + torch.sqrt(1.0 - a * a) * torch.sigmoid(_d(s["i_raw"][r])) * _d(s["x"][r])
            y[r] = pool[slot]
    return y, pool


def _exact_attention(s, c):
    """Each query head against its keys; the mask as a sum's range."""
    pt, R, D = c["page_tokens"], c["Hq"] // c["Hkv"], c["D"]
    q = _d(s["q"].flatten(0, 1))
    out = torch.zeros_like(q)
    start = 0
    for seq, n, held in s["host"]:
        if seq >= 0 and held:
            token = torch.arange(held, device=q.device)
            page, within = s["table"][seq].long()[token // pt], token % pt
            first = held - n
            rel = torch.arange(n, device=q.device)[:, None] + first - token[None]        # how far back a key is
            seen = (rel >= 0) & (rel < (c["window"] or held + 1))
            for head in range(c["Hkv"]):
                k, v = _d(s["pool"][page, 0, head, within]), _d(s["pool"][page, 1, head, within])
                for j in range(head * R, head * R + R):
                    z = torch.einsum("nd,kd->nk", q[start:start + n, j], k) / math.sqrt(D)
                    p = torch.softmax(torch.where(seen, z, torch.full_like(z, -math.inf)), -1)
                    out[start:start + n, j] = p @ v
        start += n
    return out.view(s["q"].shape)
