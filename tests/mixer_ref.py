"""Plain 64-bit references of the gated linear recurrence and of attention over paged keys and values, on the CPU."""
from __future__ import annotations

import math

import torch


def d(t):
    return t.detach().cpu().double()


def gated(x, g_raw, i_raw, a_log, offsets, state=None):
    """x, g_raw, i_raw [TT, C] in 64 bits; rows [offsets[n], offsets[n + 1]) from state [rows, C] (None: zero), token by token.
    Returns y [TT, C] and the end states; differentiable."""
    log_a = -torch.exp(a_log) * torch.sigmoid(g_raw)
    a, put = torch.exp(log_a), torch.sqrt(-torch.expm1(2 * log_a)) * torch.sigmoid(i_raw) * x
    ys, ends = [], []
    for n in range(len(offsets) - 1):
        h = torch.zeros_like(a_log) if state is None else state[n]
        for t in range(offsets[n], offsets[n + 1]):
            h = a[t] * h + put[t]
            ys.append(h)
        ends.append(h)
    return (torch.stack(ys) if ys else x), torch.stack(ends)


def gated_grads(x, g_raw, i_raw, a_log, offsets, state, dy, dlast):
    """Gradients of sum(dy y) + sum(dlast end states) by automatic differentiation: dict, and the sum of |terms| of da_log."""
    leaves = [d(t).requires_grad_() for t in (x, g_raw, i_raw)]
    rate = d(a_log).expand(x.shape).clone().requires_grad_()        # a copy per token: its gradients are da_log's terms
    s = torch.zeros(len(offsets) - 1, x.shape[1], dtype=torch.float64) if state is None else d(state)
    s = s.clone().requires_grad_()
    log_a = -torch.exp(rate) * torch.sigmoid(leaves[1])
    a, put = torch.exp(log_a), torch.sqrt(-torch.expm1(2 * log_a)) * torch.sigmoid(leaves[2]) * leaves[0]
    total = 0
    for n in range(len(offsets) - 1):
        h = s[n]
        for t in range(offsets[n], offsets[n + 1]):
            h = a[t] * h + put[t]
            total = total + (h * d(dy[t])).sum()
        if dlast is not None:
            total = total + (h * d(dlast[n])).sum()
    total.backward()
    return (dict(dx=leaves[0].grad, dg_raw=leaves[1].grad, di_raw=leaves[2].grad, da_log=rate.grad.sum(0), dinitial_state=s.grad),
            rate.grad.abs().sum(0))


def gated_back(x, g_raw, i_raw, a_log, offsets, state, dy, dlast):
    """The gradients by the chain rule, token by token, also where a decay is 1 or 0 in 64 bits: log a a / sqrt(1 - a^2) is then
    its limit, 0.  Returns them, and for each the sizes its errors go by: per channel M, H and U, the largest gradient of a
    state, state and input u = sigmoid(i) x, and per token the terms of d log a with M for the gradient, H and U for the state and u."""
    x, g, i, rate, dy = d(x), d(g_raw), d(i_raw), d(a_log), d(dy)
    log_a = -torch.exp(rate) * torch.sigmoid(g)
    a, root = torch.exp(log_a), torch.sqrt(-torch.expm1(2 * log_a))
    keep = torch.sigmoid(i)
    u = keep * x
    put = torch.where(root > 0, a * log_a / root.clamp(min=1e-300), torch.zeros_like(root))
    decay = torch.where(a > 0, a * log_a, torch.zeros_like(a))
    put = torch.where(a > 0, put, torch.zeros_like(put))
    old, dh, first = torch.zeros_like(x), torch.zeros_like(x), []
    for n in range(len(offsets) - 1):
        h = torch.zeros_like(rate) if state is None else d(state)[n]
        for t in range(offsets[n], offsets[n + 1]):
            old[t] = h
            h = a[t] * h + root[t] * u[t]
        m = torch.zeros_like(rate) if dlast is None else d(dlast)[n]
        for t in reversed(range(offsets[n], offsets[n + 1])):
            dh[t] = dy[t] + m
            m = a[t] * dh[t]
        first.append(m)
    dl = dh * (old * decay - u * a * put)
    grads = dict(dx=dh * root * keep, dg_raw=dl * torch.sigmoid(-g), di_raw=dh * root * u * torch.sigmoid(-i), da_log=dl.sum(0),
                 dinitial_state=torch.stack(first))
    M, H, U = dh.abs().amax(0), old.abs().amax(0), u.abs().amax(0)
    return grads, dict(M=M, H=H, U=U, X=x.abs().amax(0), log_a=log_a, root=root, keep=keep, terms=M * (H * decay.abs() + U * (a * put).abs()))


def rows_of(offsets, lengths, seqs):
    """(tokens of the call, table row, positions) of every row; table row None: idle."""
    for r, (a, b) in enumerate(zip(offsets, offsets[1:])):
        s = int(seqs[r])
        ok = 0 <= s < len(lengths)
        length = int(lengths[s]) if ok else 0
        yield range(a, b), s if ok else None, [length - (b - a) + i for i in range(b - a)], length


def append(pool, table, lengths, k, v, seqs, offsets):
    """k, v [tokens, Hkv, D] into a copy of pool [pages, 2, Hkv, pt, D]."""
    pool, pt = pool.clone(), pool.shape[3]
    for tokens, s, pos, _ in rows_of(offsets, lengths, seqs):
        if s is None:
            continue
        for t, p in zip(tokens, pos):
            if p >= 0 and 0 <= int(table[s, p // pt]) < pool.shape[0]:
                pool[int(table[s, p // pt]), 0, :, p % pt] = k[t]
                pool[int(table[s, p // pt]), 1, :, p % pt] = v[t]
    return pool


def attention(q, pool, table, lengths, seqs, offsets, scale, window):
    """q [tokens, Hq, D].  Returns out, the same sums with |v| (what the roundings of the weights act on), and lse."""
    pt, Hkv, Hq = pool.shape[3], pool.shape[2], q.shape[1]
    q = d(q)
    out, size = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64)
    group = torch.arange(Hq) // (Hq // Hkv)
    table, pool = table.cpu(), pool.cpu()
    for tokens, s, pos, length in rows_of(offsets, lengths, seqs):
        if s is None or not length or not len(pos):
            continue
        at = torch.arange(length)
        pages = table[s].long()[at // pt]
        k, v = d(pool[pages, 0, :, at % pt])[:, group], d(pool[pages, 1, :, at % pt])[:, group]      # [length, Hq, D]
        here = torch.tensor(pos)
        z = torch.einsum("thd,khd->thk", q[tokens.start:tokens.stop], k) * scale
        seen = at[None] <= here[:, None]
        if window:
            seen &= at[None] > here[:, None] - window
        z = z.masked_fill(~seen[:, None], -math.inf)
        any_ = seen.any(1)
        if not bool(any_.any()):
            continue
        idx = torch.arange(tokens.start, tokens.stop)[any_]
        w = torch.softmax(z[any_], -1)
        v = torch.where(torch.isfinite(v), v, torch.zeros_like(v)) if not bool(torch.isfinite(v).all()) else v
        out[idx] = torch.einsum("thk,khd->thd", w, v)
        size[idx] = torch.einsum("thk,khd->thd", w, v.abs())
        lse[idx] = torch.logsumexp(z[any_], -1)
    return out, size, lse
