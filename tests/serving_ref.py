"""Plain 64-bit references of the serving operators on the CPU: the recurrences token by token, the cache's
bookkeeping one request at a time."""
from __future__ import annotations

import numpy as np
import torch


def d(t):
    return t.detach().cpu().double()


def softplus(z):
    return torch.logaddexp(z, torch.zeros_like(z))


def ssm(x, dt_raw, b, c, a_log, dt_bias, d_skip, offsets, state):
    """x [TT, H, P], b, c [TT, G, N], dt_raw [TT, H]; rows [offsets[n], offsets[n + 1]) from state [rows, H, N, P]
    (None: zero).  Returns y [TT, H, P] and the end states."""
    x, dt_raw, b, c = d(x), d(dt_raw), d(b), d(c)
    H, P = x.shape[1:]
    G, N = b.shape[1:]
    rows = len(offsets) - 1
    S = torch.zeros(rows, H, N, P, dtype=torch.float64) if state is None else d(state).clone()
    delta = softplus(dt_raw + d(dt_bias))
    alpha = torch.exp(-torch.exp(d(a_log)) * delta)
    group = torch.arange(H) // (H // G)
    y = torch.zeros_like(x)
    for n in range(rows):
        for t in range(offsets[n], offsets[n + 1]):
            S[n] = alpha[t][:, None, None] * S[n] + (delta[t][:, None] * b[t][group])[:, :, None] * x[t][:, None, :]
            y[t] = (c[t][group][:, :, None] * S[n]).sum(1)
    if d_skip is not None:
        y += d(d_skip)[:, None] * x
    return y, S


def delta_step(q, k, v, g_raw, beta_raw, a_log, dt_bias, scale, lower_bound, gate, S):
    """One token of one row: q, k [Hk, K], v [H, V], g_raw [H, K], beta_raw [H], S [H, K, V]."""
    q, k, v, S = d(q), d(k), d(v), d(S)
    H, K = g_raw.shape
    head = torch.arange(H) // (H // q.shape[0])
    q = (q / torch.sqrt((q * q).sum(-1, keepdim=True) + 1e-6))[head]
    k = (k / torch.sqrt((k * k).sum(-1, keepdim=True) + 1e-6))[head]
    z, ea = d(g_raw) + d(dt_bias).view(H, K), torch.exp(d(a_log))[:, None]
    g = -ea * softplus(z) if gate == "softplus" else lower_bound * torch.sigmoid(ea * z)
    beta = torch.sigmoid(d(beta_raw))[:, None]
    S = torch.exp(g)[..., None] * S
    u = beta * (v - (k[..., None] * S).sum(1))
    S = S + k[..., None] * u[:, None, :]
    return scale * (q[..., None] * S).sum(1), S


def conv(x, weight, bias, offsets, history):
    """x [TT, C], history [rows, W - 1, C] or None.  Returns y and the last W - 1 inputs of each row."""
    x, w = d(x), d(weight)
    C, W = w.shape
    y, last = torch.zeros_like(x), []
    for n in range(len(offsets) - 1):
        old = torch.zeros(W - 1, C, dtype=torch.float64) if history is None else d(history[n])
        seq = torch.cat([old, x[offsets[n]:offsets[n + 1]]])
        for t in range(offsets[n + 1] - offsets[n]):
            a = (seq[t:t + W] * w.t()).sum(0) + (0 if bias is None else d(bias))
            y[offsets[n] + t] = a * torch.sigmoid(a)
        last.append(seq[len(seq) - (W - 1):])
    return y, torch.stack(last)


class Cache:
    """The cache's rows, references and pages as numpy arrays."""

    def __init__(self, pool, table, lengths, refs, page_tokens):
        self.pool, self.table, self.lengths, self.refs = (t.cpu().numpy().copy() for t in (pool, table, lengths, refs))
        self.pt = page_tokens

    def held(self, n):
        return -(-int(n) // self.pt)

    def free_pages(self):
        return [p for p in range(len(self.refs)) if self.refs[p] <= 0]

    def fork(self, parents, children):
        free, ok = self.free_pages(), []
        S, M = self.table.shape
        lengths = self.lengths.copy()
        used = 0
        for p, c in zip(parents, children):
            good = 0 <= p < S and 0 <= c < S and p != c and lengths[c] <= 0 and self.held(lengths[p]) <= M
            part = good and lengths[p] % self.pt != 0
            if part and not 0 <= self.table[p, lengths[p] // self.pt] < len(self.refs):
                good = part = False
            if part:
                used += 1
                good = used <= len(free)
            ok.append(int(good))
            if not good:
                continue
            full = lengths[p] // self.pt
            row = np.full(M, -1, np.int32)
            row[:full] = self.table[p, :full]
            for page in row[:full]:
                if 0 <= page < len(self.refs):
                    self.refs[page] += 1
            if part:
                new = free[used - 1]
                row[full] = new
                self.refs[new] = 1
                self.pool[:, new] = self.pool[:, self.table[p, full]]
            self.table[c], self.lengths[c] = row, lengths[p]
        return ok

    def extend(self, seqs, new_lengths):
        free, ok = self.free_pages(), []
        S, M = self.table.shape
        used = 0
        for s, n in zip(seqs, new_lengths):
            good = 0 <= s < S and n >= 0 and n >= self.lengths[s] and self.held(n) <= M
            if good:
                had = self.held(self.lengths[s])
                need = self.held(n) - had
                first, used = used, used + need
                good = need == 0 or used <= len(free)
                if good:
                    for j in range(need):
                        self.table[s, had + j] = free[first + j]
                        self.refs[free[first + j]] = 1
                    self.lengths[s] = n
            ok.append(int(good))
        return ok

    def free(self, seqs):
        for s in seqs:
            if 0 <= s < len(self.table):
                for page in self.table[s]:
                    if 0 <= page < len(self.refs):
                        self.refs[page] -= 1
                self.table[s], self.lengths[s] = -1, 0

    def compact(self):
        live = [p for p in range(len(self.refs)) if self.refs[p] > 0]
        L = len(live)
        to = np.full(len(self.refs), -1, np.int32)
        to[live] = live
        holes = [p for p in range(L) if self.refs[p] <= 0]
        for src, dst in zip(sorted((p for p in live if p >= L), reverse=True), holes):
            to[src] = dst
            self.pool[:, dst] = self.pool[:, src]
            self.refs[dst], self.refs[src] = self.refs[src], 0
        self.refs[L:] = 0
        for s in range(self.table.shape[0]):
            for j in range(self.table.shape[1]):
                if 0 <= self.table[s, j] < len(self.refs):
                    self.table[s, j] = to[self.table[s, j]]
        return to
