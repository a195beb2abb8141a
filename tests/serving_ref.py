"""Plain 64-bit forms of the serving operators (prompt linear attention, single-token decode, draft
verification), token by token from their definitions, for the tests."""
import math

import numpy as np
import torch


def prompt(q, k, v, log_decay, cu, S0=None, scale=1.0):
    """(O, S): O [T, h_v, d_v] (zero outside the sequences) and S [n, h_v, d_v, d_k], float64."""
    q, k, v, g = (x.double().cpu() for x in (q, k, v, log_decay))
    cu = [int(c) for c in cu]
    n, h_v, d_k, d_v = len(cu) - 1, v.shape[1], k.shape[2], v.shape[2]
    group = h_v // k.shape[1]
    q, k = q.repeat_interleave(group, 1), k.repeat_interleave(group, 1)
    lam = torch.exp(g)[:, None, None]
    O = torch.zeros_like(v)
    S = torch.zeros((n, h_v, d_v, d_k), dtype=torch.float64)
    for i in range(n):
        s = S[i] if S0 is None else S0[i].double().cpu().clone()
        for t in range(cu[i], cu[i + 1]):
            s = lam * s + v[t].unsqueeze(-1) * k[t].unsqueeze(-2)
            O[t] = torch.einsum("hvk,hk->hv", s, scale * q[t])
        S[i] = s
    return O, S


def decode(q, k, v, g, beta, pool, slots, counts, window, *, l2norm=True, scale=1.0, family="delta"):
    """(rows, pool): {row of O: value} of every token that counts, and the pool afterwards, float64."""
    k, v, g, pool = (x.double().cpu() for x in (k, v, g, pool))
    pool = pool.clone()
    q = torch.zeros_like(k) if q is None else q.double().cpu()
    beta = None if beta is None else beta.double().cpu()
    group = v.shape[1] // k.shape[1]
    if l2norm:
        q, k = (x / torch.sqrt((x * x).sum(-1, keepdim=True) + 1e-6) for x in (q, k))
    q, k = q.repeat_interleave(group, 1), k.repeat_interleave(group, 1)
    rows = {}
    for i, slot in enumerate(slots):
        if slot < 0:
            continue
        s = pool[slot]
        for t in range(i * window, i * window + counts[i]):
            alpha = torch.exp(g if family == "head" else g[t])[:, None, None]
            b = 1.0 if family == "head" else beta[t][:, None, None]
            s = alpha * s
            vt, kt = v[t].unsqueeze(-1), k[t].unsqueeze(-2)
            if family == "delta":
                vt = vt - (s * kt).sum(-1, keepdim=True)
            s = s + b * vt * kt
            rows[t] = torch.einsum("hvk,hk->hv", s, scale * q[t])
        pool[slot] = s
    return rows, pool


def _whole(p):
    p = p.double().cpu().numpy()
    return np.floor(np.clip(np.where(np.isnan(p), 0.0, p), 0.0, 1.0) * 2.0 ** 44).astype(np.int64)


def verify(target, drafted, uniforms, draft, lens):
    """(counts, tokens) as lists; a request with a negative length has count 0 and no tokens."""
    n, w = drafted.shape
    vocab = target.shape[2]
    counts, tokens = [], []
    for i in range(n):
        if lens[i] < 0:
            counts.append(0)
            tokens.append([])
            continue
        row = []
        for j in range(lens[i]):
            x = int(drafted[i, j])
            if not 0 <= x < vocab:
                break
            q = 1.0 if draft is None else float(draft[i, j, x])
            if not float(uniforms[i, j]) * q < float(target[i, j, x]):
                break
            row.append(x)
        a = len(row)
        weight = _whole(target[i, a])
        if a < lens[i]:
            less = weight.copy()
            if draft is not None:
                less = np.maximum(weight - _whole(draft[i, a]), 0)
            elif 0 <= int(drafted[i, a]) < vocab:
                less[int(drafted[i, a])] = 0
            if less.any():
                weight = less
        total = int(weight.sum())
        if total:
            u = float(uniforms[i, w])
            place = min(max(int(math.floor(u * float(total))) if u == u else 0, 0), total - 1)
            row.append(int(np.searchsorted(np.cumsum(weight), place, side="right")))
        else:
            row.append(-1)
        counts.append(a + 1)
        tokens.append(row + [-1] * (w + 1 - len(row)))
    return counts, tokens
