"""Plain 64-bit forms of the paged-cache and beam operators, token by token from their definitions, for the
tests, and inputs for them."""
import math

import torch


def ranges(n, T, cu):
    w = T // n if n else 0
    return [(i * w, (i + 1) * w) for i in range(n)] if cu is None else [(int(cu[i]), int(cu[i + 1])) for i in range(n)]


def attend(q, k_pages, v_pages, table, kv_lens, cu=None, *, scale=None, window=0):
    """{token: (O [h_q, d], lse [h_q])} of every token of a request that is no padding, float64."""
    q, k_pages, v_pages = (x.detach().cpu().double() for x in (q, k_pages, v_pages))
    table, kv_lens = table.cpu(), kv_lens.cpu().tolist()
    T, h_q, d = q.shape
    page, h_kv = k_pages.shape[1], k_pages.shape[2]
    group = h_q // h_kv
    scale = d ** -0.5 if scale is None else scale
    out = {}
    for i, (a, b) in enumerate(ranges(len(kv_lens), T, cu)):
        kv = kv_lens[i]
        if kv < 0 or b == a:
            continue
        ids = table[i, :-(-kv // page)].long()
        K = k_pages[ids].reshape(-1, h_kv, d)[:kv].repeat_interleave(group, 1)
        V = v_pages[ids].reshape(-1, h_kv, d)[:kv].repeat_interleave(group, 1)
        for t in range(a, b):
            p = kv - (b - a) + (t - a)
            lo, hi = max(0, p - window + 1) if window else 0, p + 1
            if hi <= 0:
                out[t] = torch.zeros(h_q, d, dtype=torch.float64), torch.full((h_q,), -math.inf, dtype=torch.float64)
                continue
            z = torch.einsum("hd,jhd->hj", q[t], K[lo:hi]) * scale
            lse = torch.logsumexp(z, -1)
            out[t] = torch.einsum("hj,jhd->hd", torch.softmax(z, -1), V[lo:hi]), lse
    return out


def turn(x, angle, neighbours):
    """x [..., d] with its first 2 * len(angle) values turned, float64."""
    n = len(angle)
    lo, hi = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if neighbours else (slice(0, n), slice(n, 2 * n))
    y = x.clone()
    a, b, c, s = x[..., lo], x[..., hi], torch.cos(angle), torch.sin(angle)
    y[..., lo], y[..., hi] = a * c - b * s, b * c + a * s
    return y


def append(k, v, k_pages, v_pages, table, kv_lens, cu=None, *, q=None, inv_freq=None, positions=None, sections=None,
           neighbours=False):
    """(q, k_pages, v_pages) afterwards, float64; rows of q of padding are zero."""
    k, v, k_pages, v_pages = (x.detach().cpu().double() for x in (k, v, k_pages, v_pages))
    k_pages, v_pages = k_pages.clone(), v_pages.clone()
    q_out = None if q is None else torch.zeros_like(q.cpu(), dtype=torch.float64)
    T, page = k.shape[0], k_pages.shape[1]
    freq = torch.zeros(0, dtype=torch.float64) if inv_freq is None else inv_freq.cpu().double()
    axis = torch.zeros(len(freq), dtype=torch.long)
    if positions is not None:
        positions = positions.cpu().reshape(-1, T)
        if len(positions) > 1:
            axis = torch.repeat_interleave(torch.arange(len(positions)), torch.tensor(sections))
    for i, (a, b) in enumerate(ranges(len(kv_lens), T, cu)):
        kv = int(kv_lens[i])
        if kv < 0:
            continue
        for t in range(a, b):
            p = kv - (b - a) + (t - a)
            where = torch.full((len(freq),), float(p), dtype=torch.float64) if positions is None else positions[axis, t].double()
            angle = where * freq
            if q is not None:
                q_out[t] = turn(q[t].detach().cpu().double(), angle, neighbours)
            if p >= 0:
                at = int(table[i, p // page])
                k_pages[at, p % page] = turn(k[t], angle, neighbours)
                v_pages[at, p % page] = v[t]
    return q_out, k_pages, v_pages


def cache(gen, lens, page, h_kv, d, dt, spare=2, width=None, layout="tokens"):
    """(k_pages, v_pages, table) for requests of ``lens`` tokens: random page order, entries behind a request's pages far
    outside the cache.  layout: "tokens" (page, token, head), "heads" (page, head, token), "joined" (one array
    [page, 2, token, head])."""
    used = [max(0, -(-n // page)) for n in lens]
    pages = sum(used) + spare
    order = torch.randperm(pages, generator=gen)
    width = max(1, max(used, default=0)) if width is None else width
    table = torch.full((len(lens), width), 1 << 30, dtype=torch.int32)
    at = 0
    for i, n in enumerate(used):
        table[i, :n] = order[at:at + n]
        at += n
    if layout == "joined":
        both = torch.randn(pages, 2, page, h_kv, d, generator=gen).to(dt)
        return both[:, 0], both[:, 1], table
    if layout == "heads":
        k, v = (torch.randn(pages, h_kv, page, d, generator=gen).to(dt).permute(0, 2, 1, 3) for _ in range(2))
        return k, v, table
    k, v = (torch.randn(pages, page, h_kv, d, generator=gen).to(dt) for _ in range(2))
    return k, v, table


def on_gpu(t):
    """A copy on the GPU with the same strides (``.cuda()`` keeps those of dense tensors alone)."""
    base = t if t._base is None else t._base
    return base.cuda().as_strided(t.shape, t.stride(), t.storage_offset())
