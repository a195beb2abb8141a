"""Cases, plain forms and 64-bit values of the operators for attention layers and beams.

A model with recurrent-state layers has layers of attention over a paged key-value cache between them,
and a server that decodes with beams moves both kinds of memory with the beams.  Four operators:

* ``append``: new keys and values into the paged cache, the position rotation applied on the way (to
  the queries too), one position per token or several axes of them,
* ``attend``: the new tokens' attention over the paged cache: one token, a window of drafts, or a chunk,
* ``select``: the best continuations over beams and vocabulary,
* ``reorder``: the pool's states follow the beams that were selected.

``run`` computes them in elementary torch operations where ``own`` is false, and calls the library
where it is true.
"""
import math
import random

import numpy as np
import torch

own = False

MOST_APPEND = 8192 * 48 * 128  # values of the queries, keys and values of the largest append case
MOST_KEYS = 128 * 16384 * 8 * 128  # padded values of the cache that an attend case reads
MOST_SCORES = 2048 * 32768 * 32  # padded scores of an attend case
MOST_LOGITS = 64 * 8 * 131072
MOST_MOVED = 64 * 8 * 32 * 128 * 128  # values of the states that belong to a reorder case's beams


def listed():
    heads = {"h_q": 32, "h_kv": 8, "d": 128}
    return [
        # one user's next token, far into a long context: the smallest append of a serving loop
        {"name": "append one token", "op": "append", "type": "bf16", "n": 1, "tokens": 1, "context": 32000, **heads,
         "page": 16, "rotary": 128, "axes": 1, "pairs": "halves", "cut": 1},
        # a step's chunk of several prompts, text and images: three position axes
        {"name": "append 8192 tokens", "op": "append", "type": "bf16", "n": 6, "tokens": 8192, "context": 20000, **heads,
         "page": 64, "rotary": 128, "axes": 3, "pairs": "halves", "cut": 2},
        # one user's next token over its context: latency counts
        {"name": "attend one token", "op": "attend", "type": "bf16", "n": 1, "queries": "token", "tokens": 1,
         "context": 8191, **heads, "page": 16, "window": 0, "padded": 0, "cut": 3},
        # a full batch's next tokens over ragged contexts, a few rows of it padding as a captured graph has them
        {"name": "attend batch 128", "op": "attend", "type": "bf16", "n": 128, "queries": "token", "tokens": 128,
         "context": 16383, **heads, "page": 64, "window": 0, "padded": 5, "cut": 4},
        # windows of drafted tokens, four query heads to a key head
        {"name": "attend windows 64x5", "op": "attend", "type": "bf16", "n": 64, "queries": "window", "tokens": 320,
         "context": 6000, **heads, "page": 32, "window": 0, "padded": 0, "cut": 5},
        # the last chunk of a long prompt
        {"name": "attend chunk 2048 of 32k", "op": "attend", "type": "bf16", "n": 1, "queries": "chunk", "tokens": 2048,
         "context": 30720, **heads, "page": 64, "window": 0, "padded": 0, "cut": 6},
        # a step's chunks of many requests at once: ragged, a sliding window, odd head counts and sizes
        {"name": "attend ragged chunks", "op": "attend", "type": "bf16", "n": 12, "queries": "chunk", "tokens": 6007,
         "context": 5000, "h_q": 24, "h_kv": 4, "d": 96, "page": 16, "window": 1777, "padded": 0, "cut": 7},
        # fp32 layers: short ragged chunks, small heads
        {"name": "attend ragged f32", "op": "attend", "type": "f32", "n": 6, "queries": "chunk", "tokens": 701,
         "context": 2500, "h_q": 8, "h_kv": 4, "d": 80, "page": 32, "window": 0, "padded": 0, "cut": 8},
        # one user's beams
        {"name": "select one 4 beams", "op": "select", "type": "f32", "n": 1, "beams": 4, "best": 4, "vocab": 32000, "cut": 9},
        # a batch's beams over a large vocabulary, twice as many continuations as beams (some may end)
        {"name": "select 64x8 beams", "op": "select", "type": "f32", "n": 64, "beams": 8, "best": 16, "vocab": 131072,
         "cut": 10},
        # one user's beams follow their parents in one layer's pool
        {"name": "reorder one 4 beams", "op": "reorder", "type": "f32", "n": 1, "beams": 4, "h": 32, "d_k": 128, "d_v": 128,
         "spare": 4, "layers": 1, "cut": 11},
        # a batch's beams
        {"name": "reorder 64x8 beams", "op": "reorder", "type": "f32", "n": 64, "beams": 8, "h": 32, "d_k": 128, "d_v": 128,
         "spare": 16, "layers": 1, "cut": 12},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append", "attend", "attend", "attend", "attend", "attend", "select", "select", "reorder"])
    cut = rng.randrange(1, 1 << 20)
    if op == "select":
        n, beams = _spread(rng, 1, 64), rng.choice([1, 2, 3, 4, 4, 5, 8])
        vocab = _spread(rng, 100, 131072)
        best = rng.choice([beams, beams, 2 * beams, rng.randint(1, 32)])
        return {"op": op, "type": rng.choice(["f32", "f32", "bf16"]), "n": n, "beams": beams, "best": best, "vocab": vocab,
                "cut": cut}
    if op == "reorder":
        h, (d_k, d_v) = rng.choice([1, 4, 16, 32]), rng.choice([(128, 128), (64, 64), (128, 64), (96, 120)])
        layers, beams = rng.choice([1, 1, 2, 4]), rng.randint(1, 8)
        n = max(1, min(_spread(rng, 1, 64), MOST_MOVED // (layers * beams * h * d_k * d_v)))
        return {"op": op, "type": rng.choice(["f32", "f32", "bf16"]), "n": n, "beams": beams, "h": h, "d_k": d_k, "d_v": d_v,
                "spare": rng.randint(0, 16), "layers": layers, "cut": cut}
    h_kv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 4, 6, 8])
    if h_kv * group > 32:
        group = 4
    d = rng.choice([128, 128, 128, 64, 96, 80, 8 * rng.randint(2, 16)])
    shape = {"h_q": h_kv * group, "h_kv": h_kv, "d": d, "page": rng.choice([16, 16, 32, 64, 128])}
    kind = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "append":
        n = _spread(rng, 1, 64)
        tokens = rng.choice([n, _spread(rng, n, 8192)])
        tokens = max(n, min(tokens, MOST_APPEND // ((h_kv * group + 2 * h_kv) * d)))
        axes = rng.choice([1, 1, 2, 3])
        rotary = rng.choice([d, d, 2 * max(axes, d // 4)])
        return {"op": op, "type": kind, "n": n, "tokens": tokens, "context": _spread(rng, 1, 131072), **shape,
                "rotary": rotary, "axes": axes, "pairs": rng.choice(["halves", "halves", "neighbours"]), "cut": cut}
    queries = rng.choice(["token", "token", "window", "chunk", "chunk"])
    n = _spread(rng, 1, 16 if queries == "chunk" else 128)
    context = _spread(rng, 1, 32768 if n <= 4 else 16384)
    tokens = n if queries == "token" else n * rng.randint(2, 8) if queries == "window" else _spread(rng, n, 4096)
    if kind == "f32" and queries == "chunk":  # (the CUDA cores' share of the range)
        tokens, context = max(n, min(tokens, 1024)), min(context, 4096)
    most = lambda t: 2 * t // n + 16 if n > 1 else t  # noqa: E731  (of the longest request's new tokens)
    context = max(1, min(context, MOST_KEYS // (n * h_kv * d) - most(tokens)))
    while tokens > n and n * most(tokens) * (context + most(tokens)) * h_kv * group > MOST_SCORES:
        tokens = n * max(1, tokens // (2 * n)) if queries == "window" else max(n, tokens // 2)
    return {"op": op, "type": kind, "n": n, "queries": queries, "tokens": tokens, "context": context, **shape,
            "window": rng.choice([0, 0, 0, _spread(rng, 1, 8192)]),
            "padded": rng.randint(0, n // 8) if queries == "token" else 0, "cut": cut}


def _dtype(case):
    return torch.bfloat16 if case["type"] == "bf16" else torch.float32


def _lengths(case):
    """(new tokens, tokens in the cache with them) of each request: ragged; padding has -1 in the cache."""
    n, tokens, context = case["n"], case["tokens"], case["context"]
    rng = random.Random(case["cut"])
    if n == 1:
        return [tokens], [context + tokens]
    if tokens % n == 0 and case.get("queries") != "chunk":
        new = [tokens // n] * n
    else:  # the longest at most twice the mean, so that what is padded stays within the range
        share = [rng.uniform(0.15, 1.0) for _ in range(n)]
        total = sum(share)
        new = [min(int(tokens * s / total), 2 * tokens // n) for s in share]
        i = 0
        while sum(new) < tokens:
            new[i % n] += min(tokens - sum(new), max(1, tokens // n // 4))
            i += 1
        if case["op"] == "append" and n > 4:
            new[1], new[2] = new[1] + new[2], 0  # a request of no new tokens
    kv = [a + max(0, int(context * (1.0 if i == 0 else rng.uniform(0.02, 1.0)))) for i, a in enumerate(new)]
    for i in range(n - case.get("padded", 0), n):
        kv[i] = -1
    return new, kv


def _sections(case):
    """Rotated pairs of each position axis."""
    pairs, axes = case["rotary"] // 2, case["axes"]
    first = pairs // 4 if axes > 1 else pairs
    rest = pairs - first
    return [pairs] if axes == 1 else [first, rest] if axes == 2 else [first, rest // 2, rest - rest // 2]


def _parents(case):
    """Each beam's parent: the best beams have several children, the last ones often none."""
    rng = random.Random(case["cut"])
    b = case["beams"]
    weight = [0.75 ** j for j in range(b)]
    return [rng.choices(range(b), weight, k=b) for _ in range(case["n"])]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed * 1000003 + case["cut"])
    dt, n = _dtype(case), case["n"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device=dev)

    if case["op"] == "select":
        b, V = case["beams"], case["vocab"]
        # peaked rows, as a model's logits over a vocabulary are; beams of one request near each other
        return {"case": case, "logits": (3.0 * normal(n, b, V)).to(dt),
                "scores": (-20.0 - 4.0 * torch.rand((n, b), generator=gen, device=dev)).sort(-1, descending=True)[0]}
    if case["op"] == "reorder":
        slots = n * case["beams"] + case["spare"]
        pool = normal(*([case["layers"]] if case["layers"] > 1 else []), slots, case["h"], case["d_v"], case["d_k"]).to(dt)
        place = torch.randperm(slots, generator=gen, device=dev)[:n * case["beams"]]
        return {"case": case, "pool": pool, "slots": place.reshape(n, -1).to(torch.int32), "parents": ints(_parents(case))}
    h_q, h_kv, d, page = case["h_q"], case["h_kv"], case["d"], case["page"]
    new, kv = _lengths(case)
    T, width = sum(new), max(1, -(-max(kv) // page))
    # one row of queries, keys and values per token, as the projection in front of the layer leaves them
    rows = normal(T, (h_q + 2 * h_kv) * d).to(dt)
    q = rows[:, :h_q * d].view(T, h_q, d)
    cu = ints(np.concatenate([[0], np.cumsum(new)]).tolist())
    s = {"case": case, "q": q, "cu": cu, "kv_lens": ints(kv), "new": new, "kv": kv}
    table = np.full((n, width), -1, np.int32)
    if case["op"] == "append":
        s["k"] = rows[:, h_q * d:(h_q + h_kv) * d].view(T, h_kv, d)
        s["v"] = rows[:, (h_q + h_kv) * d:].view(T, h_kv, d)
        first = [(b - a) // page for a, b in zip(new, kv)]
        used = [-(-b // page) - f for b, f in zip(kv, first)]
        pages = sum(used) + 3
        order = torch.randperm(pages, generator=gen, device=dev).cpu().numpy()
        at = 0
        for i in range(n):  # (the pages before the written ones are not looked at: any of them will do)
            table[i, :first[i]] = order[-1]
            table[i, first[i]:first[i] + used[i]] = order[at:at + used[i]]
            at += used[i]
        pairs = case["rotary"] // 2
        s["inv_freq"] = (1e6 ** (-torch.arange(pairs, device=dev, dtype=torch.float64) / pairs)).float()
        s["positions"] = None
        if case["axes"] > 1:  # text has one position on every axis, an image's rows and columns run on the others
            pos = np.concatenate([np.arange(b - a, b) for a, b in zip(new, kv)])
            s["positions"] = ints(np.stack([pos, pos // 32 + pos % 7, pos // 32 + pos % 32][:case["axes"]]).tolist())
    else:
        used = [max(0, -(-b // page)) for b in kv]
        pages = sum(used) + 3
        order = torch.randperm(pages, generator=gen, device=dev).cpu().numpy()
        at = 0
        for i in range(n):
            table[i, :used[i]] = order[at:at + used[i]]
            at += used[i]
        s["q"] = (1.5 * q.float()).to(dt)  # (contiguous, as the rotation leaves them)
        s["O"] = torch.zeros((T, h_q, d), dtype=dt, device=dev)
        s["lse"] = torch.zeros((T, h_q), device=dev)
    s["table"] = torch.from_numpy(table).to(dev)
    s["k_pages"], s["v_pages"] = normal(pages, page, h_kv, d).to(dt), normal(pages, page, h_kv, d).to(dt)
    return s


# ------------------------------------------------------------------ append


def _cache_positions(s):
    """(request, position in the cache) of each token."""
    cu, kv = s["cu"].long(), s["kv_lens"].long()
    t = torch.arange(s["q"].shape[0], device=cu.device)
    i = torch.bucketize(t, cu[1:], right=True)
    return i, t - cu[i + 1] + kv[i]


def _plain_append(s):
    case = s["case"]
    i, pos = _cache_positions(s)
    page, half = case["page"], case["rotary"] // 2
    where = s["positions"] if s["positions"] is not None else pos[None]
    axis = torch.repeat_interleave(torch.arange(case["axes"], device=pos.device), torch.tensor(_sections(case), device=pos.device))
    angle = where.double()[axis].t() * s["inv_freq"].double()  # [T, pairs]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def rotated(x):
        y = x.float()
        r = y[..., :2 * half]
        if case["pairs"] == "halves":
            a, b = r[..., :half], r[..., half:]
            r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        else:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        return torch.cat([r, y[..., 2 * half:]], -1).to(x.dtype)

    at = s["table"][i, pos // page].long()
    s["k_pages"][at, pos % page] = rotated(s["k"])
    s["v_pages"][at, pos % page] = s["v"]
    return {"q": rotated(s["q"]), "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _own_append(s, api):
    case = s["case"]
    q = api.gdn_kv_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["kv_lens"], s["cu"], q=s["q"],
                          inv_freq=s["inv_freq"], positions=s["positions"],
                          sections=_sections(case) if case["axes"] > 1 else None, neighbours=case["pairs"] == "neighbours")
    return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _exact_append(case, seed):
    """Token by token: each pair turned as a complex number of 64-bit parts."""
    s = prepare(case, seed)
    page, pairs = case["page"], case["rotary"] // 2
    freq = s["inv_freq"].double().cpu().numpy()
    axis = np.repeat(np.arange(case["axes"]), _sections(case))
    given = None if s["positions"] is None else s["positions"].cpu().numpy().astype(np.float64)
    table = s["table"].cpu().numpy()
    lo, hi = (slice(0, pairs), slice(pairs, 2 * pairs)) if case["pairs"] == "halves" else \
        (slice(0, 2 * pairs, 2), slice(1, 2 * pairs, 2))
    q, k, v = (s[x].double() for x in "qkv")
    k_pages, v_pages = s["k_pages"].double(), s["v_pages"].double()
    turn, at_page, at_slot, t = [], [], [], 0
    for i, (a, b) in enumerate(zip(s["new"], s["kv"])):
        for p in range(b - a, b):
            angle = (given[axis, t] if given is not None else p) * freq
            turn.append(np.cos(angle) + 1j * np.sin(angle))
            at_page.append(table[i, p // page])
            at_slot.append(p % page)
            t += 1
    turn = torch.from_numpy(np.stack(turn)).to(q.device)[:, None]
    for x in (q, k):
        z = torch.complex(x[..., lo].contiguous(), x[..., hi].contiguous()) * turn
        x[..., lo], x[..., hi] = z.real, z.imag
    at_page, at_slot = (torch.tensor(np.array(x), dtype=torch.long, device=q.device) for x in (at_page, at_slot))
    k_pages[at_page, at_slot], v_pages[at_page, at_slot] = k, v
    return {"q": q, "k_pages": k_pages, "v_pages": v_pages}


# ------------------------------------------------------------------ attend


def _plain_attend(s):
    case = s["case"]
    n, h_kv, d, page = case["n"], case["h_kv"], case["d"], case["page"]
    group, cu, kv = case["h_q"] // h_kv, s["cu"].long(), s["kv_lens"].long()
    dev, most, far = cu.device, max(s["new"]), max(s["kv"])
    at = torch.arange(most, device=dev)
    length = cu[1:] - cu[:-1]
    there = (at[None] < length[:, None]) & (kv[:, None] >= 0)  # [n, most]
    rows = torch.where(there, cu[:-1, None] + at[None], 0)
    q = s["q"][rows].float().reshape(n, most, h_kv, group, d).permute(0, 2, 1, 3, 4).reshape(n, h_kv, most * group, d)
    table = s["table"][:, :-(-far // page)].clamp(min=0).long()

    def laid(pages):  # [n, h_kv, far, d]
        return pages[table].reshape(n, -1, h_kv, d)[:, :far].permute(0, 2, 1, 3).float()

    j = torch.arange(far, device=dev)
    pos = kv[:, None] - length[:, None] + at[None]  # [n, most]
    seen = j[None, None] <= pos[..., None]
    if case["window"]:
        seen = seen & (j[None, None] > pos[..., None] - case["window"])
    score = torch.matmul(q, laid(s["k_pages"]).transpose(-1, -2)) * d ** -0.5
    score = score.reshape(n, h_kv, most, group, far).masked_fill_(~seen[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    weight = score.sub_(top).exp_()
    total = weight.sum(-1)
    value = torch.matmul(weight.reshape(n, h_kv, most * group, far), laid(s["v_pages"])).reshape(n, h_kv, most, group, d)
    value = torch.where(total[..., None] > 0, value / total[..., None], 0.0)
    lse = torch.log(total) + top[..., 0]
    s["O"][rows[there]] = value.permute(0, 2, 1, 3, 4).reshape(n, most, -1, d)[there].to(s["O"].dtype)
    s["lse"][rows[there]] = lse.permute(0, 2, 1, 3).reshape(n, most, -1)[there]
    return {"O": s["O"], "lse": s["lse"]}


def _own_attend(s, api):
    case = s["case"]
    api.gdn_paged_attn(s["q"], s["k_pages"], s["v_pages"], s["table"], s["kv_lens"],
                       s["cu"] if case["queries"] == "chunk" else None, max_q=max(s["new"]), window=case["window"],
                       O_out=s["O"], lse_out=s["lse"])
    return {"O": s["O"], "lse": s["lse"]}


def _exact_attend(case, seed):
    """Request by request and head by head, from the softmax's definition in 64 bits."""
    s = prepare(case, seed)
    page, d, w = case["page"], case["d"], case["window"]
    group, t = case["h_q"] // case["h_kv"], 0
    if case["tokens"] * case["context"] * case["h_q"] * d > 1.2e12:
        return None
    O, lse = s["O"].double(), s["lse"].double()
    for i, (a, b) in enumerate(zip(s["new"], s["kv"])):
        t += a
        if b < 0 or a == 0:
            continue
        ids = s["table"][i, :-(-b // page)].long()
        pos = torch.arange(b - a, b, device=O.device)
        first = max(0, b - a - w + 1) if w else 0  # the first key that any of the new tokens sees
        j = torch.arange(first, b, device=O.device)
        hidden = j[None] > pos[:, None]
        if w:
            hidden |= pos[:, None] - j[None] >= w
        for h in range(case["h_kv"]):
            K, V = (x[ids, :, h].reshape(-1, d)[first:b].double() for x in (s["k_pages"], s["v_pages"]))
            for g in range(h * group, (h + 1) * group):
                z = (s["q"][t - a:t, g].double() @ K.t()) / math.sqrt(d)
                z.masked_fill_(hidden, -math.inf)
                lse[t - a:t, g] = torch.logsumexp(z, -1)
                O[t - a:t, g] = torch.exp_(z.sub_(lse[t - a:t, g, None])) @ V
    return {"O": O, "lse": lse}


# ------------------------------------------------------------------ select


def _plain_select(s):
    x, k = s["logits"].double(), s["case"]["best"]
    n, b, V = x.shape
    top = x.amax(-1)
    lse = top + torch.log(torch.exp(x - top[..., None]).sum(-1))
    total = (s["scores"].double() - lse)[..., None] + x
    value, index = torch.sort(total.reshape(n, b * V), dim=-1, descending=True, stable=True)
    value, index = value[:, :k], index[:, :k]
    return {"scores": value.float(), "parents": (index // V).to(torch.int32), "tokens": (index % V).to(torch.int32)}


def _own_select(s, api):
    scores, parents, tokens = api.gdn_beam_select(s["logits"], s["scores"], s["case"]["best"])
    return {"scores": scores, "parents": parents, "tokens": tokens}


def _exact_select(case, seed):
    """Beam by beam its best continuations, then the best of all beams' by (total, beam, token)."""
    s = prepare(case, seed)
    k, V = case["best"], case["vocab"]
    logits, scores = s["logits"].double(), s["scores"].double().cpu().numpy()
    lse = torch.logsumexp(logits, -1).cpu().numpy()
    # every entry that can be among a beam's first k: those not below its k-th largest value
    border = logits.topk(min(k, V), -1)[0][..., -1:]
    out = np.empty((case["n"], k)), np.empty((case["n"], k), np.int32), np.empty((case["n"], k), np.int32)
    for i in range(case["n"]):
        all_of = []
        for b, v in (logits[i] >= border[i]).nonzero().tolist():
            all_of.append((-((scores[i, b] - lse[i, b]) + float(logits[i, b, v])), b, v))
        for j, (total, b, v) in enumerate(sorted(all_of)[:k]):
            out[0][i, j], out[1][i, j], out[2][i, j] = -total, b, v
    return {"scores": out[0], "parents": out[1], "tokens": out[2]}


# ------------------------------------------------------------------ reorder


def _plain_reorder(s):
    slots, parents = s["slots"].long(), s["parents"].long()
    n, b = slots.shape
    beam = torch.arange(b, device=slots.device)
    same = parents[:, :, None] == parents[:, None, :]
    keeps = ~(same & (beam[None, None] < beam[None, :, None])).any(-1)  # no earlier beam has this parent
    childless = ~(parents[:, None, :] == beam[None, :, None]).any(-1)
    # the k-th beam that does not keep its parent's slot takes the slot of the k-th childless one
    order = torch.argsort(torch.where(childless, beam, b + beam), dim=-1)
    rank = (~keeps).long().cumsum(-1) - 1
    own_slot = slots.gather(1, parents)
    free = slots.gather(1, order.gather(1, rank.clamp(min=0)))
    out = torch.where(keeps, own_slot, free)
    rows = s["pool"] if s["case"]["layers"] > 1 else s["pool"][None]
    rows[:, out[~keeps]] = rows[:, own_slot[~keeps]]
    return {"slots": out.to(torch.int32), "pool": s["pool"]}


def _own_reorder(s, api):
    slots = api.gdn_beam_reorder(s["pool"], s["slots"], s["parents"], layers=s["case"]["layers"] > 1)
    return {"slots": slots, "pool": s["pool"]}


def _exact_reorder(case, seed):
    s = prepare(case, seed)
    out, source, target = [], [], []
    for slots, parents in zip(s["slots"].tolist(), s["parents"].tolist()):
        free = [x for j, x in enumerate(slots) if j not in parents]
        taken, row = set(), []
        for p in parents:
            if p in taken:
                source.append(slots[p])
                target.append(free.pop(0))
                row.append(target[-1])
            else:
                taken.add(p)
                row.append(slots[p])
        out.append(row)
    pool = s["pool"].double()
    rows = pool if case["layers"] > 1 else pool[None]
    for a, b in zip(source, target):
        rows[:, b] = rows[:, a]
    return {"slots": np.array(out, np.int32), "pool": pool}


# ------------------------------------------------------------------ what the tools call


def run(state):
    op = state["case"]["op"]
    if own:
        from gated_deltanet_state_chunked_gb300 import api
        return {"append": _own_append, "attend": _own_attend, "select": _own_select, "reorder": _own_reorder}[op](state, api)
    return {"append": _plain_append, "attend": _plain_attend, "select": _plain_select, "reorder": _plain_reorder}[op](state)


def exact(case, seed):
    return {"append": _exact_append, "attend": _exact_attend, "select": _exact_select,
            "reorder": _exact_reorder}[case["op"]](case, seed)


def work(case):
    size = 2 if case["type"] == "bf16" else 4
    n = case["n"]
    if case["op"] == "select":
        values = n * case["beams"] * case["vocab"]
        return {"bytes": values * size + n * (case["beams"] + 3 * case["best"]) * 4, "flops": 3.0 * values}
    if case["op"] == "reorder":
        copies = sum(case["beams"] - len(set(p)) for p in _parents(case))
        return {"bytes": 2.0 * copies * case["layers"] * case["h"] * case["d_k"] * case["d_v"] * size + n * case["beams"] * 12,
                "flops": 0.0}
    new, kv = _lengths(case)
    h_q, h_kv, d = case["h_q"], case["h_kv"], case["d"]
    if case["op"] == "append":
        T = sum(new)
        return {"bytes": 2.0 * T * (h_q + 2 * h_kv) * d * size + case["axes"] * T * 4, "flops": 3.0 * T * (h_q + h_kv) * case["rotary"]}
    w = case["window"]
    keys = pairs = tokens = 0
    for a, b in zip(new, kv):
        if b < 0 or a == 0:
            continue
        tokens += a
        keys += min(b, a + w - 1) if w else b
        # visible keys of positions b - a .. b - 1
        whole = max(0, min(a, w - (b - a))) if w else a  # of them, those that the window does not cut
        pairs += whole * (b - a) + whole * (whole + 1) // 2 + (a - whole) * w
    return {"bytes": 2.0 * keys * h_kv * d * size + tokens * h_q * (2 * d * size + 4), "flops": 4.0 * pairs * h_q * d}
