"""Cases, plain forms and 64-bit values of the serving operators beside the state rebuild.

Three operators, as a server of a model with recurrent-state layers calls them one after another:

* ``prompt``: linear attention with a decay for each head over packed prompts (the chunked form),
* ``token``: the recurrent form on a pool of states, for single tokens and for windows of drafted
  tokens (all outputs with the states kept, or the states advanced by each request's count),
* ``verify``: drafted tokens against the target's probabilities, from given random numbers.

``run`` computes them in elementary torch operations where ``own`` is false, and calls the library
where it is true.
"""
import math
import random

import numpy as np
import torch

own = False

FIX = 44  # probabilities are compared and summed as whole multiples of 2^-44
MOST_PROMPT = 99583 * 32  # tokens times v-heads of the largest prompt case
MOST_TOKEN = 256 * 32 * 128 * 128  # state values of the largest token case
MOST_VERIFY = 128 * 131072  # probabilities in one row of each request of the largest verify case
#: with the drafts that prepare() makes, about this share of the requests ends in a rejection
REJECTED = 0.8


def listed():
    layer = {"h_k": 16, "h_v": 32, "d_k": 128, "d_v": 128}
    return [
        # the repository's tiny configuration: one short prompt, few heads; latency counts
        {"name": "prompt tiny f32", "op": "prompt", "type": "f32", "n": 1, "tokens": 256, "h_k": 2, "h_v": 2,
         "d_k": 64, "d_v": 64, "enter": False, "state_only": False, "cut": 1},
        # one request's replay tail of a 32K prefix at the repository's layer shape
        {"name": "prompt tail 3277", "op": "prompt", "type": "bf16", "n": 1, "tokens": 3277, **layer,
         "enter": False, "state_only": False, "cut": 1},
        # many requests at once, each with the state that its cached prefix left: a loaded server
        {"name": "prompt 64 tails", "op": "prompt", "type": "bf16", "n": 64, "tokens": 99583, **layer,
         "enter": True, "state_only": False, "cut": 2},
        # a whole 32K prefix whose outputs nobody reads: the state for the prefix cache
        {"name": "prompt 32k state", "op": "prompt", "type": "bf16", "n": 1, "tokens": 32768, **layer,
         "enter": False, "state_only": True, "cut": 1},
        # fp32 inputs, ragged lengths (some of them tiny) and head sizes that are not powers of two
        {"name": "prompt ragged f32", "op": "prompt", "type": "f32", "n": 24, "tokens": 16411, "h_k": 8, "h_v": 16,
         "d_k": 96, "d_v": 120, "enter": True, "state_only": False, "cut": 3},
        # one user's next token: the smallest call of a serving loop
        {"name": "token one", "op": "token", "type": "bf16", "family": "delta", "mode": "step", "n": 1, "window": 1,
         **layer, "slots": 4, "padded": 0, "cut": 1},
        # a full batch's next tokens, a few rows of it padding as a captured graph has them
        {"name": "token batch 256", "op": "token", "type": "bf16", "family": "delta", "mode": "step", "n": 256,
         "window": 1, **layer, "slots": 272, "padded": 5, "cut": 2},
        # fp32 layers with one decay per head, value heads smaller than key heads
        {"name": "token head decay f32", "op": "token", "type": "f32", "family": "head", "mode": "step", "n": 48,
         "window": 1, "h_k": 16, "h_v": 16, "d_k": 128, "d_v": 80, "slots": 64, "padded": 0, "cut": 3},
        # drafted windows: every position's output, the states as they were
        {"name": "window outputs 64x5", "op": "token", "type": "bf16", "family": "delta", "mode": "outputs", "n": 64,
         "window": 5, **layer, "slots": 80, "padded": 0, "cut": 4},
        # the same windows after verification: each state advanced by what its request accepted
        {"name": "window commit 64x5", "op": "token", "type": "bf16", "family": "delta", "mode": "commit", "n": 64,
         "window": 5, **layer, "slots": 80, "padded": 3, "cut": 5},
        # one user's drafts
        {"name": "verify one", "op": "verify", "type": "f32", "n": 1, "window": 4, "vocab": 32000, "draft": True,
         "cut": 1},
        # a batch's drafts over a large vocabulary
        {"name": "verify batch 128", "op": "verify", "type": "f32", "n": 128, "window": 5, "vocab": 131072,
         "draft": True, "cut": 2},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "prompt", "token", "token", "token", "verify", "verify"])
    cut = rng.randrange(1, 1 << 20)
    if op == "verify":
        n = _spread(rng, 1, 128)
        vocab = _spread(rng, 100, 131072)
        return {"op": op, "type": rng.choice(["f32", "f32", "bf16"]), "n": n, "window": rng.randint(1, 8),
                "vocab": vocab, "draft": rng.random() < 0.7, "cut": cut}
    h_k = rng.choice([1, 2, 3, 4, 8, 16])
    h_v = h_k * rng.choice([1, 2, 2, 4] if h_k <= 8 else [1, 2])
    d_k, d_v = rng.choice([(128, 128), (128, 128), (64, 64), (128, 64), (96, 128), (72, 104), (8 * rng.randint(2, 16), 8 * rng.randint(2, 16))])
    kind = rng.choice(["bf16", "bf16", "f32"])
    shape = {"h_k": h_k, "h_v": h_v, "d_k": d_k, "d_v": d_v}
    if op == "prompt":
        n = _spread(rng, 1, 64)
        tokens = _spread(rng, n, 32768)
        return {"op": op, "type": kind, "n": n, "tokens": min(tokens, MOST_PROMPT // h_v), **shape,
                "enter": rng.random() < 0.5, "state_only": rng.random() < 0.25, "cut": cut}
    n = _spread(rng, 1, 256)
    mode = rng.choice(["step", "step", "outputs", "commit"])
    n = max(1, min(n, MOST_TOKEN // (h_v * d_k * d_v)))
    return {"op": op, "type": kind, "family": rng.choice(["delta", "delta", "scalar", "head"]), "mode": mode, "n": n,
            "window": 1 if mode == "step" else rng.randint(2, 8), **shape, "slots": n + rng.randint(0, 16),
            "padded": rng.randint(0, n // 8), "cut": cut}


def _lengths(case):
    """Lengths of the packed prompts: ragged, a few empty or tiny where there are many."""
    n, tokens = case["n"], case["tokens"]
    if n == 1:
        return [tokens]
    rng = random.Random(case["cut"])
    share = [rng.uniform(0.05, 1.0) for _ in range(n)]
    for i in range(3, n, 9):
        share[i] = rng.choice([0.0, 0.002])
    total = sum(share)
    lens = [int(tokens * s / total) for s in share]
    lens[0] += tokens - sum(lens)
    return lens


def _counts(case):
    """Tokens of each request's window that count."""
    n, w = case["n"], case["window"]
    if case["mode"] != "commit":
        return [w] * n
    rng = random.Random(case["cut"])
    return [rng.randint(1, w) for _ in range(n)]


def _dtype(case):
    return torch.bfloat16 if case["type"] == "bf16" else torch.float32


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed * 1000003 + case["cut"])
    dt = _dtype(case)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    def unit(*shape):
        x = normal(*shape)
        return (x / x.norm(dim=-1, keepdim=True)).to(dt)

    if case["op"] == "verify":
        n, w, V = case["n"], case["window"], case["vocab"]
        # peaked rows, as a softmax over a vocabulary is; the draft's logits near the target's
        logits = 2.5 * normal(n, w + 1, V)
        near = logits[:, :w] + 0.8 * normal(n, w, V)
        target = torch.softmax(logits, -1).to(dt)
        draft = torch.softmax(near, -1).to(dt)
        pick = torch.multinomial(draft.float().reshape(n * w, V), 1, generator=gen).reshape(n, w)
        lens = torch.randint(max(0, w - 2), w + 1, (n,), generator=gen, device=dev)
        return {"case": case, "target": target, "draft": draft if case["draft"] else None,
                "drafted": pick.to(torch.int32), "lens": lens.to(torch.int32),
                "uniforms": torch.rand((n, w + 1), generator=gen, device=dev)}
    h_k, h_v, d_k, d_v = case["h_k"], case["h_v"], case["d_k"], case["d_v"]
    # one decay per head: memories from about two tokens to some hundreds
    slope = torch.exp2(-8.0 * (torch.arange(h_v, device=dev) + 1) / h_v)
    log_decay = -slope * (0.9 + 0.2 * torch.rand(h_v, generator=gen, device=dev))
    if case["op"] == "prompt":
        lens = _lengths(case)
        T, n = sum(lens), len(lens)
        cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=dev)
        return {"case": case, "q": unit(T, h_k, d_k), "k": unit(T, h_k, d_k), "v": normal(T, h_v, d_v).to(dt),
                "log_decay": log_decay, "cu": cu, "lens": lens,
                "S0": normal(n, h_v, d_v, d_k) if case["enter"] else None}
    n, w, slots = case["n"], case["window"], case["slots"]
    place = torch.randperm(slots, generator=gen, device=dev)[:n].to(torch.int32)
    if case["padded"]:
        place[n - case["padded"]:] = -1
    s = {"case": case, "q": unit(n * w, h_k, d_k), "k": unit(n * w, h_k, d_k), "v": normal(n * w, h_v, d_v).to(dt),
         "pool": normal(slots, h_v, d_v, d_k), "place": place,
         "O": torch.zeros((n * w, h_v, d_v), dtype=dt, device=dev),
         "counts": torch.tensor(_counts(case), dtype=torch.int32, device=dev)}
    if case["family"] == "head":
        s["g"], s["beta"] = log_decay, None
    else:
        s["g"] = -torch.nn.functional.softplus(normal(n * w, h_v) + 2.0) * 0.1
        s["beta"] = torch.sigmoid(normal(n * w, h_v))
    return s


# ------------------------------------------------------------------ prompts


def _plain_prompt(s):
    case, lens, g = s["case"], s["lens"], s["log_decay"].double()
    n, h_v, d_k, d_v = len(lens), case["h_v"], case["d_k"], case["d_v"]
    dev, C = g.device, 128
    most = max(max(lens), 1)
    chunks = -(-most // C)
    padded = chunks * C
    cu = s["cu"].long()
    length = cu[1:] - cu[:-1]
    at = torch.arange(padded, device=dev)
    there = at[None, :] < length[:, None]  # [n, padded]
    rows = torch.where(there, cu[:-1, None] + at[None, :], 0)

    def laid(x, heads):  # packed rows -> [n, h_v, padded, d], zero behind each prompt's end
        y = x[rows].float() * there[:, :, None, None]
        return y.repeat_interleave(h_v // heads, dim=2).permute(0, 2, 1, 3).contiguous()

    k, v = laid(s["k"], case["h_k"]), laid(s["v"], h_v)
    # the state behind the last token: sum of lambda^(len - 1 - s) v_s k_s^T
    left = (length[:, None] - 1 - at[None, :]).clamp(min=0)
    weight = torch.exp(g[None, :, None] * left[:, None, :]).float()
    S = torch.matmul((v * weight[..., None]).transpose(-1, -2), k)
    if s["S0"] is not None:
        S = S + torch.exp(g[None, :] * length[:, None]).float()[:, :, None, None] * s["S0"]
    if case["state_only"]:
        return {"S": S}
    q = laid(s["q"], case["h_k"])
    q, k, v = (x.reshape(n, h_v, chunks, C, -1) for x in (q, k, v))
    i = torch.arange(C, device=dev)
    apart = i[:, None] - i[None, :]
    decay = torch.where(apart >= 0, torch.exp(g[:, None, None] * apart.clamp(min=0)), 0.0).float()  # [h, C, C]
    o = torch.matmul(torch.matmul(q, k.transpose(-1, -2)) * decay[None, :, None], v)
    # the state before each chunk from the chunks' own states
    own_state = torch.matmul(k.transpose(-1, -2), v * torch.exp(g[:, None] * (C - 1 - i)).float()[None, :, None, :, None])
    j = torch.arange(chunks, device=dev)
    gap = j[:, None] - 1 - j[None, :]
    carry = torch.where(gap >= 0, torch.exp(g[:, None, None] * (C * gap.clamp(min=0))), 0.0).float()  # [h, to, from]
    before = torch.matmul(carry[None], own_state.reshape(n, h_v, chunks, -1)).reshape(n, h_v, chunks, d_k, d_v)
    if s["S0"] is not None:
        before = before + (torch.exp(g[:, None] * (C * j)).float()[None, :, :, None, None]
                           * s["S0"].transpose(-1, -2)[:, :, None])
    o = o + torch.matmul(q, before) * torch.exp(g[:, None] * (i + 1)).float()[None, :, None, :, None]
    o = o.reshape(n, h_v, padded, d_v).permute(0, 2, 1, 3)
    return {"O": o[there].to(_dtype(case)), "S": S}


def _own_prompt(s, api):
    O, S = api.gdn_linear_attn(s["q"], s["k"], s["v"], s["log_decay"], s["cu"], s["S0"],
                               state_only=s["case"]["state_only"])
    return {"S": S} if O is None else {"O": O, "S": S}


def _exact_prompt(case, seed):
    """Token after token in 64 bits: S <- lambda S + v k^T, o = S q."""
    s = prepare(case, seed)
    lens, h_v, dev = s["lens"], case["h_v"], s["q"].device
    n, most = len(lens), max(max(s["lens"]), 1)
    S = torch.zeros((n, h_v, case["d_v"], case["d_k"]), dtype=torch.float64, device=dev)
    if s["S0"] is not None:
        S += s["S0"]
    lam = torch.exp(s["log_decay"].double())
    start = s["cu"][:-1].long()
    O = None if case["state_only"] else torch.zeros(s["v"].shape, dtype=torch.float64, device=dev)
    order = sorted(range(n), key=lambda i: -lens[i])  # the longest first: those still running are a prefix
    rank = torch.tensor(order, device=dev)
    S, start = S[rank], start[rank]
    group = h_v // case["h_k"]
    running = n
    for t in range(most):
        while running and lens[order[running - 1]] <= t:
            running -= 1
        if not running:
            break
        at = start[:running] + t
        kt = s["k"][at].double().repeat_interleave(group, dim=1)
        part = S[:running]
        part.mul_(lam[None, :, None, None]).addcmul_(s["v"][at].double().unsqueeze(-1), kt.unsqueeze(-2))
        if O is not None:
            qt = s["q"][at].double().repeat_interleave(group, dim=1)
            O[at] = torch.matmul(part, qt.unsqueeze(-1)).squeeze(-1)
    back = torch.empty_like(S)
    back[rank] = S
    return {"S": back} if O is None else {"O": O, "S": back}


# ------------------------------------------------------------------ single tokens and windows


def _plain_token(s):
    case = s["case"]
    n, w, group = case["n"], case["window"], case["h_v"] // case["h_k"]
    live = s["place"] >= 0
    where = s["place"][live].long()
    S = s["pool"][where]
    count = s["counts"][live]

    def windowed(x):
        return x.reshape(n, w, *x.shape[1:])[live].float()

    norm = case["family"] != "head"
    q, k, v = windowed(s["q"]), windowed(s["k"]), windowed(s["v"])
    if norm:
        q = q / torch.sqrt((q * q).sum(-1, keepdim=True) + 1e-6)
        k = k / torch.sqrt((k * k).sum(-1, keepdim=True) + 1e-6)
    q, k = q.repeat_interleave(group, dim=2), k.repeat_interleave(group, dim=2)
    if case["family"] == "head":
        alpha = torch.exp(s["g"])[None, None].expand(len(q), w, -1)
        beta = torch.ones_like(alpha)
    else:
        alpha, beta = torch.exp(windowed(s["g"])), windowed(s["beta"])
    outs = []
    for j in range(w):  # at most a window of tokens, each on the state that the one before left
        kj, vj = k[:, j, :, None, :], v[:, j]
        add = vj
        if case["family"] == "delta":
            add = vj - alpha[:, j, :, None] * (S * kj).sum(-1)
        new = alpha[:, j, :, None, None] * S + (beta[:, j, :, None] * add)[..., None] * kj
        S = torch.where((j < count)[:, None, None, None], new, S) if case["mode"] == "commit" else new
        if case["mode"] != "commit":
            outs.append((S * q[:, j, :, None, :]).sum(-1))
    if case["mode"] != "commit":
        s["O"].view(n, w, *s["O"].shape[1:])[live] = torch.stack(outs, 1).to(_dtype(case))
    if case["mode"] != "outputs":
        s["pool"][where] = S
    return _of_token(s)


def _of_token(s):
    mode = s["case"]["mode"]
    return {"O": s["O"]} if mode == "outputs" else {"pool": s["pool"]} if mode == "commit" else {"O": s["O"], "pool": s["pool"]}


def _own_token(s, api):
    case = s["case"]
    mode, family = case["mode"], case["family"]
    api.gdn_decode(s["q"], s["k"], s["v"], s["g"], s["beta"], s["pool"], s["place"],
                   counts=s["counts"] if mode == "commit" else None,
                   O_out=None if mode == "commit" else s["O"], l2norm_qk=family != "head",
                   state_only=mode == "commit", keep_state=mode == "outputs", scalar_decay=family == "scalar",
                   head_decay=family == "head")
    return _of_token(s)


def _exact_token(case, seed):
    """The update by its transition matrices in 64 bits: S <- S (alpha (I - beta k k^T)) + beta v k^T."""
    s = prepare(case, seed)
    n, w, h_v, d_k, dev = case["n"], case["window"], case["h_v"], case["d_k"], s["q"].device
    group = h_v // case["h_k"]
    pool, O = s["pool"].double(), s["O"].double()
    place, counts = s["place"].tolist(), s["counts"].tolist()
    eye = torch.eye(d_k, dtype=torch.float64, device=dev)
    for i in range(n):
        if place[i] < 0:
            continue
        S = pool[place[i]].clone()
        for j in range(counts[i]):
            row = i * w + j
            q, k = s["q"][row].double(), s["k"][row].double()
            if case["family"] != "head":
                q, k = (x / torch.sqrt(x.square().sum(-1, keepdim=True) + 1e-6) for x in (q, k))
            q, k = q.repeat_interleave(group, dim=0), k.repeat_interleave(group, dim=0)
            v = s["v"][row].double()
            g = (s["g"] if case["family"] == "head" else s["g"][row]).double()
            beta = torch.ones_like(g) if case["family"] == "head" else s["beta"][row].double()
            outer = k.unsqueeze(-1) * k.unsqueeze(-2)
            move = eye - beta[:, None, None] * outer if case["family"] == "delta" else eye.expand(h_v, d_k, d_k)
            S = torch.matmul(S, torch.exp(g)[:, None, None] * move) + (beta[:, None] * v).unsqueeze(-1) * k.unsqueeze(-2)
            if case["mode"] != "commit":
                O[row] = torch.matmul(S, q.unsqueeze(-1)).squeeze(-1)
        if case["mode"] != "outputs":
            pool[place[i]] = S
    return _of_token({"case": case, "O": O, "pool": pool})


# ------------------------------------------------------------------ verification of drafts


def _fixed(p):
    """Probabilities as whole multiples of 2^-FIX, rounded down; what is no number counts as 0."""
    return (torch.nan_to_num(p.double(), nan=0.0).clamp(0.0, 1.0) * float(1 << FIX)).floor().to(torch.int64)


def _plain_verify(s):
    case, target, draft = s["case"], s["target"], s["draft"]
    n, w, V = case["n"], case["window"], case["vocab"]
    drafted, lens, u = s["drafted"].long(), s["lens"].long(), s["uniforms"]
    p = target[:, :w].gather(-1, drafted.unsqueeze(-1)).squeeze(-1).double()
    q = draft.gather(-1, drafted.unsqueeze(-1)).squeeze(-1).double() if draft is not None else torch.ones_like(p)
    j = torch.arange(w, device=p.device)
    accept = (u[:, :w].double() * q < p) & (j[None, :] < lens[:, None])
    a = accept.long().cumprod(-1).sum(-1)  # accepted drafts
    i = torch.arange(n, device=p.device)
    rejected = a < lens
    last = _fixed(target[i, a])
    at = a.clamp(max=w - 1)
    if draft is not None:
        less = _fixed(draft[i, at])
    else:
        less = torch.zeros_like(last).scatter_(-1, drafted[i, at].unsqueeze(-1), 1 << FIX)
    rest = (last - less).clamp(min=0)
    use_rest = rejected & (rest.sum(-1) > 0)
    weight = torch.where(use_rest[:, None], rest, last)
    total = weight.sum(-1)
    place = torch.floor(u[:, w].double() * total.double()).to(torch.int64)
    place = torch.minimum(place.clamp(min=0), total - 1)
    token = (weight.cumsum(-1) <= place[:, None]).sum(-1)
    token = torch.where(total > 0, token, -1)
    slots = torch.arange(w + 1, device=p.device)[None, :]
    filled = torch.cat([drafted, drafted[:, :1]], -1)
    out = torch.where(slots < a[:, None], filled, torch.where(slots == a[:, None], token[:, None], -1))
    return {"counts": (a + 1).to(torch.int32), "tokens": out.to(torch.int32)}


def _own_verify(s, api):
    counts, tokens = api.gdn_verify_draft(s["target"], s["drafted"], s["uniforms"], s["draft"], s["lens"])
    return {"counts": counts, "tokens": tokens}


def _exact_verify(case, seed):
    s = prepare(case, seed)
    w, V = case["window"], case["vocab"]
    drafted, lens, u = s["drafted"].tolist(), s["lens"].tolist(), s["uniforms"].double().tolist()
    counts, tokens = [], []
    for i in range(case["n"]):
        row = []
        for j in range(lens[i]):
            x = drafted[i][j]
            q = float(s["draft"][i, j, x]) if s["draft"] is not None else 1.0
            if not u[i][j] * q < float(s["target"][i, j, x]):
                break
            row.append(x)
        a = len(row)

        def whole(p):
            return np.floor(np.clip(p.double().cpu().numpy(), 0.0, 1.0) * 2.0 ** FIX).astype(np.int64)

        weight = whole(s["target"][i, a])
        if a < lens[i]:
            if s["draft"] is not None:
                less = np.maximum(weight - whole(s["draft"][i, a]), 0)
            else:
                less = weight.copy()
                less[drafted[i][a]] = 0
            weight = less if less.any() else weight
        total = int(weight.sum())
        place = min(max(int(math.floor(u[i][w] * float(total))), 0), total - 1)
        row.append(int(np.searchsorted(np.cumsum(weight), place, side="right")) if total else -1)
        counts.append(a + 1)
        tokens.append(row + [-1] * (w + 1 - len(row)))
    return {"counts": np.array(counts, np.int32), "tokens": np.array(tokens, np.int32)}


# ------------------------------------------------------------------ what the tools call


def run(state):
    op = state["case"]["op"]
    if own:
        from gated_deltanet_state_chunked_gb300 import api
        return {"prompt": _own_prompt, "token": _own_token, "verify": _own_verify}[op](state, api)
    return {"prompt": _plain_prompt, "token": _plain_token, "verify": _plain_verify}[op](state)


def exact(case, seed):
    return {"prompt": _exact_prompt, "token": _exact_token, "verify": _exact_verify}[case["op"]](case, seed)


def work(case):
    size = 2 if case["type"] == "bf16" else 4
    n = case["n"]
    if case["op"] == "verify":
        # one row of the target for each request, one of the draft where its draft was rejected
        rows = n * (1.0 + (REJECTED if case["draft"] else 0.0))
        return {"bytes": rows * case["vocab"] * size + n * (case["window"] * 3 + 3) * 4, "flops": rows * case["vocab"]}
    h_k, h_v, d_k, d_v = case["h_k"], case["h_v"], case["d_k"], case["d_v"]
    state = h_v * d_k * d_v * 4
    if case["op"] == "prompt":
        T = case["tokens"]
        qk = (1 if case["state_only"] else 2) * h_k * d_k
        vo = (1 if case["state_only"] else 2) * h_v * d_v
        return {"bytes": T * (qk + vo) * size + n * state * (2 if case["enter"] else 1),
                "flops": T * h_v * d_k * d_v * (2.0 if case["state_only"] else 4.0)}
    live = n - case["padded"]
    used = sum(_counts(case)[:live])
    commit, keeps = case["mode"] == "commit", case["mode"] == "outputs"
    per = (1 if commit else 2) * (h_k * d_k + h_v * d_v) * size + (0 if case["family"] == "head" else 8 * h_v)
    return {"bytes": live * state * (1 if keeps else 2) + used * per,
            "flops": used * h_v * d_k * d_v * ((6.0 if case["family"] == "delta" else 4.0) - (2.0 if commit else 0.0))}
