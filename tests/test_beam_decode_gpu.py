"""The calls of a beam-decoding step one after another, as a server makes them: one attention layer over a paged cache and one
recurrent-state layer, beams that share the full pages of their past and own their open page and their state.  Against a
64-bit model that keeps every beam's whole past and knows no pages, slots or pools.

Parents and tokens are equal in every step.  A beam's score is a sum of up to 14 log probabilities, each from fp32 sums of at
most 64 products of size 1 through three layers: within 1e-6 of its size (about 5) a step, 1e-4 in all.
"""
import math

import pytest
import torch

from gated_deltanet_state_chunked_gb300 import _lib, api

pytestmark = pytest.mark.gpu

N, B, V, STEPS, PAGE, H_Q, H_KV, D = 2, 3, 61, 14, 4, 4, 2, 32


@pytest.fixture(scope="module", autouse=True)
def _library():
    _lib.load(build=True)
    torch.cuda.init()


def _weights():
    gen = torch.Generator().manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64).float().double() / 4  # noqa: E731
    return dict(embed=4 * r(V, 64), qkv=r(64, (H_Q + 2 * H_KV) * D), o=r(H_Q * D, 64), dq=r(64, D), dk=r(64, D), dv=r(64, 2 * D),
                g=r(64, 2), b=r(64, 2), do=r(2 * D, 64), head=2 * r(64, V)), (1e3 ** (-torch.arange(D // 2) / (D // 2))).float()


class _Model:
    """Whole pasts, 64 bits: a beam is (tokens, score)."""

    def __init__(self, w, freq):
        self.w, self.freq = w, freq.double()

    def logits(self, tokens):
        w = self.w
        x = w["embed"][torch.tensor(tokens)]
        T = len(tokens)
        q, k, v = (x @ w["qkv"]).split([H_Q * D, H_KV * D, H_KV * D], 1)
        angle = torch.arange(T, dtype=torch.float64)[:, None] * self.freq

        def turned(y, h):
            y = y.reshape(T, h, D)
            a, b = y[..., :D // 2], y[..., D // 2:]
            c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
            return torch.cat([a * c - b * s, b * c + a * s], -1)

        q, k, v = turned(q, H_Q), turned(k, H_KV).repeat_interleave(H_Q // H_KV, 1), v.reshape(T, H_KV, D).repeat_interleave(H_Q // H_KV, 1)
        z = torch.einsum("thd,jhd->htj", q, k) * D ** -0.5
        z = z.masked_fill(torch.ones(T, T).triu(1).bool(), -math.inf)
        y = x + torch.einsum("htj,jhd->thd", torch.softmax(z, -1), v).reshape(T, -1) @ w["o"]
        S = torch.zeros(2, D, D, dtype=torch.float64)
        for t in range(T):
            qt, kt = y[t] @ w["dq"], y[t] @ w["dk"]
            qt, kt = (u / torch.sqrt((u * u).sum() + 1e-6) for u in (qt, kt))
            a, b = torch.exp(-torch.sigmoid(y[t] @ w["g"])), torch.sigmoid(y[t] @ w["b"])
            S = a[:, None, None] * S
            S = S + (b[:, None] * ((y[t] @ w["dv"]).reshape(2, D) - S @ kt))[:, :, None] * kt
            out = (S @ qt).reshape(-1)
        return (y[-1] + out @ w["do"]) @ w["head"]


def test_beam_decoding_of_a_hybrid_model():
    w, freq = _weights()
    model = _Model(w, freq)
    dev = "cuda"
    g = {k: x.float().to(dev) for k, x in w.items()}
    freq_d = freq.to(dev)
    start = [[3, 17, 5, 41, 8, 2], [44, 9]]  # prompts, fed token by token to every beam alike
    beams = [[(list(s[:1]), 0.0 if b == 0 else -math.inf) for b in range(B)] for s in start]
    rows = N * B
    width = 6
    k_pages, v_pages = (torch.full((rows * width + 4, PAGE, H_KV, D), math.nan, device=dev) for _ in range(2))
    free = list(range(k_pages.shape[0]))
    pool = torch.zeros(rows + 3, 2, D, D, device=dev)
    slots = torch.arange(rows, dtype=torch.int32, device=dev).reshape(N, B)
    table = torch.full((rows, width), -1, dtype=torch.int32, device=dev)
    length = [0] * N
    tokens = torch.tensor([[s[0]] * B for s in start], dtype=torch.int32, device=dev)
    scores = torch.tensor([[0.0] + [-math.inf] * (B - 1)] * N, device=dev)
    for step in range(STEPS):
        # new pages where the open one is full (each beam gets its own)
        for i in range(N):
            if length[i] % PAGE == 0:
                for b in range(B):
                    table[i * B + b, length[i] // PAGE] = free.pop()
            length[i] += 1
        kv = torch.tensor([n for n in length for _ in range(B)], dtype=torch.int32, device=dev)
        x = g["embed"][tokens.reshape(-1).long()]
        qkv = (x @ g["qkv"]).view(rows, H_Q + 2 * H_KV, D)
        q, k, v = qkv[:, :H_Q], qkv[:, H_Q:H_Q + H_KV], qkv[:, H_Q + H_KV:]
        q = api.gdn_kv_append(k, v, k_pages, v_pages, table, kv, q=q, inv_freq=freq_d)
        o = api.gdn_paged_attn(q, k_pages, v_pages, table, kv)
        y = x + o.reshape(rows, -1) @ g["o"]
        o = api.gdn_decode((y @ g["dq"]).view(rows, 1, D), (y @ g["dk"]).view(rows, 1, D), (y @ g["dv"]).view(rows, 2, D),
                           -torch.sigmoid(y @ g["g"]), torch.sigmoid(y @ g["b"]), pool, slots.reshape(-1))
        logits = ((y + o.reshape(rows, -1) @ g["do"]) @ g["head"]).view(N, B, V)
        # a prompt's next token is given, the others are selected
        scores_new, parents, picked = api.gdn_beam_select(logits, scores)
        for i in range(N):
            if step + 1 < len(start[i]):
                parents[i], picked[i], scores_new[i] = torch.arange(B, device=dev), start[i][step + 1], scores[i]
        scores, tokens = scores_new, picked.clamp(min=0)
        old = slots
        slots = api.gdn_beam_reorder(pool, old, parents)
        # tables follow their parents; open pages that are not full are copied like the states, by the same call
        where = torch.arange(N, device=dev)[:, None] * B + parents.clamp(min=0).long()
        new_table = table[where.reshape(-1)].clone()
        for i in range(N):
            if length[i] % PAGE:
                at = length[i] // PAGE
                open_pages = table[i * B:(i + 1) * B, at].reshape(1, B).contiguous()
                own = [api.gdn_beam_reorder(pages, open_pages, parents[i:i + 1].contiguous()) for pages in (k_pages, v_pages)]
                assert torch.equal(own[0], own[1])
                new_table[i * B:(i + 1) * B, at] = own[0][0]
        table = new_table
        api.gdn_get_status()
        # the 64-bit model takes the same step
        for i in range(N):
            if step + 1 < len(start[i]):
                beams[i] = [(past + [start[i][step + 1]], s) for past, s in beams[i]]
                continue
            every = []
            for b, (past, s) in enumerate(beams[i]):
                if s > -math.inf:
                    lp = torch.log_softmax(model.logits(past), -1)
                    every += [(-(s + float(lp[t])), b, t) for t in range(V)]
            best = sorted(every)[:B]
            assert parents[i].tolist() == [b for _, b, _ in best], (step, i)
            assert picked[i].tolist() == [t for _, _, t in best], (step, i)
            beams[i] = [(beams[i][b][0] + [t], -s) for s, b, t in best]
            assert max(abs(a - b[1]) for a, b in zip(scores[i].tolist(), beams[i])) <= 1e-4
    assert len({tuple(past) for past, _ in beams[0]}) == B  # (the beams did part)
