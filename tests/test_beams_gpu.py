"""GPU tests of gdn_beam_select and gdn_beam_reorder against plain 64-bit forms.

Beams and tokens are equal, and so are copied rows, bit by bit.  A score is one rounding to fp32 (2^-24 of itself) of a
total whose log sum is within 1e-7 of itself, log sums below 40 here: 2^-24 |total| + 4e-6.
"""
import math

import pytest
import torch

from gated_deltanet_state_chunked_gb300 import _lib, api

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _library():
    _lib.load(build=True)
    torch.cuda.init()


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _select(logits, scores, best):
    """(totals, beams, tokens), from the definition: what is no number takes its beam out."""
    x, s = logits.cpu().double(), scores.cpu().double()
    n, b, V = x.shape
    dead = torch.isnan(x).any(-1) | (x == math.inf).any(-1) | torch.isnan(s)
    lse = torch.logsumexp(torch.where(dead[..., None], 0.0, x), -1)
    total = torch.where(dead[..., None] | (x == -math.inf), -math.inf, (s - lse)[..., None] + x)
    # a beam's continuations in the order of (logit, token), then all of them by total
    inner = torch.argsort(torch.where(torch.isnan(x), -math.inf, x), dim=-1, descending=True, stable=True)
    value, at = torch.sort(total.gather(-1, inner).reshape(n, b * V), dim=-1, descending=True, stable=True)
    at = at // V * V + inner.reshape(n, b * V).gather(-1, at)
    k = min(best, b * V)
    value = torch.cat([value[:, :k], torch.full((n, best - k), -math.inf, dtype=torch.float64)], 1)
    at = torch.cat([at[:, :k], torch.zeros((n, best - k), dtype=torch.long)], 1)
    none = value == -math.inf
    return value, torch.where(none, -1, at // V), torch.where(none, -1, at % V)


def _check(logits, scores, best, **kw):
    got = api.gdn_beam_select(logits, scores, best, **kw)
    torch.cuda.synchronize()
    want = _select(logits, scores, best)
    assert got[1].cpu().tolist() == want[1].tolist()
    assert got[2].cpu().tolist() == want[2].tolist()
    s, w = got[0].cpu().double(), want[0]
    # fp32 ends at (2 - 2^-23) 2^127: a total of 2^128 and more rounds to infinity (-6e38 in the far-apart rows)
    w = torch.where(w.abs() >= 2.0 ** 128, torch.sign(w) * math.inf, w)
    fine = torch.isfinite(w)
    assert torch.equal(s[~fine], w[~fine])
    assert bool(((s - w)[fine].abs() <= 2.0 ** -24 * w[fine].abs() + 4e-6).all())
    return got


def _logits(gen, n, b, V, dt, width=3.0):
    return (width * torch.randn(n, b, V, generator=gen)).to(dt).cuda()


def _scores(gen, n, b):
    return (-20 - 4 * torch.rand(n, b, generator=gen)).cuda()


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("n,b,best,V", [
    (1, 1, 1, 1), (1, 1, 4, 3), (3, 2, 7, 5), (1, 4, 4, 32000), (2, 3, 6, 2048), (2, 3, 6, 2049), (1, 4, 64, 511), (5, 8, 16, 16385),
    (40, 8, 16, 16384), (40, 8, 16, 33000), (2, 64, 64, 5000), (1, 1, 64, 524288), (700, 2, 3, 1000)])
def test_select(dt, n, b, best, V):
    gen = _gen(1)
    _check(_logits(gen, n, b, V, dt), _scores(gen, n, b), best)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("n,b,best,V", [(1, 4, 8, 5000), (90, 4, 8, 17000), (90, 4, 64, 17000), (1, 64, 64, 3000)])
def test_ties_go_to_the_lower_beam_and_token(dt, n, b, best, V):
    gen = _gen(2)
    scores = torch.full((n, b), -3.5, device="cuda")
    _check(torch.zeros(n, b, V, dtype=dt, device="cuda"), scores, best)  # nothing but ties
    row = torch.randint(0, 4, (1, 1, V), generator=gen).to(dt).cuda()
    _check(row.expand(n, b, V).contiguous(), scores, best)  # equal rows of few different values
    x = torch.full((n, b, V), -5.0, dtype=dt)
    x[:, :, V // 2:V // 2 + 3] = 2.0
    _check(x.cuda(), scores, best)


@pytest.mark.parametrize("V", [3000, 40000])
@pytest.mark.parametrize("n", [1, 60])
def test_sorted_rows_and_large_values_in_one_thread(V, n):
    up = torch.arange(V, dtype=F32).mul(1e-3).expand(n, 4, V)
    scores = torch.tensor([[-1.0, -1.5, -2.0, -2.25]]).expand(n, 4).contiguous().cuda()
    _check(up.contiguous().cuda(), scores, 16)
    _check(up.flip(-1).contiguous().cuda(), scores, 16)
    x = torch.zeros(n, 4, V)
    for step in (512, 2048, 4):  # values that one thread, or neighbouring threads, hold
        x[:, :, ::step] = 5 + torch.arange(len(x[0, 0, ::step])) * 1e-2
        _check(x.cuda(), scores, 64)


@pytest.mark.parametrize("dt", [F32, BF16])
def test_masked_dead_and_what_is_no_number(dt):
    gen = _gen(3)
    for n, V in ((2, 700), (100, 20000)):
        x, s = _logits(gen, n, 4, V, dt), _scores(gen, n, 4)
        s[0, 1:] = -math.inf  # a first step: one live beam
        x[1, 0, 5] = math.nan
        x[1, 1, 6] = math.inf
        x[1, 2] = -math.inf
        x[1, 3, 3:] = -math.inf  # three tokens allowed, in all
        x[1, 3, :3] = torch.tensor([1.0, 3.0, 2.0])
        got = _check(x, s, 8)
        assert got[2][1, :3].tolist() == [1, 2, 0] and got[2][1, 3:].tolist() == [-1] * 5
        s[1] = -math.inf
        got = _check(x, s, 8)
        assert got[1][1].tolist() == [-1] * 8


def test_far_apart_logits():
    x = torch.tensor([[[-1e30, 88.0, -200.0, 1e-3], [3e38, -3e38, 0.0, 1.0]]]).cuda()
    _check(x, torch.tensor([[-1e3, -2.0]]).cuda(), 8)


def test_rows_of_a_wider_array():
    gen = _gen(4)
    x = _logits(gen, 3, 4, 1111, BF16)
    _check(x[:, :, :1000], _scores(gen, 3, 4), 5)
    with pytest.raises(ValueError):
        api.gdn_beam_select(x.transpose(0, 1), _scores(gen, 4, 3), 5)


@pytest.mark.parametrize("dt", [F32, BF16])
def test_select_offsets_past_32_bits(dt):
    """Rows 2^30 values apart: what the same rows give side by side, bit by bit."""
    gen = _gen(11)
    n, b, V, step = 2, 2, 50000, 2**30
    x = _logits(gen, n, b, V, dt)
    far = torch.empty((n * b - 1) * step + V, dtype=dt, device="cuda").as_strided((n, b, V), (b * step, step, 1))
    far.copy_(x)
    scores = _scores(gen, n, b)
    assert all(torch.equal(one, other) for one, other in zip(_check(x, scores, 9), api.gdn_beam_select(far, scores, 9)))


def test_select_captured_beside_another_graph():
    gen = _gen(5)
    x, s = _logits(gen, 4, 4, 30000, F32), _scores(gen, 4, 4)
    api.gdn_beam_select(x, s)
    torch.cuda.synchronize()
    outs, graphs = [], []
    for best in (4, 8):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(api.gdn_beam_select(x, s, best))
        graphs.append(g)
    for seed in (6, 7):
        x.copy_(_logits(_gen(seed), 4, 4, 30000, F32))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for out, best in zip(outs, (4, 8)):
            want = _select(x, s, best)
            assert out[1].cpu().tolist() == want[1].tolist() and out[2].cpu().tolist() == want[2].tolist()


def test_select_on_other_streams():
    gen = _gen(8)
    x, s = _logits(gen, 8, 8, 30000, F32), _scores(gen, 8, 8)
    one = api.gdn_beam_select(x, s, 16)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [api.gdn_beam_select(x, s, 16, stream=streams[i % 3]) for i in range(30)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for out in outs for a, b in zip(one, out))


# ------------------------------------------------------------------ reorder


def _reorder(pool, slots, parents, layers):
    rows = pool.clone() if layers else pool.clone()[None]
    source = rows.clone()
    out = []
    for s, p in zip(slots, parents):
        if s[0] < 0:
            out.append([-1] * len(s))
            continue
        free = [x for j, x in enumerate(s) if j not in p]
        seen, row = set(), []
        for q in p:
            if q >= 0 and q not in seen:
                seen.add(q)
                row.append(s[q])
            else:
                row.append(free.pop(0))
                if q >= 0:
                    rows[:, row[-1]] = source[:, s[q]]
        out.append(row)
    return out, rows if layers else rows[0]


@pytest.mark.parametrize("beams", [1, 2, 5, 8, 64])
@pytest.mark.parametrize("layers", [0, 1, 3])
@pytest.mark.parametrize("row", [(4,), (2, 8, 128), (3, 33, 500)])
def test_reorder(beams, layers, row):
    gen = _gen(9)
    n = 5
    pool = torch.randn(*([layers] if layers else []), n * beams + 3, *row, generator=gen)
    slots = torch.randperm(n * beams + 3, generator=gen)[:n * beams].reshape(n, beams).to(torch.int32)
    parents = torch.randint(0, beams, (n, beams), generator=gen).to(torch.int32)
    parents[0] = torch.arange(beams)             # everyone goes on
    parents[1] = beams - 1                       # the last one's children alone
    parents[2] = torch.arange(beams).flip(0)     # a permutation: nothing is copied
    if beams > 2:
        parents[3, 1] = -1                       # a beam that continues none
        parents[3, 2] = -7
    slots[4, 0] = -1                             # padding
    p = pool.cuda()
    got = api.gdn_beam_reorder(p, slots.cuda(), parents.cuda(), layers=bool(layers))
    api.gdn_get_status()
    out, want = _reorder(pool, slots.tolist(), parents.tolist(), bool(layers))
    assert got.tolist() == out
    assert torch.equal(p.cpu(), want)


def test_reorder_rows_of_other_types_and_strides():
    gen = _gen(10)
    pages = torch.randn(12, 2, 16, 2, 8, generator=gen).to(BF16).cuda()  # one array of key and value pages
    slots, parents = torch.tensor([[3, 7, 1], [0, 2, 9]], dtype=torch.int32), torch.tensor([[1, 1, 0], [2, 2, 2]], dtype=torch.int32)
    before = pages.clone()
    api.gdn_beam_reorder(pages[:, 0], slots.cuda(), parents.cuda())
    _, want = _reorder(before[:, 0].cpu(), slots.tolist(), parents.tolist(), False)
    assert torch.equal(pages[:, 0].cpu(), want) and torch.equal(pages[:, 1], before[:, 1])
    with pytest.raises(ValueError):
        api.gdn_beam_reorder(pages.transpose(2, 3), slots.cuda(), parents.cuda())
    tokens = torch.arange(24, dtype=torch.int64).reshape(12, 2)
    t = tokens.cuda()
    api.gdn_beam_reorder(t, slots.cuda(), parents.cuda())
    assert torch.equal(t.cpu(), _reorder(tokens, slots.tolist(), parents.tolist(), False)[1])
    api.gdn_get_status()


def test_reorder_rows_past_32_bits():
    """Rows of 2^31 bytes and 48, the last of them behind 4 GB."""
    pool = torch.zeros(3, 2**31 + 48, dtype=torch.uint8, device="cuda")
    for i in range(3):
        pool[i, ::65521] = i + 1
        pool[i, -1] = 10 + i
    last = pool[2].clone()
    slots = api.gdn_beam_reorder(pool, torch.tensor([[0, 2]], dtype=torch.int32).cuda(), torch.tensor([[1, 1]], dtype=torch.int32).cuda())
    api.gdn_get_status()
    assert slots.tolist() == [[2, 0]]
    assert torch.equal(pool[0], last) and torch.equal(pool[2], last) and int(pool[1, -1]) == 11 and int(pool[1, 0]) == 2


def test_reorder_reports_what_is_malformed():
    pool = torch.arange(40.0).reshape(10, 4).cuda()
    for slots, parents, live in (([[-1, 1], [1, 2], [0, 99]], [[0, 0], [0, 0], [0, 0]], (1,)),  # (padding's other slots do not matter)
                                 ([[0, 1], [10, 2]], [[0, 0], [0, 0]], (0,)),   # past the pool
                                 ([[0, 1], [3, -1]], [[0, 0], [0, 0]], (0,)),
                                 ([[0, 0], [3, 4]], [[0, 0], [1, 1]], (1,)),    # named twice
                                 ([[0, 1], [1, 4]], [[0, 0], [1, 1]], (0,)),    # an earlier request's
                                 ([[0, 1], [3, 4]], [[0, 2], [1, 1]], (1,))):   # a parent that is no beam
        p = pool.clone()
        got = api.gdn_beam_reorder(p, torch.tensor(slots, dtype=torch.int32).cuda(), torch.tensor(parents, dtype=torch.int32).cuda())
        with pytest.raises(_lib.GdnError) as e:
            api.gdn_get_status()
        assert e.value.code == _lib.GDN_ERR_SHAPE
        out, want = _reorder(pool.cpu(), [slots[i] for i in live], [parents[i] for i in live], False)
        assert [got[i].tolist() for i in live] == out
        assert all(got[i].tolist() == [-1, -1] for i in range(len(slots)) if i not in live)
        assert torch.equal(p.cpu(), want)


def test_reorder_captured():
    gen = _gen(11)
    pool = torch.randn(12, 4, 64, generator=gen)
    p = pool.cuda()
    slots, parents = torch.tensor([[0, 5, 3]], dtype=torch.int32), torch.zeros((1, 3), dtype=torch.int32)
    sd, pd = slots.cuda(), parents.cuda()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        out = api.gdn_beam_reorder(p, sd, pd)
    for par in ([0, 0, 1], [2, 2, 2], [2, 1, 0]):
        pd.copy_(torch.tensor([par], dtype=torch.int32))
        g.replay()
        api.gdn_get_status()
        want_slots, pool = _reorder(pool, sd.tolist(), [par], False)
        assert out.tolist() == want_slots and torch.equal(p.cpu(), pool)
        sd.copy_(out)
