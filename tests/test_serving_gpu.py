"""GPU tests of gdn_linear_attn, gdn_decode and gdn_verify_draft against 64-bit token loops.

Tolerances, from the types (relative 2-norm, taken over each (sequence, v-head) block by itself):
* fp32 results (every state; outputs of fp32 inputs): 1e-5, the library's bar for fp32.  One fp32
  rounding is 2^-24 = 6e-8; a sum of 128 terms of mixed sign, or 128 carried steps, gathers about
  sqrt(128) of them, 7e-7, and an output three such sums.
* bf16 outputs: rounding one value to bf16 moves it by up to 2^-8 = 3.9e-3 of itself and by 1.7e-3
  in the quadratic mean over a binade.  Besides the output itself, the decay-weighted scores and the
  state may each be rounded once as operands: sqrt(3) * 1.7e-3 = 2.9e-3, a little more on a small
  block: 4e-3.  (gdn_decode rounds only the output: 2^-8 holds value by value.)
"""
import math

import pytest
import torch

from gated_deltanet_state_chunked_gb300 import _lib, api
from tests import serving_ref as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TOL_F32, TOL_O_BF16 = 1e-5, 4e-3


@pytest.fixture(scope="module", autouse=True)
def _library():
    _lib.load(build=True)
    torch.cuda.init()


def _gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def _unit(gen, *shape):
    x = torch.randn(*shape, generator=gen)
    return x / x.norm(dim=-1, keepdim=True)


def _rel(x, y):
    d, n = float((x - y).norm()), float(y.norm())
    return d / n if n else (0.0 if d == 0.0 else math.inf)


def _prompt_inputs(lens, h_k, h_v, d_k, d_v, dt, seed, with_S0, extra=0):
    gen = _gen(seed)
    T = sum(lens) + extra
    cu = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32)
    x = dict(q=_unit(gen, T, h_k, d_k).to(dt), k=_unit(gen, T, h_k, d_k).to(dt),
             v=torch.randn(T, h_v, d_v, generator=gen).to(dt),
             log_decay=-torch.exp2(-8 * torch.rand(h_v, generator=gen)), cu_seqlens=cu,
             S0=torch.randn(len(lens), h_v, d_v, d_k, generator=gen) if with_S0 else None)
    return x


def _cuda(x):
    return {k: None if v is None else v.cuda() for k, v in x.items()}


def _check_prompt(x, O, S, scale=1.0, tol_o=None):
    dt = x["k"].dtype
    cu = x["cu_seqlens"].tolist()
    O_ref, S_ref = ref.prompt(x["q"], x["k"], x["v"], x["log_decay"], cu, x["S0"], scale)
    tol_o = tol_o or (TOL_F32 if dt == F32 else TOL_O_BF16)
    n, h_v = S_ref.shape[:2]
    S = S.double().cpu()
    O = None if O is None else O.double().cpu()
    for i in range(n):
        for h in range(h_v):
            assert _rel(S[i, h], S_ref[i, h]) <= TOL_F32, (i, h, "S")
            if O is not None and cu[i + 1] > cu[i]:
                a, b = O[cu[i]:cu[i + 1], h], O_ref[cu[i]:cu[i + 1], h]
                assert _rel(a, b) <= tol_o, (i, h, "O")


RAGGED = [1, 63, 0, 64, 65, 127, 128, 129, 300, 2]


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("h_k,h_v,d_k,d_v", [(2, 2, 64, 64), (2, 4, 128, 128), (1, 3, 72, 104), (2, 2, 8, 128),
                                             (1, 2, 128, 8), (1, 1, 96, 120)])
@pytest.mark.parametrize("with_S0", [False, True])
def test_prompt_ragged(dt, h_k, h_v, d_k, d_v, with_S0):
    x = _prompt_inputs(RAGGED, h_k, h_v, d_k, d_v, dt, 11 + d_k + d_v, with_S0)
    O, S = api.gdn_linear_attn(**_cuda(x), scale=0.5)
    api.gdn_get_status()
    _check_prompt(x, O, S, 0.5)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[1], [128], [1000], [2049], [700, 1, 900]])
def test_prompt_lengths(dt, d, lens):
    """Single sequences from one token to several segments of one sequence."""
    x = _prompt_inputs(lens, 1, 2, d, d, dt, 31 + sum(lens), True)
    O, S = api.gdn_linear_attn(**_cuda(x))
    api.gdn_get_status()
    _check_prompt(x, O, S)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("lens", [RAGGED, [1500]])
def test_prompt_state_only(dt, lens):
    x = _prompt_inputs(lens, 2, 4, 128, 128, dt, 17, True)
    d = _cuda(x)
    d["q"] = None
    O, S = api.gdn_linear_attn(**d, state_only=True)
    api.gdn_get_status()
    assert O is None
    _check_prompt(x, None, S)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("decay", [0.0, -1e-6, -3.0, -60.0, float("-inf")])
def test_prompt_extreme_decays(dt, decay):
    """No decay, a hardly visible one, one that a chunk underflows, one that a token does, and none left."""
    x = _prompt_inputs([300, 129], 1, 2, 128, 64, dt, 5, True)
    x["log_decay"] = torch.tensor([decay, -0.1])
    O, S = api.gdn_linear_attn(**_cuda(x))
    api.gdn_get_status()
    _check_prompt(x, O, S)


@pytest.mark.parametrize("dt", [F32, BF16])
def test_prompt_rows_outside_and_poison(dt):
    """Rows behind the last sequence hold NaN and infinities: they reach nothing, and their outputs stay."""
    lens = [70, 130, 5]
    x = _prompt_inputs(lens, 2, 2, 64, 64, dt, 3, True, extra=40)
    T = sum(lens)
    for name in ("q", "k", "v"):
        x[name][T:] = float("nan")
        x[name][T + 7:] = float("inf")
    d = _cuda(x)
    O = torch.full_like(d["v"], 7.0)
    O2, S = api.gdn_linear_attn(**d, O_out=O)
    api.gdn_get_status()
    assert O2 is O and bool((O[T:] == 7.0).all())
    x = {k: v[:T] if k in "qkv" else v for k, v in x.items()}
    _check_prompt(x, O[:T], S)


@pytest.mark.parametrize("dt", [F32, BF16])
def test_prompt_neighbours_do_not_leak(dt):
    """A sequence of NaN between two others touches neither."""
    lens = [100, 60, 200]
    x = _prompt_inputs(lens, 1, 2, 128, 128, dt, 4, False)
    clean = {k: None if v is None else v.clone() for k, v in x.items()}
    for name in ("q", "k", "v"):
        x[name][100:160] = float("nan")
    O, S = api.gdn_linear_attn(**_cuda(x))
    O_ref, S_ref = ref.prompt(clean["q"], clean["k"], clean["v"], clean["log_decay"], clean["cu_seqlens"].tolist())
    tol = TOL_F32 if dt == F32 else TOL_O_BF16
    for i, (a, b) in ((0, (0, 100)), (2, (160, 360))):
        assert _rel(S[i].double().cpu(), S_ref[i]) <= TOL_F32
        assert _rel(O[a:b].double().cpu(), O_ref[a:b]) <= tol
    assert bool(torch.isnan(S[1]).all())


@pytest.mark.parametrize("dt", [F32, BF16])
def test_prompt_in_place_state(dt):
    x = _prompt_inputs([400, 30], 1, 2, 128, 128, dt, 9, True)
    d = _cuda(x)
    O, S = api.gdn_linear_attn(**d, S_out=d["S0"])
    assert S.data_ptr() == d["S0"].data_ptr()
    _check_prompt(x, O, S)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("cu", [[0, 30, 20, 90], [0, 90, 0, 90], [0, 30, 60, 91], [-1, 30, 60, 90]])
def test_prompt_malformed_offsets(dt, cu):
    """Ranges that step back, overlap or leave the tokens are skipped and reported, the others done."""
    x = _prompt_inputs([30, 30, 30], 1, 1, 64, 64, dt, 21, False)
    d = _cuda(x)
    d["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    S = torch.full((3, 1, 64, 64), 5.0, device="cuda")
    O = torch.full_like(d["v"], 7.0)
    api.gdn_linear_attn(**d, S_out=S, O_out=O)
    with pytest.raises(_lib.GdnError) as ei:
        api.gdn_get_status()
    assert ei.value.code == _lib.GDN_ERR_SHAPE
    api.gdn_get_status()
    done, high = 0, cu[0]
    for i in range(3):
        a, b = cu[i], cu[i + 1]
        ok = a >= 0 and b >= a and b <= 90 and a >= high
        high = max(high, b)
        if ok:
            done += 1
            O_ref, S_ref = ref.prompt(x["q"], x["k"], x["v"], x["log_decay"], [a, b])
            assert _rel(S[i].double().cpu(), S_ref[0]) <= TOL_F32
        else:
            assert bool((S[i] == 5.0).all())
    assert done


def test_prompt_far_offsets():
    """Element offsets beyond 2^31: a short prompt behind 600 K tokens of others."""
    T, h = 600_000, 32
    gen = _gen(77)
    tail = 150
    q = torch.zeros(T, 1, 128, dtype=BF16, device="cuda")
    k, v = torch.zeros_like(q), torch.zeros(T, h, 128, dtype=BF16, device="cuda")
    x = _prompt_inputs([tail], 1, h, 128, 128, BF16, 78, False)
    for name, t in (("q", q), ("k", k), ("v", v)):
        t[T - tail:] = x[name].cuda()
    cu = torch.tensor([0, T - tail, T], dtype=torch.int32, device="cuda")
    O, S = api.gdn_linear_attn(q, k, v, x["log_decay"].cuda(), cu)
    api.gdn_get_status()
    _check_prompt(x, O[T - tail:], S[1:])
    assert float(S[0].abs().max()) == 0.0


@pytest.mark.parametrize("dt", [F32, BF16])
def test_prompt_stream_and_graph(dt):
    """Another stream than the current one; then captured, and replayed with other contents."""
    x = _prompt_inputs([900, 40], 1, 2, 128, 128, dt, 51, True)
    y = _prompt_inputs([900, 40], 1, 2, 128, 128, dt, 52, True)
    y["cu_seqlens"] = torch.tensor([0, 500, 940], dtype=torch.int32)
    d = _cuda(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    O, S = api.gdn_linear_attn(**d, stream=side)
    side.synchronize()
    _check_prompt(x, O, S)
    graph = torch.cuda.CUDAGraph()
    O2, S2 = torch.empty_like(O), torch.empty_like(S)
    with torch.cuda.graph(graph):
        api.gdn_linear_attn(**d, O_out=O2, S_out=S2)
    for z in (y, x):
        for name, t in _cuda(z).items():
            d[name].copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        api.gdn_get_status()
        _check_prompt(z, O2, S2)


def test_prompt_overlapping_calls_and_two_graphs():
    """Two calls in flight on two streams, and two captured graphs replayed side by side."""
    xs = [_prompt_inputs([1400 + 100 * i], 1, 2, 128, 128, BF16, 60 + i, True) for i in range(2)]
    ds = [_cuda(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    outs = [None, None]
    for _ in range(3):
        for i in range(2):
            outs[i] = api.gdn_linear_attn(**ds[i], stream=streams[i])
    torch.cuda.synchronize()
    for x, o in zip(xs, outs):
        _check_prompt(x, *o)
    graphs, res = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        O, S = torch.empty_like(outs[i][0]), torch.empty_like(outs[i][1])
        with torch.cuda.graph(g):
            api.gdn_linear_attn(**ds[i], O_out=O, S_out=S)
        graphs.append(g)
        res.append((O, S))
    for _ in range(3):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
    torch.cuda.synchronize()
    for x, o in zip(xs, res):
        _check_prompt(x, *o)


# ------------------------------------------------------------------ decode


def _decode_inputs(n, w, h_k, h_v, d_k, d_v, dt, seed, family, n_slots, unit=False):
    gen = _gen(seed)
    T = n * w
    x = dict(q=torch.randn(T, h_k, d_k, generator=gen), k=torch.randn(T, h_k, d_k, generator=gen),
             v=torch.randn(T, h_v, d_v, generator=gen))
    if unit:
        x["q"], x["k"] = _unit(gen, T, h_k, d_k), _unit(gen, T, h_k, d_k)
    x = {k: v.to(dt) for k, v in x.items()}
    if family == "head":
        x["g"], x["beta"] = -torch.exp2(-8 * torch.rand(h_v, generator=gen)), None
    else:
        x["g"] = -0.1 * torch.nn.functional.softplus(torch.randn(T, h_v, generator=gen) + 2)
        x["beta"] = torch.sigmoid(torch.randn(T, h_v, generator=gen))
    x["S_pool"] = torch.randn(n_slots, h_v, d_v, d_k, generator=gen)
    x["slots"] = torch.randperm(n_slots, generator=gen)[:n].to(torch.int32)
    return x


def _check_decode(x, w, O, pool, counts=None, keep=False, family="delta", before=None, **kw):
    n = x["slots"].numel()
    counts = [w] * n if counts is None else counts
    rows, pool_ref = ref.decode(x["q"], x["k"], x["v"], x["g"], x["beta"], x["S_pool"], x["slots"].tolist(), counts, w,
                                family=family, **kw)
    pool = pool.cpu()
    if keep:
        assert torch.equal(pool, x["S_pool"])
    else:
        for s in range(pool.shape[0]):
            if s in x["slots"].tolist():
                for h in range(pool.shape[1]):
                    assert _rel(pool[s, h].double(), pool_ref[s, h]) <= 2e-6, (s, h)
            else:
                assert torch.equal(pool[s], x["S_pool"][s])
    if O is None:
        return
    O = O.cpu()
    for t in range(O.shape[0]):
        if t in rows:
            d = (O[t].double() - rows[t]).abs()
            # sums of up to 128 terms in fp32, then the output's own rounding
            bound = 2e-6 * float(rows[t].norm()) + (rows[t].abs() * 2.0 ** -8 if O.dtype == BF16 else 0.0)
            assert bool((d <= bound).all()), t
        elif before is not None:
            assert torch.equal(O[t], before[t])


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("family", ["delta", "scalar", "head"])
@pytest.mark.parametrize("h_k,h_v,d_k,d_v", [(2, 4, 128, 128), (1, 2, 64, 64), (2, 2, 8, 128), (1, 3, 40, 72),
                                             (1, 1, 128, 8), (1, 1, 96, 120)])
@pytest.mark.parametrize("n,w", [(1, 1), (3, 1), (5, 4)])
def test_decode(dt, family, h_k, h_v, d_k, d_v, n, w):
    x = _decode_inputs(n, w, h_k, h_v, d_k, d_v, dt, 7 * n + w + d_k, family, n + 2)
    d = _cuda(x)
    O = api.gdn_decode(**d, scale=0.5, scalar_decay=family == "scalar", head_decay=family == "head")
    api.gdn_get_status()
    _check_decode(x, w, O, d["S_pool"], family=family, scale=0.5)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("n", [1, 40, 300])
def test_decode_batches(dt, n):
    """From one request to more CTAs than the GPU holds at once."""
    x = _decode_inputs(n, 1, 1, 8, 128, 128, dt, n, "delta", n + 3)
    d = _cuda(x)
    O = api.gdn_decode(**d)
    api.gdn_get_status()
    _check_decode(x, 1, O, d["S_pool"])


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("family", ["delta", "head"])
def test_decode_without_norm_and_slots(dt, family):
    x = _decode_inputs(4, 2, 2, 2, 64, 64, dt, 5, family, 4, unit=True)
    x["slots"] = torch.arange(4, dtype=torch.int32)
    d = _cuda(x)
    d["slots"] = None
    O = api.gdn_decode(**d, l2norm_qk=False, head_decay=family == "head")
    api.gdn_get_status()
    _check_decode(x, 2, O, d["S_pool"], family=family, l2norm=False)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("mode", ["step", "outputs", "commit"])
def test_decode_windows_counts_padding(dt, mode):
    """Counts from none to the whole window, padded requests, poison in every row that does not count."""
    n, w = 7, 5
    x = _decode_inputs(n, w, 2, 4, 128, 128, dt, 13, "delta", 9)
    counts = [5, 0, 1, 3, 5, 2, 4]
    x["slots"][4] = -1
    for i in range(n):
        a = i * w if x["slots"][i] < 0 else i * w + counts[i]
        for name in ("q", "k", "v", "g", "beta"):
            x[name][a:(i + 1) * w] = float("nan") if i % 2 else float("inf")
    d = _cuda(x)
    before = torch.full((n * w, 4, 128), 7.0, dtype=dt)
    O = None if mode == "commit" else before.cuda()
    if mode == "commit":
        d["q"] = None
    got = api.gdn_decode(**d, counts=torch.tensor(counts, dtype=torch.int32, device="cuda"), O_out=O,
                         state_only=mode == "commit", keep_state=mode == "outputs")
    api.gdn_get_status()
    assert got is O
    live = [c if s >= 0 else 0 for c, s in zip(counts, x["slots"].tolist())]
    if mode == "commit":
        x["q"] = None
    _check_decode(x, w, O, d["S_pool"], counts=live, keep=mode == "outputs", before=before)


def test_decode_bad_slots_and_counts_are_reported():
    n, w = 6, 2
    x = _decode_inputs(n, w, 1, 2, 64, 64, F32, 23, "delta", 8)
    slots, counts = [3, 8, 3, 5, 1, 0], [2, 2, 2, 3, -1, 1]  # past the pool, a slot twice, past the window, below it
    for bad, s, c in ((True, slots, counts), (False, [3, -1, 4, 5, 1, 0], [2, 2, 2, 2, 0, 1])):
        d = _cuda(x)
        O = torch.full((n * w, 2, 64), 7.0, device="cuda")
        d["slots"] = torch.tensor(s, dtype=torch.int32, device="cuda")
        api.gdn_decode(**d, counts=torch.tensor(c, dtype=torch.int32, device="cuda"), O_out=O)
        if bad:
            with pytest.raises(_lib.GdnError) as ei:
                api.gdn_get_status()
            assert ei.value.code == _lib.GDN_ERR_SHAPE
            live = [3, -1, -1, -1, -1, 0]
        else:
            live = s
        api.gdn_get_status()
        y = dict(x, slots=torch.tensor(live, dtype=torch.int32))
        _check_decode(y, w, O, d["S_pool"], counts=[max(0, min(w, k)) for k in c],
                      before=torch.full((n * w, 2, 64), 7.0))


def test_decode_same_slot_behind_an_empty_window():
    """The first request that updates a slot has it, not one whose window counts no token."""
    n, w = 4, 2
    x = _decode_inputs(n, w, 1, 2, 64, 64, F32, 24, "delta", 4)
    d = _cuda(x)
    d["slots"] = torch.tensor([2, 2, 1, 2], dtype=torch.int32, device="cuda")
    O = torch.full((n * w, 2, 64), 7.0, device="cuda")
    api.gdn_decode(**d, counts=torch.tensor([0, 2, 1, 2], dtype=torch.int32, device="cuda"), O_out=O)
    with pytest.raises(_lib.GdnError) as ei:
        api.gdn_get_status()
    assert ei.value.code == _lib.GDN_ERR_SHAPE
    y = dict(x, slots=torch.tensor([-1, 2, 1, -1], dtype=torch.int32))
    _check_decode(y, w, O, d["S_pool"], counts=[0, 2, 1, 0], before=torch.full((n * w, 2, 64), 7.0))


def test_decode_same_slot_with_states_kept():
    """Requests may share a state that nobody writes (several drafted branches of one request)."""
    n, w = 3, 4
    x = _decode_inputs(n, w, 1, 2, 128, 128, BF16, 29, "delta", 2)
    x["slots"] = torch.tensor([1, 1, 0], dtype=torch.int32)
    d = _cuda(x)
    O = api.gdn_decode(**d, keep_state=True)
    api.gdn_get_status()
    assert torch.equal(d["S_pool"].cpu(), x["S_pool"])
    for i in range(n):
        y = {k: v[i * w:(i + 1) * w] if k in ("q", "k", "v", "g", "beta") else v for k, v in x.items()}
        y["slots"] = x["slots"][i:i + 1]
        _check_decode(y, w, O[i * w:(i + 1) * w], d["S_pool"], keep=True)


def test_decode_far_slots():
    """A pool of more than 2^32 elements: the last state's offset needs 64 bits."""
    n_slots = 66_000
    x = _decode_inputs(2, 1, 1, 4, 128, 128, BF16, 41, "delta", 2)
    pool = torch.zeros((n_slots, 4, 128, 128), device="cuda")
    x["slots"] = torch.tensor([1, 0], dtype=torch.int32)
    where = torch.tensor([n_slots - 2, n_slots - 1], dtype=torch.int32, device="cuda")
    pool[-2:] = x["S_pool"].cuda()
    d = _cuda(x)
    d["S_pool"], d["slots"] = pool, torch.stack([where[1], where[0]])
    O = api.gdn_decode(**d)
    api.gdn_get_status()
    _check_decode(x, 1, O, pool[-2:])
    assert float(pool[:4].abs().max()) == 0.0


def test_decode_steps_equal_window_and_graph():
    """A captured single-token step, replayed over a window, ends where the window form ends.

    Not bit by bit: the window form unrolls its tokens on the entering state (o_t = c_t S q_t +
    sum_i R_it (k_i.q_t) d_i), the steps round the state to fp32 after each token.  Both evaluate the
    same real expression, so both are held to the 64-bit loop with the bounds of the other tests."""
    n, w = 4, 6
    x = _decode_inputs(n, w, 2, 4, 128, 128, BF16, 43, "delta", 6)
    d = _cuda(x)
    pool = d["S_pool"].clone()
    O = api.gdn_decode(**d)
    at = {k: d[k].view(n, w, *d[k].shape[1:]) for k in ("q", "k", "v", "g", "beta")}
    one = {k: t[:, 0].contiguous().clone() for k, t in at.items()}
    out = torch.empty((n, 4, 128), dtype=BF16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.gdn_decode(**one, S_pool=pool, slots=d["slots"], O_out=out)
    steps = torch.empty_like(O)
    for t in range(w):
        for k in one:
            one[k].copy_(at[k][:, t])
        graph.replay()
        steps.view(n, w, 4, 128)[:, t] = out
    _check_decode(x, w, steps, pool)
    _check_decode(x, w, O, d["S_pool"])


# ------------------------------------------------------------------ verification


def _verify_inputs(n, w, vocab, dt, seed, spread=2.5, noise=0.8):
    gen = _gen(seed)
    logits = spread * torch.randn(n, w + 1, vocab, generator=gen)
    target = torch.softmax(logits, -1).to(dt)
    draft = torch.softmax(logits[:, :w] + noise * torch.randn(n, w, vocab, generator=gen), -1).to(dt)
    drafted = torch.zeros(n, w, dtype=torch.int32)
    if w:
        drafted = torch.multinomial(draft.float().reshape(n * w, vocab), 1, generator=gen).reshape(n, w).to(torch.int32)
    return target, draft, drafted, torch.rand(n, w + 1, generator=gen)


def _check_verify(target, drafted, uniforms, draft, lens, status=False):
    n, w = drafted.shape
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    counts = torch.full((n,), 77, dtype=torch.int32, device="cuda")
    tokens = torch.full((n, w + 1), 77, dtype=torch.int32, device="cuda")
    lens_t = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    api.gdn_verify_draft(c(target), c(drafted), c(uniforms), c(draft), lens_t, counts_out=counts, tokens_out=tokens)
    if status:
        with pytest.raises(_lib.GdnError) as ei:
            api.gdn_get_status()
        assert ei.value.code == _lib.GDN_ERR_SHAPE
    api.gdn_get_status()
    lens = [w] * n if lens is None else [-1 if k > w else k for k in lens]
    counts_ref, tokens_ref = ref.verify(target, drafted, uniforms, draft, lens)
    counts, tokens = counts.tolist(), tokens.tolist()
    for i in range(n):
        if lens[i] < 0:  # nothing written
            assert counts[i] == 77 and tokens[i] == [77] * (w + 1), i
        else:
            assert (counts[i], tokens[i]) == (counts_ref[i], tokens_ref[i]), i
    return counts, tokens


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("with_draft", [True, False])
@pytest.mark.parametrize("n,w,vocab", [(1, 1, 1), (3, 2, 7), (5, 4, 1000), (40, 3, 32000), (2, 5, 131072), (3, 1, 33),
                                       (2, 40, 257), (3, 2, 49999)])
def test_verify(dt, with_draft, n, w, vocab):
    target, draft, drafted, u = _verify_inputs(n, w, vocab, dt, n + w + vocab)
    _check_verify(target, drafted, u, draft if with_draft else None, None)


@pytest.mark.parametrize("dt", [F32, BF16])
def test_verify_ragged_and_padded(dt):
    target, draft, drafted, u = _verify_inputs(9, 4, 500, dt, 3)
    lens = [0, 4, 2, -1, 3, 1, -5, 0, 4]
    drafted[0, 0] = -9  # behind a request's drafts: not looked at
    target[2, 4] = float("nan")
    draft[2, 3] = float("nan")
    _check_verify(target, drafted, u, draft, lens)


def test_verify_no_drafts_samples_the_target():
    target, draft, drafted, u = _verify_inputs(64, 0, 300, F32, 4)
    _check_verify(target, drafted, u, None, None)
    _check_verify(target, drafted, u, draft, None)


def test_verify_identical_distributions_accept_everything():
    target, _, drafted, u = _verify_inputs(16, 3, 200, F32, 5, noise=0.0)
    drafted = torch.multinomial(target[:, :3].reshape(48, 200), 1, generator=_gen(6)).reshape(16, 3).to(torch.int32)
    counts, _ = _check_verify(target, drafted, u, target[:, :3].contiguous(), None)
    assert counts == [4] * 16


def test_verify_edges():
    """Zero rows, NaN and infinite entries, masked vocabularies, random numbers at and past their ends."""
    n, w, vocab = 10, 2, 96
    target, draft, drafted, u = _verify_inputs(n, w, vocab, F32, 8)
    target[0] = 0.0  # nothing to sample from: rejected, token -1
    target[1, 0] = float("nan")
    target[2, 0, 5:] = 0.0  # a masked vocabulary
    target[3, 0, ::2] = float("nan")
    target[4, 0, 3] = float("inf")
    draft[5, 0] = float("nan")  # u * NaN < p is false: rejected, the weights are p's
    draft[6, 0] = 1.0  # p - q is zero throughout: p itself
    u[6, 0] = 0.999
    u[7] = 1.0
    u[8] = float("nan")
    u[9] = -0.5
    _check_verify(target, drafted, u, draft, None)
    _check_verify(target, drafted, u, None, None)


def test_verify_one_hot_rows():
    """Greedy targets: the argmax is taken, whatever the random numbers."""
    n, w, vocab = 6, 3, 1000
    _, draft, drafted, u = _verify_inputs(n, w, vocab, F32, 9)
    best = torch.randint(vocab, (n, w + 1), generator=_gen(10))
    target = torch.nn.functional.one_hot(best, vocab).float()
    drafted[2:] = best[2:, :w].to(torch.int32)
    counts, tokens = _check_verify(target, drafted, u, None, None)
    for i in range(2, n):
        assert counts[i] == w + 1 and tokens[i] == best[i].tolist()


def test_verify_bad_drafts_are_reported():
    target, draft, drafted, u = _verify_inputs(4, 3, 50, F32, 12)
    drafted[1, 0] = 50
    drafted[2, 1] = -1
    u[2, 0] = 0.0
    _check_verify(target, drafted, u, draft, None, status=True)
    _check_verify(target, drafted, u, None, None, status=True)
    target, draft, drafted, u = _verify_inputs(4, 3, 50, F32, 12)
    _check_verify(target, drafted, u, draft, [3, 4, 2, 1], status=True)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("vocab,width", [(1000, 1003), (997, 1024)])
def test_verify_strided_rows(dt, vocab, width):
    """Vocabulary slices of padded rows, their bases and strides off every vector's boundary."""
    target, draft, drafted, u = _verify_inputs(5, 3, vocab, dt, 14)
    wide_t, wide_d = torch.full((5, 4, width), 9.0, dtype=dt), torch.full((5, 3, width), 9.0, dtype=dt)
    off = width - vocab
    wide_t[:, :, off:], wide_d[:, :, off:] = target, draft
    counts, tokens = api.gdn_verify_draft(wide_t.cuda()[:, :, off:], drafted.cuda(), u.cuda(), wide_d.cuda()[:, :, off:])
    api.gdn_get_status()
    assert (counts.tolist(), tokens.tolist()) == ref.verify(target, drafted, u, draft, [3] * 5)
    with pytest.raises(ValueError, match="evenly spaced"):
        api.gdn_verify_draft(target.cuda().transpose(0, 1).contiguous().transpose(0, 1), drafted.cuda(), u.cuda())


def test_verify_distribution():
    """The emitted first token follows the target: chi-square over 20000 seeded draws, and the sampled
    token of a rejection is never one where the draft has more weight than the target."""
    vocab, n = 8, 20000
    gen = _gen(15)
    p, q = torch.softmax(torch.randn(vocab, generator=gen), -1), torch.softmax(torch.randn(vocab, generator=gen), -1)
    drafted = torch.multinomial(q, n, replacement=True, generator=gen).to(torch.int32).reshape(n, 1)
    u = torch.rand(n, 2, generator=gen)
    counts, tokens = api.gdn_verify_draft(p.expand(n, 2, vocab).contiguous().cuda(), drafted.cuda(), u.cuda(),
                                          q.expand(n, 1, vocab).contiguous().cuda())
    first = tokens[:, 0].cpu().long()
    seen = torch.bincount(first, minlength=vocab).double()
    chi2 = float(((seen - n * p.double()) ** 2 / (n * p.double())).sum())
    assert chi2 < 40.0  # 7 degrees of freedom: above 40 once in a million draws
    rejected = counts.cpu() == 1
    assert bool((p > q)[first[rejected]].all())


# ------------------------------------------------------------------ together


@pytest.mark.parametrize("family", ["delta", "head"])
def test_speculative_step_without_the_host(family):
    """Rebuild or prompt, drafted window, verification and commit in one captured graph: the pool ends
    where single tokens, one after another, take it."""
    gen = _gen(91)
    n, w, h_k, h_v, d, vocab = 3, 4, 1, 2, 128, 64
    lens = [150, 37, 260]
    T = sum(lens)
    cu = torch.tensor([0, 150, 187, 447], dtype=torch.int32, device="cuda")
    q, k = (_unit(gen, T, h_k, d).to(BF16).cuda() for _ in range(2))
    v = torch.randn(T, h_v, d, generator=gen).to(BF16).cuda()
    x = _decode_inputs(n, w, h_k, h_v, d, d, BF16, 92, family, n, unit=True)
    win = {a: None if x[a] is None else x[a].cuda() for a in ("q", "k", "v", "g", "beta")}
    head = torch.randn(h_v * d, vocab, generator=gen).cuda()
    slots = torch.tensor([2, 0, 1], dtype=torch.int32, device="cuda")
    drafted = torch.randint(vocab, (n, w - 1), generator=gen).to(torch.int32).cuda()
    u = (0.01 * torch.rand(n, w, generator=gen)).cuda()
    pool = torch.empty((n, h_v, d, d), device="cuda")
    S = torch.empty_like(pool)
    O = torch.empty((n * w, h_v, d), dtype=BF16, device="cuda")
    counts = torch.empty(n, dtype=torch.int32, device="cuda")
    tokens = torch.empty((n, w), dtype=torch.int32, device="cuda")
    kw = dict(head_decay=family == "head", l2norm_qk=family == "delta")
    if family == "delta":
        g = -0.1 * torch.rand(T, h_v, generator=gen).cuda()
        beta = torch.rand(T, h_v, generator=gen).cuda()

    def step():
        if family == "head":
            api.gdn_linear_attn(q, k, v, win["g"], cu, S_out=S, state_only=True)
        else:
            api.gdn_replay(q, k, v, g, beta, cu, S_out=S, state_only=True)
        pool.index_copy_(0, slots.long(), S)
        api.gdn_decode(**win, S_pool=pool, slots=slots, O_out=O, keep_state=True, **kw)
        target = torch.softmax(O.reshape(n, w, -1).float() @ head, -1)
        api.gdn_verify_draft(target, drafted, u, counts_out=counts, tokens_out=tokens)
        api.gdn_decode(**win, S_pool=pool, slots=slots, counts=counts, state_only=True, **kw)
        return target

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        target = step()
    pool.zero_()
    graph.replay()
    torch.cuda.synchronize()
    api.gdn_get_status()
    got = counts.tolist()
    assert (got, tokens.tolist()) == ref.verify(target, drafted, u, None, [w - 1] * n)
    assert 1 < sum(got) < n * w + 1
    entering = torch.empty_like(pool)
    entering.index_copy_(0, slots.long(), S)
    x["S_pool"], x["slots"] = entering.cpu(), slots.cpu()
    _, after = ref.decode(x["q"], x["k"], x["v"], x["g"], x["beta"], x["S_pool"], slots.tolist(), got, w, family=family,
                          l2norm=family == "delta")
    assert _rel(pool.double().cpu(), after) <= 2e-6


# ------------------------------------------------------------------ together with others, and again


def test_prompt_many_short_sequences_beside_a_replay():
    """Two hundred sequences from none to 300 tokens (work items of one chunk and of none follow each
    other), beside a replay on another stream; every repetition gives the same bits."""
    gen = _gen(101)
    lens = torch.randint(0, 300, (200,), generator=gen).tolist()
    lens[3:9] = [128, 1, 0, 0, 127, 129]
    x = _prompt_inputs(lens, 1, 3, 128, 128, BF16, 102, True)
    d = _cuda(x)
    r = _prompt_inputs([900, 700], 2, 4, 128, 128, BF16, 103, False)
    rd = _cuda(r)
    g = -0.1 * torch.rand(1600, 4, generator=gen).cuda()
    beta = torch.rand(1600, 4, generator=gen).cuda()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    runs, replays = [], []
    for _ in range(4):
        with torch.cuda.stream(side):
            replays.append(api.gdn_replay(rd["q"], rd["k"], rd["v"], g, beta, rd["cu_seqlens"]))
        runs.append(api.gdn_linear_attn(**d))
    torch.cuda.synchronize()
    api.gdn_get_status()
    for O, S in runs[1:]:
        assert torch.equal(O, runs[0][0]) and torch.equal(S, runs[0][1])
    for O, S in replays[1:]:
        assert torch.equal(O, replays[0][0]) and torch.equal(S, replays[0][1])
    _check_prompt(x, *runs[0])


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("lens", [[5000], [40, 3000, 0, 777, 2500, 1], [640] * 3])
def test_prompt_cut_sequences(dt, lens):
    """Few heads: sequences cut into segments, whole ones among them, ends inside chunks and on them."""
    x = _prompt_inputs(lens, 1, 1, 64, 96, dt, 200 + len(lens), True)
    d = _cuda(x)
    O, S = api.gdn_linear_attn(**d)
    _, S2 = api.gdn_linear_attn(**dict(d, q=None), state_only=True)
    api.gdn_get_status()
    _check_prompt(x, O, S)
    _check_prompt(x, None, S2)


@pytest.mark.parametrize("n,w", [(3, 17), (200, 9)])
def test_decode_windows_longer_than_unrolled(n, w):
    x = _decode_inputs(n, w, 1, 2, 128, 64, BF16, 300 + w, "delta", n)
    d = _cuda(x)
    counts = [(5 * i) % (w + 1) for i in range(n)]
    O = torch.zeros(n * w, 2, 64, dtype=BF16, device="cuda")
    api.gdn_decode(**d, counts=torch.tensor(counts, dtype=torch.int32, device="cuda"), O_out=O)
    api.gdn_get_status()
    _check_decode(x, w, O, d["S_pool"], counts=counts, before=torch.zeros(n * w, 2, 64, dtype=BF16))


@pytest.mark.parametrize("w", range(2, 9))
@pytest.mark.parametrize("n,h_k,h_v,d_k,d_v", [(80, 1, 2, 128, 128), (80, 2, 2, 72, 120), (80, 1, 2, 64, 40),
                                               (3, 1, 2, 128, 128), (3, 1, 2, 40, 24)])
def test_decode_every_window_length(n, h_k, h_v, d_k, d_v, w):
    """Each unrolled length on few states and on many, on heads above and below 64 rows; windows of
    which none, some or all tokens count, the rows behind them NaN."""
    dt = BF16 if w % 2 else F32
    x = _decode_inputs(n, w, h_k, h_v, d_k, d_v, dt, 700 + w, "delta", n + 2)
    counts = [(3 * i + 1) % (w + 1) for i in range(n)]
    d = _cuda(x)
    for i in range(n):
        for a in ("q", "k", "v", "g", "beta"):
            d[a][i * w + counts[i]:(i + 1) * w] = float("nan")
    O = torch.full((n * w, h_v, d_v), 7.0, dtype=dt, device="cuda")
    api.gdn_decode(**d, counts=torch.tensor(counts, dtype=torch.int32, device="cuda"), O_out=O)
    api.gdn_get_status()
    _check_decode(x, w, O, d["S_pool"], counts=counts, before=torch.full((n * w, h_v, d_v), 7.0, dtype=dt))


def test_decode_extreme_gates():
    """Gates from none to a full wipe (alpha = 0), per token and per head."""
    for family in ("delta", "scalar", "head"):
        x = _decode_inputs(2, 4, 1, 3, 64, 64, F32, 400, family, 2)
        if family == "head":
            x["g"] = torch.tensor([0.0, -200.0, float("-inf")])
        else:
            x["g"][1] = float("-inf")
            x["g"][2] = 0.0
            x["g"][5] = -200.0
        d = _cuda(x)
        O = api.gdn_decode(**d, scalar_decay=family == "scalar", head_decay=family == "head")
        api.gdn_get_status()
        _check_decode(x, 4, O, d["S_pool"], family=family)


def test_calls_on_another_stream_than_their_outputs():
    """Outputs that a call allocates belong to the stream it runs on."""
    side = torch.cuda.Stream()
    x = _decode_inputs(2, 1, 1, 2, 128, 128, BF16, 500, "delta", 2)
    d = _cuda(x)
    target, draft, drafted, u = _verify_inputs(4, 3, 5000, F32, 501)
    c = [t.cuda() for t in (target, drafted, u, draft)]
    torch.cuda.synchronize()
    O = api.gdn_decode(**d, stream=side)
    counts, tokens = api.gdn_verify_draft(*c, stream=side)
    side.synchronize()
    _check_decode(x, 1, O, d["S_pool"])
    assert (counts.tolist(), tokens.tolist()) == ref.verify(target, drafted, u, draft, [3] * 4)


def test_verify_largest_vocabulary_and_many_requests():
    target, draft, drafted, u = _verify_inputs(2, 2, 1 << 19, F32, 600)
    _check_verify(target, drafted, u, draft, None)
    target, draft, drafted, u = _verify_inputs(700, 2, 9000, BF16, 601)
    _check_verify(target, drafted, u, draft, None)
    _check_verify(target, drafted, u, None, None)
