"""GPU tests of the serving calls' kernels by dispatch: every decode kernel in every family, mode and type
on few states and on many, and prompts of more sequences than one pass of the plan takes.

64-bit forms over all requests, or sequences, at once; tolerances as in test_serving_gpu.py.
"""
import pytest
import torch

from gated_deltanet_state_chunked_gb300 import _lib, api

pytestmark = pytest.mark.gpu

F32, BF16, F64 = torch.float32, torch.bfloat16, torch.float64
TOL_F32 = 1e-5
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _library():
    _lib.load(build=True)
    torch.cuda.init()


def _gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


# ------------------------------------------------------------------ decode


def _decode_inputs(n, w, h_k, h_v, d_k, d_v, dt, family, seed):
    gen = _gen(seed)
    x = dict(q=torch.randn(n, w, h_k, d_k, generator=gen).to(dt), k=torch.randn(n, w, h_k, d_k, generator=gen).to(dt),
             v=torch.randn(n, w, h_v, d_v, generator=gen).to(dt), pool=torch.randn(n + 3, h_v, d_v, d_k, generator=gen),
             slots=torch.randperm(n + 3, generator=gen)[:n])
    if family == "head":
        x["g"], x["beta"] = -torch.exp2(-8 * torch.rand(h_v, generator=gen)), None
    else:
        x["g"] = -0.1 * torch.nn.functional.softplus(torch.randn(n, w, h_v, generator=gen) + 2)
        x["beta"] = torch.sigmoid(torch.randn(n, w, h_v, generator=gen))
    return x


def _decode_reference(x, counts, family):
    """(O [n, w, h_v, d_v], states [n, h_v, d_v, d_k]) in 64 bits; O is of interest where a token counts."""
    q, k = (t.double() / torch.sqrt(t.double().square().sum(-1, keepdim=True) + 1e-6) for t in (x["q"], x["k"]))
    v = x["v"].double()
    n, w, h_v = v.shape[:3]
    q, k = (t.repeat_interleave(h_v // k.shape[2], 2) for t in (q, k))
    S = x["pool"][x["slots"]].double()
    O = torch.zeros_like(v)
    for t in range(w):
        alpha = torch.exp(x["g"].double()).expand(n, h_v) if family == "head" else torch.exp(x["g"][:, t].double())
        beta = torch.ones_like(alpha) if family == "head" else x["beta"][:, t].double()
        new = alpha[..., None, None] * S
        add = v[:, t]
        if family == "delta":
            add = add - torch.einsum("nhvk,nhk->nhv", new, k[:, t])
        new = new + (beta[..., None] * add)[..., None] * k[:, t, :, None]
        S = torch.where((t < counts)[:, None, None, None], new, S)
        O[:, t] = torch.einsum("nhvk,nhk->nhv", S, q[:, t])
    return O, S


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("family", ["delta", "scalar", "head"])
@pytest.mark.parametrize("mode", ["step", "outputs", "commit"])
@pytest.mark.parametrize("w", [1, 2, 4, 5, 6, 11])
@pytest.mark.parametrize("n,h_k,h_v,d_k,d_v", [(80, 1, 2, 128, 128), (77, 2, 2, 72, 104), (80, 1, 2, 56, 40), (5, 1, 2, 96, 72)])
def test_decode_paths(dt, family, mode, w, n, h_k, h_v, d_k, d_v):
    """154 states and more take other kernels than fewer do (152 SMs), heads of up to 64 rows others than
    larger ones.  Some windows count no token or a few; the rows behind are NaN."""
    x = _decode_inputs(n, w, h_k, h_v, d_k, d_v, dt, family, 31 * w + d_k + n)
    counts = torch.tensor([(3 * i + 1) % (w + 1) for i in range(n)])
    O_ref, S_ref = _decode_reference(x, counts, family)
    behind = torch.arange(w)[None, :] >= counts[:, None]
    d = {a: None if x[a] is None else x[a].clone() for a in ("q", "k", "v", "g", "beta")}
    for a in ("q", "k", "v") + (() if family == "head" else ("g", "beta")):
        d[a][behind] = NAN
        d[a] = d[a].flatten(0, 1)
    d = {a: None if t is None else t.cuda() for a, t in d.items()}
    pool, O = x["pool"].cuda(), None
    if mode == "commit":
        d["q"] = None
    else:
        O = torch.full((n * w, h_v, d_v), 7.0, dtype=dt, device="cuda")
    api.gdn_decode(**d, S_pool=pool, slots=x["slots"].to(torch.int32).cuda(), counts=counts.to(torch.int32).cuda(), O_out=O,
                   state_only=mode == "commit", keep_state=mode == "outputs", scalar_decay=family == "scalar",
                   head_decay=family == "head")
    api.gdn_get_status()
    pool = pool.cpu()
    if mode == "outputs":
        assert torch.equal(pool, x["pool"])
    else:
        got = pool[x["slots"]].double()
        err = (got - S_ref).flatten(2).norm(dim=-1) / S_ref.flatten(2).norm(dim=-1)
        assert float(err.max()) <= 2e-6
        rest = torch.ones(n + 3, dtype=torch.bool)
        rest[x["slots"][counts > 0]] = False
        assert torch.equal(pool[rest], x["pool"][rest])
    if O is not None:
        O = O.cpu().view(n, w, h_v, d_v)
        assert bool((O[behind] == 7.0).all())
        bound = 2e-6 * O_ref.norm(dim=(-2, -1), keepdim=True) + (O_ref.abs() * 2.0 ** -8 if dt == BF16 else 0.0)
        assert bool(((O.double() - O_ref).abs() <= bound)[~behind].all())


@pytest.mark.parametrize("w", [1, 3])
def test_decode_thousands_of_requests_and_a_slot_named_twice(w):
    """The second of two requests on one slot, far apart, is skipped and reported, all others are done."""
    n = 2500
    x = _decode_inputs(n, w, 1, 1, 8, 16, F32, "delta", 900 + w)
    x["slots"][2111] = x["slots"][5]
    counts = torch.full((n,), w)
    counts[2111] = 0
    O_ref, S_ref = _decode_reference(x, counts, "delta")
    d = {a: x[a].flatten(0, 1).cuda() for a in ("q", "k", "v", "g", "beta")}
    pool = x["pool"].cuda()
    O = torch.full((n * w, 1, 16), 7.0, device="cuda")
    api.gdn_decode(**d, S_pool=pool, slots=x["slots"].to(torch.int32).cuda(), O_out=O)
    with pytest.raises(_lib.GdnError) as ei:
        api.gdn_get_status()
    assert ei.value.code == _lib.GDN_ERR_SHAPE
    api.gdn_get_status()
    O = O.cpu().view(n, w, 1, 16)
    done = torch.arange(n) != 2111
    assert bool((O[2111] == 7.0).all())
    err = (O[done].double() - O_ref[done]).abs() - 2e-6 * O_ref[done].norm(dim=(-2, -1), keepdim=True)
    assert float(err.max()) <= 0.0
    got = pool.cpu()[x["slots"]].double()
    assert float(((got - S_ref).flatten(2).norm(dim=-1) / S_ref.flatten(2).norm(dim=-1))[done].max()) <= 2e-6


# ------------------------------------------------------------------ prompts


def _prompt_reference(q, k, v, g, S0, ranges):
    """(O [T, d_v], S [n, d_v, d_k]) of one head in 64 bits, all sequences token by token at once."""
    q, k, v, S = q.double(), k.double(), v.double(), S0.double().clone()
    begin = torch.tensor([a for a, _ in ranges])
    length = torch.tensor([b - a for a, b in ranges])
    O = torch.zeros_like(v)
    lam = torch.exp(g.double())
    for t in range(int(length.max())):
        run = torch.nonzero(length > t).flatten()
        at = begin[run] + t
        S[run] = lam * S[run] + v[at].unsqueeze(-1) * k[at].unsqueeze(-2)
        O[at] = torch.einsum("nvk,nk->nv", S[run], q[at])
    return O, S


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("state_only", [False, True])
@pytest.mark.parametrize("d_k,d_v", [(8, 16), (64, 64)])
def test_prompt_thousands_of_sequences(dt, state_only, d_k, d_v):
    """The plan goes through 1024 sequences at a time: long ones in each pass, cut into segments (and more
    segments than it sorts), and an offset that offsets of the next pass step below."""
    gen = _gen(1100 + d_k)
    n = 2500
    lens = torch.randint(0, 40, (n,), generator=gen)
    lens[100], lens[1500], lens[2400] = 1100, 900, 3001
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)])
    T = int(cu[-1])
    cu[1020] += 200  # sequence 1019 reaches over the next ones, which are left out
    ranges, skipped, high = [], torch.zeros(n, dtype=torch.bool), -1
    for i in range(n):
        a, b = int(cu[i]), int(cu[i + 1])
        skipped[i] = not (a >= max(high, 0) and a <= b <= T)
        high = max(high, a, b)
        ranges.append((0, 0) if skipped[i] else (a, b))
    assert bool(skipped[1024:].any()) and not bool(skipped[1100:].any())
    q, k = (torch.nn.functional.normalize(torch.randn(T, 1, d_k, generator=gen), dim=-1).to(dt) for _ in range(2))
    v = torch.randn(T, 1, d_v, generator=gen).to(dt)
    g, S0 = torch.tensor([-0.03]), torch.randn(n, 1, d_v, d_k, generator=gen)
    O_ref, S_ref = _prompt_reference(q[:, 0], k[:, 0], v[:, 0], g, S0[:, 0], ranges)
    S = torch.full((n, 1, d_v, d_k), 5.0, device="cuda")
    O = None if state_only else torch.full((T, 1, d_v), 7.0, dtype=dt, device="cuda")
    api.gdn_linear_attn(None if state_only else q.cuda(), k.cuda(), v.cuda(), g.cuda(), cu.to(torch.int32).cuda(), S0.cuda(),
                        S_out=S, O_out=O, state_only=state_only)
    with pytest.raises(_lib.GdnError) as ei:
        api.gdn_get_status()
    assert ei.value.code == _lib.GDN_ERR_SHAPE
    api.gdn_get_status()
    S = S.cpu().double()[:, 0]
    assert bool((S[skipped] == 5.0).all())
    err = (S - S_ref).flatten(1).norm(dim=-1) / S_ref.flatten(1).norm(dim=-1)
    assert float(err[~skipped].max()) <= TOL_F32
    if O is None:
        return
    # The state (for S q) and the scores are rounded once each to bf16 as operands, by 2^-8 of themselves at
    # most, and so is the output: the sum of all terms' sizes, from the same recurrence on absolute values,
    # bounds what the operands' roundings do.  (1.02: the roundings of rounded terms.)
    size, _ = _prompt_reference(q[:, 0].abs(), k[:, 0].abs(), v[:, 0].abs(), g, S0[:, 0].abs(), ranges)
    r = 2.0 ** -8 if dt == BF16 else 0.0
    bound = r * O_ref.abs() + (1.02 * r + TOL_F32) * size
    O = O.cpu().double()[:, 0]
    done = torch.zeros(T, dtype=torch.bool)
    for a, b in ranges:
        done[a:b] = True
    assert bool(((O - O_ref).abs() <= bound)[done].all())
    assert bool((O[~done] == 7.0).all())


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("state_only", [False, True])
@pytest.mark.parametrize("a,b", [(0, 3000), (37, 500), (5, 2400), (2990, 3000), (40, 40), (3000, 3000), (10, 5), (-1, 64),
                                 (100, 3001)])
def test_prompt_one_sequence_inside_its_tensor(dt, state_only, a, b):
    """A call is cut by the tokens its tensors have; its only sequence may be shorter, empty or malformed."""
    gen = _gen(1300)
    T, d_k, d_v = 3000, 64, 72
    q, k = (torch.nn.functional.normalize(torch.randn(T, 1, d_k, generator=gen), dim=-1).to(dt) for _ in range(2))
    v, g, S0 = torch.randn(T, 1, d_v, generator=gen).to(dt), torch.tensor([-0.01]), torch.randn(1, 1, d_v, d_k, generator=gen)
    S = torch.full((1, 1, d_v, d_k), 5.0, device="cuda")
    O = None if state_only else torch.full((T, 1, d_v), 7.0, dtype=dt, device="cuda")
    api.gdn_linear_attn(q.cuda(), k.cuda(), v.cuda(), g.cuda(), torch.tensor([a, b], dtype=torch.int32, device="cuda"),
                        S0.cuda(), S_out=S, O_out=O, state_only=state_only)
    good = 0 <= a <= b <= T
    if not good:
        with pytest.raises(_lib.GdnError) as ei:
            api.gdn_get_status()
        assert ei.value.code == _lib.GDN_ERR_SHAPE
        a = b = 0
    api.gdn_get_status()
    O_ref, S_ref = _prompt_reference(q[:, 0], k[:, 0], v[:, 0], g, S0[:, 0], [(a, b)])
    size, _ = _prompt_reference(q[:, 0].abs(), k[:, 0].abs(), v[:, 0].abs(), g, S0[:, 0].abs(), [(a, b)])
    S = S.cpu().double()[:, 0]
    assert float((S - S_ref).norm()) <= TOL_F32 * float(S_ref.norm()) if good else bool((S == 5.0).all())
    if O is not None:
        O, r = O.cpu().double()[:, 0], 2.0 ** -8 if dt == BF16 else 0.0
        assert bool(((O - O_ref).abs() <= r * O_ref.abs() + (1.02 * r + TOL_F32) * size)[a:b].all())
        assert bool((O[:a] == 7.0).all()) and bool((O[b:] == 7.0).all())


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("h_k,h_v", [(300, 300), (100, 200)])
def test_more_heads_than_multiprocessors(dt, h_k, h_v):
    """Sequences are not cut then; decode has as many states in one request."""
    gen = _gen(1400 + h_v)
    lens, d_k, d_v = [1100, 0, 70], 16, 24
    T, n = sum(lens), len(lens)
    q, k = (torch.nn.functional.normalize(torch.randn(T, h_k, d_k, generator=gen), dim=-1).to(dt) for _ in range(2))
    v, g = torch.randn(T, h_v, d_v, generator=gen).to(dt), -torch.exp2(-8 * torch.rand(h_v, generator=gen))
    S0 = torch.randn(n, h_v, d_v, d_k, generator=gen)
    cu = torch.tensor([0, 1100, 1100, 1170])
    O, S = api.gdn_linear_attn(q.cuda(), k.cuda(), v.cuda(), g.cuda(), cu.to(torch.int32).cuda(), S0.cuda())
    api.gdn_get_status()
    O, S = O.cpu().double(), S.cpu().double()
    ranges = list(zip(cu.tolist(), cu.tolist()[1:]))
    r = 2.0 ** -8 if dt == BF16 else 0.0
    for h in (0, 1, h_v // 2, h_v - 1):
        one = (q[:, h * h_k // h_v], k[:, h * h_k // h_v], v[:, h])
        O_ref, S_ref = _prompt_reference(*one, g[h], S0[:, h], ranges)
        size, _ = _prompt_reference(*(t.abs() for t in one), g[h], S0[:, h].abs(), ranges)
        err = (S[:, h] - S_ref).flatten(1).norm(dim=-1) / S_ref.flatten(1).norm(dim=-1)
        assert float(err.max()) <= TOL_F32
        assert bool(((O[:, h] - O_ref).abs() <= r * O_ref.abs() + (1.02 * r + TOL_F32) * size).all())
    x = _decode_inputs(2, 1, h_k, h_v, d_k, d_v, dt, "delta", 1500 + h_v)
    O_ref, S_ref = _decode_reference(x, torch.tensor([1, 1]), "delta")
    pool = x["pool"].cuda()
    O = api.gdn_decode(*(x[a].flatten(0, 1).cuda() for a in ("q", "k", "v", "g", "beta")), pool, x["slots"].to(torch.int32).cuda())
    api.gdn_get_status()
    got = pool.cpu()[x["slots"]].double()
    assert float(((got - S_ref).flatten(2).norm(dim=-1) / S_ref.flatten(2).norm(dim=-1)).max()) <= 2e-6
    bound = 2e-6 * O_ref.norm(dim=(-2, -1), keepdim=True) + r * O_ref.abs()
    assert bool(((O.cpu().double().view(2, 1, h_v, d_v) - O_ref).abs() <= bound).all())


def test_more_exact_ways_to_a_bf16_prompt():
    """What the header names for callers who need more than bf16 outputs give: widened inputs, and the replay
    of the scalar family with one decay per head.  Both are the same recurrence; the replay at fp32 accuracy
    rounds its outputs alone (2^-8 of each value)."""
    gen = _gen(1600)
    T, h_k, h_v, d = 700, 1, 2, 128
    q, k = (torch.nn.functional.normalize(torch.randn(T, h_k, d, generator=gen), dim=-1).to(BF16).cuda() for _ in range(2))
    v, g = torch.randn(T, h_v, d, generator=gen).to(BF16).cuda(), torch.tensor([-0.4, -0.004]).cuda()
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    O1, S1 = api.gdn_linear_attn(q.float(), k.float(), v.float(), g, cu)
    O2, S2 = api.gdn_replay(q, k, v, g.expand(T, h_v).contiguous(), torch.ones(T, h_v, device="cuda"), cu, l2norm_qk=False,
                            scalar_decay=True, precise=True)
    api.gdn_get_status()
    for h in range(h_v):
        one = [t.cpu() for t in (q[:, 0], k[:, 0], v[:, h])]
        O_ref, S_ref = _prompt_reference(*one, g[h].cpu(), torch.zeros(1, d, d), [(0, T)])
        size, _ = _prompt_reference(*(t.abs() for t in one), g[h].cpu(), torch.zeros(1, d, d), [(0, T)])
        for S in (S1, S2):
            assert float((S[0, h].cpu().double() - S_ref[0]).norm()) <= TOL_F32 * float(S_ref[0].norm())
        assert float((O1[:, h].cpu().double() - O_ref).norm()) <= TOL_F32 * float(O_ref.norm())
        assert bool(((O2[:, h].cpu().double() - O_ref).abs() <= 2.0 ** -8 * O_ref.abs() + TOL_F32 * size).all())
