"""GPU tests of gdn_kv_append and gdn_paged_attn against 64-bit loops.

Tolerances, from the types:
* fp32 outputs: 1e-5 of the norm of a (token, head) row, the library's bar for fp32.  A score is a sum of up to 128 products
  of values of size 1, scaled by d^-1/2: each rounding moves it by 2^-24 of at most its largest partial sum (about 3), sqrt(128)
  of them together by 2e-6, which a weight takes over as its relative error; the sums of weights and of weighted values
  gather as much again.  lse: 1e-5 (absolute) up to values of 20, of which 2^-24 is 1e-6.
* bf16 outputs, (token, head) row by row: a rounding is off by at most 2^-9 of a value's binade top, 2^-8 = 3.9e-3 of the
  value itself.  The weights are rounded once and the output once, so a row is within 2 * 2^-8 of
  |p| . |v|; against its own norm that is 1.7e-3 sqrt(2) in the mean and, as the weights' errors are independent,
  below 6e-3 for a row of 64 values and more; a row of few keys and of few values (d = 8) can come closer to
  2 * 2^-8 * sum(p |v|) / |o|, which is what is allowed value by value.
* what is copied (values, unrotated parts) is equal bit by bit; rotated values: one rounding of the type (2^-8 or
  2^-24) of the value, and fp32 sums of two products below it: 2^-22 of the pair's norm.
"""
import math

import pytest
import torch

from gated_deltanet_state_chunked_gb300 import _lib, api
from tests import paged_ref as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _library():
    _lib.load(build=True)
    torch.cuda.init()


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32)


def _cu(new):
    return _ints([0] + list(torch.tensor(new).cumsum(0)))


def _check_rows(O, lse, want, weight, dt):
    """Rows of O and lse against {token: (O, lse)}; weight {token: sum of p |v|} bounds the roundings of bf16."""
    O, lse = O.cpu().double(), None if lse is None else lse.cpu().double()
    for t, (o, s) in want.items():
        off = (O[t] - o).abs()
        if dt is F32:
            assert bool((off.norm(dim=-1) <= 1e-5 * o.norm(dim=-1).clamp(min=1e-30)).all()), (t, off.max())
        else:
            assert bool((off <= 2 * 2.0 ** -8 * weight[t] + 1e-30).all()), (t, (off / weight[t]).max())
            if O.shape[2] >= 64:
                assert float(off.norm()) <= 6e-3 * float(o.norm()) + 1e-30, t
        if lse is not None:
            fine = torch.isfinite(s)
            assert torch.equal(lse[t][~fine], s[~fine])
            assert bool(((lse[t] - s)[fine].abs() <= 1e-5 * (1 + s[fine].abs() / 20)).all()), (t, lse[t] - s)


def _weights(q, k_pages, v_pages, *a, **kw):
    return {t: o for t, (o, _) in ref.attend(q, k_pages, v_pages.abs(), *a, **kw).items()}


def _run(new, kv, h_q, h_kv, d, page, dt, seed, *, window=0, scale=None, layout="tokens", fused=False, cu=True, max_q="exact"):
    gen = _gen(seed)
    k_pages, v_pages, table = ref.cache(gen, kv, page, h_kv, d, dt, layout=layout)
    T = sum(new)
    rows = torch.randn(T, (h_q + (2 * h_kv if fused else 0)) * d, generator=gen).to(dt)
    q = rows[:, :h_q * d].view(T, h_q, d) if not fused else rows.as_strided((T, h_q, d), (rows.shape[1], d, 1))
    cu_t = _cu(new) if cu else None
    kv_t = _ints(kv)
    want = ref.attend(q, k_pages, v_pages, table, kv_t, cu_t, window=window, scale=scale)
    weight = _weights(q, k_pages, v_pages, table, kv_t, cu_t, window=window, scale=scale)
    O = torch.full((T, h_q, d), 7.0, dtype=dt, device="cuda")
    lse = torch.full((T, h_q), 7.0, device="cuda")
    api.gdn_paged_attn(ref.on_gpu(q), ref.on_gpu(k_pages), ref.on_gpu(v_pages), table.cuda(), kv_t.cuda(),
                       None if cu_t is None else cu_t.cuda(), max_q=max(max(new), 1) if max_q == "exact" else max_q, window=window,
                       scale=scale, O_out=O, lse_out=lse)
    api.gdn_get_status()
    _check_rows(O, lse, want, weight, dt)
    for t in range(T):
        if t not in want:
            assert bool((O[t] == 7).all()) and bool((lse[t] == 7).all())


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("group", [1, 2, 3, 4, 8])
@pytest.mark.parametrize("d", [128, 64, 80, 8])
def test_single_tokens(dt, group, d):
    kv = [1, 2, 63, 64, 65, 257, 1030, -1, 128]
    _run([1] * len(kv), kv, 2 * group, 2, d, 16, dt, 1, cu=False)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("page", [1, 2, 16, 128, 512])
@pytest.mark.parametrize("layout", ["tokens", "heads", "joined"])
def test_pages_and_layouts(dt, page, layout):
    _run([3, 3, 3], [5, 300, 129], 4, 2, 64, page, dt, 2, cu=False, layout=layout, fused=True)
    _run([40, 1, 70], [45, 300, 129], 4, 2, 64, page, dt, 3, layout=layout, fused=True)
    _run([5, 5, 5], [5, 300, 129], 8, 2, 96, page, dt, 3, cu=False, layout=layout)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("window", [0, 1, 7, 64, 200])
def test_chunks_and_windows(dt, window):
    _run([130, 0, 1, 257, 33], [130, 50, 400, 700, 33], 6, 2, 128, 32, dt, 4, window=window)
    _run([5] * 4, [5, 6, 333, 129], 8, 2, 96, 32, dt, 5, window=window, cu=False)


@pytest.mark.parametrize("dt", [F32, BF16])
def test_tokens_without_a_key(dt):
    """More new tokens than the cache holds: the first ones see nothing."""
    _run([40, 3, 1], [17, 0, 0], 4, 2, 64, 16, dt, 6)
    _run([3, 3], [2, 0], 4, 2, 64, 16, dt, 7, cu=False)
    for window in (1, 5, 2**31 - 1):
        _run([40, 3, 1], [17, 0, 0], 4, 2, 64, 16, dt, 6, window=window)
        _run([3, 3], [2, 40], 4, 2, 64, 16, dt, 7, cu=False, window=window)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("n", [1, 3, 40, 700])
def test_many_requests(dt, n):
    gen = _gen(8)
    kv = torch.randint(1, 150 if n > 100 else 2000, (n,), generator=gen).tolist()
    _run([1] * n, kv, 4, 2, 64, 16, dt, 9, cu=False)


@pytest.mark.parametrize("dt", [F32, BF16])
def test_one_long_request_among_short(dt):
    _run([1] * 12, [9000] + [3] * 11, 4, 1, 128, 64, dt, 10, cu=False)
    _run([300, 2, 1], [5000, 2, 900], 4, 1, 128, 64, dt, 11)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("h_q,h_kv", [(1, 1), (5, 5), (7, 1), (32, 1), (128, 1), (24, 8)])
def test_heads(dt, h_q, h_kv):
    _run([2, 9, 1], [30, 200, 77], h_q, h_kv, 72, 16, dt, 12)


@pytest.mark.parametrize("dt", [F32, BF16])
def test_scale(dt):
    _run([4, 4], [100, 70], 2, 2, 64, 16, dt, 13, scale=0.0)
    _run([4, 4], [100, 70], 2, 2, 64, 16, dt, 14, scale=-0.3)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("page", [4, 32])
@pytest.mark.parametrize("scale", [0.0, -0.3])
@pytest.mark.parametrize("window", [0, 37])
def test_scale_of_chunks(dt, page, scale, window):
    """A scale that makes the smallest product the largest score, in the kernels of many rows."""
    _run([100, 30, 260], [300, 64, 250], 4, 2, 64, page, dt, 21, scale=scale, window=window)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("what", ["k", "v"])
def test_values_that_are_no_numbers_reach_only_who_sees_them(dt, bad, what):
    """One such value in the middle of a chunk, and behind every request's end; rows that do not see it are as without it."""
    gen = _gen(15)
    new, kv, h_q, h_kv, d, page = [100, 6], [150, 40], 4, 2, 64, 16
    k_pages, v_pages, table = ref.cache(gen, [192, 64], page, h_kv, d, dt)
    q = torch.randn(sum(new), h_q, d, generator=gen).to(dt)
    args = (table, _ints(kv), _cu(new))
    for window in (0, 20):
        clean = ref.attend(q, k_pages, v_pages, *args, window=window)
        weight = _weights(q, k_pages, v_pages, *args, window=window)
        x = (k_pages if what == "k" else v_pages).clone()
        seat = 90  # position of the value: seen by tokens 40 .. 99 of request 0 (by 40 .. 59 in a window of 20)
        x[int(table[0, seat // page]), seat % page, 1, 3] = bad
        for p in range(150, 192):
            x[int(table[0, p // page]), p % page] = bad
        for p in range(40, 64):
            x[int(table[1, p // page]), p % page] = bad
        kp, vp = (x, v_pages) if what == "k" else (k_pages, x)
        O, lse = (torch.empty(s, dtype=t, device="cuda") for s, t in (((106, h_q, d), dt), ((106, h_q), F32)))
        api.gdn_paged_attn(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), _ints(kv).cuda(), _cu(new).cuda(), max_q=100, window=window,
                           O_out=O, lse_out=lse)
        api.gdn_get_status()
        sees = {t for t in range(40, 100 if not window else 60)}
        # heads 2 and 3 read key head 1
        for t in list(clean):
            if t in sees:
                full = ref.attend(q, kp, vp, *args, window=window)[t][0]
                got = O[t].cpu().double()
                assert torch.equal(torch.isnan(got[2:]), torch.isnan(full[2:])), t
                assert torch.equal(torch.isinf(got[2:]), torch.isinf(full[2:])), t
        part = {t: v for t, v in clean.items() if t not in sees}
        _check_rows(O, lse, part, weight, dt)
        first = {t: (v[0][:2], v[1][:2]) for t, v in clean.items()}
        _check_rows(O[:, :2], lse[:, :2], first, {t: x[:2] for t, x in weight.items()}, dt)


@pytest.mark.parametrize("dt", [F32, BF16])
def test_sums_past_the_type(dt):
    """Values near the type's largest: their weighted sum before it is divided is past fp32, the output is not."""
    gen = _gen(16)
    k_pages, v_pages, table = ref.cache(gen, [100, 700], 16, 1, 64, dt)
    v_pages = torch.full_like(v_pages, 3e38)
    q = torch.randn(22, 4, 64, generator=gen).to(dt)
    for new in ([20, 2], [1, 21]):
        O = api.gdn_paged_attn(q.cuda(), k_pages.cuda(), v_pages.cuda(), table.cuda(), _ints([100, 700]).cuda(), _cu(new).cuda(),
                               max_q=21)
        assert bool(torch.isfinite(O).all())
        assert float((O.double() / v_pages[0, 0, 0, 0].double().cuda() - 1).abs().max()) <= (2.0 ** -8 if dt is BF16 else 1e-5)


def test_malformed_requests_are_skipped_and_reported():
    gen = _gen(17)
    dt, h, d, page = BF16, 2, 64, 16
    k_pages, v_pages, table = ref.cache(gen, [64] * 4, page, h, d, dt)
    q = torch.randn(12, 4, d, generator=gen).to(dt)
    for cu, kv, max_q, live in (([0, 3, 2, 9, 12], [30, 40, 50, 64], 12, (0, 3)),      # starts below an earlier offset
                                ([0, 3, 6, 9, 13], [30, 40, 50, 64], 12, (0, 1, 2)),   # past the rows
                                ([-1, 3, 6, 9, 12], [30, 40, 50, 64], 12, (1, 2, 3)),
                                ([0, 3, 6, 9, 12], [30, 65, 50, 64], 12, (0, 2, 3)),   # longer than the table
                                ([0, 2, 6, 9, 12], [30, 40, 50, 64], 3, (0, 2, 3))):   # more new tokens than max_q
        O = torch.full((12, 4, d), 7.0, dtype=dt, device="cuda")
        api.gdn_paged_attn(q.cuda(), k_pages.cuda(), v_pages.cuda(), table.cuda(), _ints(kv).cuda(), _ints(cu).cuda(), max_q=max_q,
                           O_out=O)
        with pytest.raises(_lib.GdnError) as e:
            api.gdn_get_status()
        assert e.value.code == _lib.GDN_ERR_SHAPE
        api.gdn_get_status()
        rows = set()
        for i in live:
            one = ref.attend(q[cu[i]:cu[i + 1]], k_pages, v_pages, table[i:i + 1], _ints(kv[i:i + 1]))
            w = _weights(q[cu[i]:cu[i + 1]], k_pages, v_pages, table[i:i + 1], _ints(kv[i:i + 1]))
            _check_rows(O[cu[i]:cu[i + 1]], None, one, w, dt)
            rows |= set(range(cu[i], cu[i + 1]))
        for t in set(range(12)) - rows:
            assert bool((O[t] == 7).all()), (cu, t)


def test_bad_pages_are_reported():
    """Pages outside the cache are not read: the other requests' outputs stand."""
    gen = _gen(18)
    k_pages, v_pages, table = ref.cache(gen, [64, 64], 16, 2, 64, BF16)
    q = torch.randn(4, 4, 64, generator=gen).to(BF16)
    for page in (-1, k_pages.shape[0], 1 << 30, -(1 << 31)):
        bad = table.clone()
        bad[0, 2] = page
        for new in ([2, 2], [1, 3]):
            O = api.gdn_paged_attn(q.cuda(), k_pages.cuda(), v_pages.cuda(), bad.cuda(), _ints([60, 64]).cuda(), _cu(new).cuda(), max_q=3)
            with pytest.raises(_lib.GdnError) as e:
                api.gdn_get_status()
            assert e.value.code == _lib.GDN_ERR_SHAPE
            want = ref.attend(q[new[0]:], k_pages, v_pages, table[1:], _ints([64]))
            _check_rows(O[new[0]:], None, want, _weights(q[new[0]:], k_pages, v_pages, table[1:], _ints([64])), BF16)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("page", [4, 16, 128])
def test_bad_pages_beside_chunks(dt, page):
    """The same in the kernels of many rows: another request's tiles lie in the same stretch of work."""
    gen = _gen(22)
    new, kv = [50, 70], [300, 290]
    k_pages, v_pages, table = ref.cache(gen, kv, page, 2, 64, dt)
    q = torch.randn(sum(new), 4, 64, generator=gen).to(dt)
    want = ref.attend(q[50:], k_pages, v_pages, table[1:], _ints(kv[1:]))
    weight = _weights(q[50:], k_pages, v_pages, table[1:], _ints(kv[1:]))
    for bad in (-1, k_pages.shape[0], 1 << 30, -(1 << 31)):
        t = table.clone()
        t[0, 1] = bad
        O = api.gdn_paged_attn(q.cuda(), k_pages.cuda(), v_pages.cuda(), t.cuda(), _ints(kv).cuda(), _cu(new).cuda(), max_q=70)
        with pytest.raises(_lib.GdnError) as e:
            api.gdn_get_status()
        assert e.value.code == _lib.GDN_ERR_SHAPE
        _check_rows(O[50:], None, want, weight, dt)


@pytest.mark.parametrize("dt", [F32, BF16])
def test_captured_and_replayed(dt):
    """A call captured once and replayed with other lengths, pages and queries, beside another graph and eager calls."""
    gen = _gen(19)
    h_q, h_kv, d, page = 4, 2, 64, 16
    k_pages, v_pages, table = ref.cache(gen, [600, 600, 600], page, h_kv, d, dt)
    q = torch.randn(9, h_q, d, generator=gen).to(dt)
    dev = [x.cuda() for x in (q, k_pages, v_pages, table)]
    kv, cu = _ints([3, 3, 3]).cuda(), _ints([0, 3, 6, 9]).cuda()
    O, O2 = torch.zeros(9, h_q, d, dtype=dt, device="cuda"), torch.zeros(9, h_q, d, dtype=dt, device="cuda")
    api.gdn_paged_attn(*dev, kv, cu, max_q=9, O_out=O)
    torch.cuda.synchronize()
    graphs = []
    for out, q_most in ((O, 9), (O2, 9)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            api.gdn_paged_attn(*dev, kv, cu, max_q=q_most, O_out=out)
        graphs.append(g)
    for lens, offs in (([600, 20, 333], [0, 1, 8, 9]), ([5, 590, 2], [0, 3, 3, 9]), ([-1, 64, 0], [0, 4, 5, 9])):
        kv.copy_(_ints(lens))
        cu.copy_(_ints(offs))
        O.fill_(7)
        O2.fill_(7)
        for g in graphs:
            g.replay()
        O3 = api.gdn_paged_attn(*dev, kv, cu, max_q=9)
        api.gdn_get_status()
        want = ref.attend(q, k_pages, v_pages, table, _ints(lens), _ints(offs))
        weight = _weights(q, k_pages, v_pages, table, _ints(lens), _ints(offs))
        for out in (O, O2, O3):
            _check_rows(out, None, want, weight, dt)
        assert torch.equal(O, O2)


@pytest.mark.parametrize("dt", [F32, BF16])
def test_offsets_past_32_bits(dt):
    """A cache of more than 2^31 values: its last pages give what the same pages give in a small cache, bit by bit."""
    gen = _gen(23)
    kv, page, h_kv, d = [700, 300], 16, 8, 128
    k_pages, v_pages, table = (x.cuda() for x in ref.cache(gen, kv, page, h_kv, d, dt))
    n = k_pages.shape[0]
    far = 2**31 // (page * h_kv * d) + 5
    k_far, v_far = (torch.empty(far + n, page, h_kv, d, dtype=dt, device="cuda") for _ in range(2))
    k_far[far:], v_far[far:] = k_pages, v_pages
    for new in ([1, 1], [5, 2], [100, 40]):
        cu, lens = _cu(new).cuda(), _ints(kv).cuda()
        rows = torch.randn(sum(new), 3, 2 * h_kv, d, generator=gen).to(dt).cuda()
        q, k, v = rows[:, 0], rows[:, 1, :h_kv], rows[:, 2, :h_kv]
        freq = torch.rand(d // 2, generator=gen).cuda()
        near, off = ([api.gdn_kv_append(k, v, *pages, t, lens, cu, q=q, inv_freq=freq), *pages, t]
                     for pages, t in (((k_pages, v_pages), table), ((k_far, v_far), table + far)))
        assert torch.equal(near[0], off[0]) and torch.equal(k_far[far:], k_pages) and torch.equal(v_far[far:], v_pages)
        assert torch.equal(api.gdn_paged_attn(*near, lens, cu, max_q=max(new)), api.gdn_paged_attn(*off, lens, cu, max_q=max(new)))
        api.gdn_get_status()


def test_two_streams_at_once():
    gen = _gen(20)
    k_pages, v_pages, table = ref.cache(gen, [3000] * 4, 16, 2, 128, BF16)
    q = torch.randn(4, 8, 128, generator=gen).to(BF16)
    dev = [x.cuda() for x in (q, k_pages, v_pages, table)]
    kv = _ints([3000, 2000, 100, 1]).cuda()
    one = api.gdn_paged_attn(*dev, kv)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    for _ in range(20):
        for s in streams:
            outs.append(api.gdn_paged_attn(*dev, kv, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(one, o) for o in outs)


# ------------------------------------------------------------------ append


def _run_append(new, kv, h_q, h_kv, d, page, dt, seed, *, rotary=None, axes=0, sections=None, neighbours=False, layout="tokens",
                with_q=True, cu=True, positions=None):
    gen = _gen(seed)
    rotary = d if rotary is None else rotary
    k_pages, v_pages, table = ref.cache(gen, kv, page, h_kv, d, dt, layout=layout)
    T = sum(new)
    rows = torch.randn(T, (h_q + 2 * h_kv) * d, generator=gen).to(dt)
    cut = lambda a, h: rows.as_strided((T, h, d), (rows.shape[1], d, 1), a * d)  # noqa: E731
    q, k, v = cut(0, h_q), cut(h_q, h_kv), cut(h_q + h_kv, h_kv)
    freq = None if not rotary else (1e4 ** (-torch.arange(rotary // 2, dtype=torch.float64) / (rotary // 2))).float()
    if axes:
        positions = torch.randint(0, 200000, (axes, T), generator=gen).to(torch.int32)
        positions = positions[0] if axes == 1 else positions
    cu_t, kv_t = _cu(new) if cu else None, _ints(kv)
    kw = dict(inv_freq=freq, positions=positions, sections=sections, neighbours=neighbours)
    q_ref, k_ref, v_ref = ref.append(k, v, k_pages, v_pages, table, kv, cu_t, q=q if with_q else None, **kw)
    dev = {x: None if y is None else y.cuda() if torch.is_tensor(y) else y for x, y in kw.items()}
    kp, vp = ref.on_gpu(k_pages), ref.on_gpu(v_pages)
    q_out = torch.zeros(T, h_q, d, dtype=dt, device="cuda") if with_q else None
    api.gdn_kv_append(ref.on_gpu(k), ref.on_gpu(v), kp, vp, table.cuda(), kv_t.cuda(), None if cu_t is None else cu_t.cuda(),
                      q=ref.on_gpu(q) if with_q else None, q_out=q_out, **dev)
    api.gdn_get_status()
    assert torch.equal(vp.cpu().double(), v_ref)
    step = 2.0 ** -8 if dt is BF16 else 2.0 ** -24
    for got, want in ((kp, k_ref), (q_out, q_ref)):
        if got is None:
            continue
        got = got.cpu().double()
        assert torch.equal(got[..., rotary:], want[..., rotary:])
        pair = want[..., :rotary].norm(dim=-1, keepdim=True)
        assert bool(((got - want).abs() <= step * want.abs() + 2.0 ** -22 * pair).all())


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("d,rotary", [(128, 128), (64, 64), (80, 80), (96, 32), (128, 2), (24, 12), (72, 72), (8, 8), (40, 0)])
@pytest.mark.parametrize("neighbours", [False, True])
def test_append(dt, d, rotary, neighbours):
    _run_append([3, 0, 40, 1], [3, 17, 55, 129], 6, 2, d, 16, dt, 30, rotary=rotary, neighbours=neighbours)
    _run_append([1] * 5, [1, 2, 16, 17, -1], 4, 4, d, 16, dt, 31, rotary=rotary, neighbours=neighbours, cu=False)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("axes,sections", [(1, None), (2, [8, 24]), (3, [8, 12, 12]), (4, [0, 1, 30, 1])])
def test_append_axes(dt, axes, sections):
    _run_append([3, 40], [3, 55], 4, 2, 64, 16, dt, 32, axes=axes, sections=sections)
    _run_append([3, 40], [3, 55], 4, 2, 128, 16, dt, 33, rotary=64, axes=axes, sections=sections, neighbours=True)


@pytest.mark.parametrize("layout", ["tokens", "heads", "joined"])
@pytest.mark.parametrize("page", [1, 8, 256])
def test_append_layouts(layout, page):
    _run_append([9, 70], [12, 300], 4, 2, 64, page, BF16, 34, layout=layout, with_q=False)


def test_append_far_positions():
    """Positions up to 2^31 - 1 turn by angles reduced exactly."""
    T = 8
    pos = _ints([0, 1, 99991, 1 << 20, (1 << 24) + 1, (1 << 28) + 5, (1 << 31) - 1, -3])
    _run_append([T], [T], 2, 1, 64, 16, F32, 35, positions=pos)


def test_append_tokens_without_a_place():
    _run_append([7, 2], [4, 0], 2, 1, 64, 4, BF16, 36)


def test_append_reports_bad_pages_and_ranges():
    gen = _gen(37)
    k_pages, v_pages, table = ref.cache(gen, [64, 64], 16, 2, 64, BF16)
    k, v = (torch.randn(6, 2, 64, generator=gen).to(BF16) for _ in range(2))
    for cu, kv, page in (([0, 3, 6], [20, 30], -1), ([0, 3, 6], [20, 30], k_pages.shape[0]), ([0, 4, 3], [20, 30], None),
                         ([0, 3, 7], [20, 30], None), ([0, 3, 6], [20, 65], None)):
        t = table.clone()
        if page is not None:
            t[1, 1] = page
        kp, vp = k_pages.cuda(), v_pages.cuda()
        api.gdn_kv_append(k.cuda(), v.cuda(), kp, vp, t.cuda(), _ints(kv).cuda(), _ints(cu).cuda())
        with pytest.raises(_lib.GdnError) as e:
            api.gdn_get_status()
        assert e.value.code == _lib.GDN_ERR_SHAPE
        n = cu[1]
        _, k_ref, v_ref = ref.append(k[:n], v[:n], k_pages, v_pages, table[:1], kv[:1])
        assert torch.equal(kp.cpu().double(), k_ref) and torch.equal(vp.cpu().double(), v_ref)


def test_append_in_place_and_captured():
    gen = _gen(38)
    k_pages, v_pages, table = ref.cache(gen, [64, 64], 16, 2, 64, F32)
    q, k, v = (torch.randn(4, h, 64, generator=gen) for h in (4, 2, 2))
    freq = torch.rand(32, generator=gen)
    kp, vp, qd, kv = k_pages.cuda(), v_pages.cuda(), q.cuda(), _ints([2, 2]).cuda()
    args = (k.cuda(), v.cuda(), kp, vp, table.cuda(), kv)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    fd = freq.cuda()
    api.gdn_kv_append(*args, q=qd, q_out=qd, inv_freq=fd, stream=side)
    torch.cuda.synchronize()
    q_ref, k_ref, v_ref = ref.append(k, v, k_pages, v_pages, table, [2, 2], q=q, inv_freq=freq)
    assert float((qd.cpu().double() - q_ref).norm() / q_ref.norm()) < 1e-6
    g = torch.cuda.CUDAGraph()
    q_in, q_out = q.cuda(), torch.empty(4, 4, 64, device="cuda")
    with torch.cuda.graph(g):
        api.gdn_kv_append(*args, q=q_in, q_out=q_out, inv_freq=fd)
    for lens in ([30, 31], [64, -1]):
        kv.copy_(_ints(lens))
        g.replay()
        api.gdn_get_status()
        _, k_ref, v_ref = ref.append(k, v, k_ref, v_ref, table, lens, inv_freq=freq)
        assert float((kp.cpu().double() - k_ref).norm() / k_ref.norm()) < 1e-6
        assert torch.equal(vp.cpu().double(), v_ref)
