"""GPU tests of the serving calls at their edges.  64-bit forms; tolerances as in test_serving_gpu.py."""
import pytest
import torch

from gated_deltanet_state_chunked_gb300 import _lib, api
from tests import serving_ref as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TOL_F32, TOL_O_BF16 = 1e-5, 4e-3
INF, NAN = float("inf"), float("nan")


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


def _prompt(lens, h_k, h_v, d_k, d_v, dt, seed):
    gen = _gen(seed)
    T = sum(lens)
    return dict(q=_unit(gen, T, h_k, d_k).to(dt), k=_unit(gen, T, h_k, d_k).to(dt),
                v=torch.randn(T, h_v, d_v, generator=gen).to(dt),
                log_decay=-torch.exp2(-8 * torch.rand(h_v, generator=gen)),
                cu_seqlens=torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32),
                S0=torch.randn(len(lens), h_v, d_v, d_k, generator=gen))


def _cuda(x):
    return {k: None if v is None else v.cuda() for k, v in x.items()}


def _same_where_finite(x, y, tol, what):
    """x is finite exactly where y is, and near it there (2-norm of every head's finite entries)."""
    x = x.double().cpu()
    there = torch.isfinite(y)
    assert torch.equal(torch.isfinite(x), there), what
    a, b = torch.where(there, x, 0.0), torch.where(there, y, 0.0)
    assert float((a - b).norm()) <= tol * float(b.norm()), what


def _check_not_finite(x, in_place=False):
    cu = x["cu_seqlens"].tolist()
    O_ref, S_ref = ref.prompt(x["q"], x["k"], x["v"], x["log_decay"], cu, x["S0"])
    d = _cuda(x)
    O, S = api.gdn_linear_attn(**d, S_out=d["S0"] if in_place else None)
    _, S2 = api.gdn_linear_attn(**dict(_cuda(x), q=None), state_only=True)
    api.gdn_get_status()
    tol = TOL_F32 if x["k"].dtype == F32 else TOL_O_BF16
    for h in range(O.shape[1]):
        for i, (a, b) in enumerate(zip(cu, cu[1:])):
            _same_where_finite(O[a:b, h], O_ref[a:b, h], tol, ("O", i, h))
            _same_where_finite(S[i, h], S_ref[i, h], TOL_F32, ("S", i, h))
            _same_where_finite(S2[i, h], S_ref[i, h], TOL_F32, ("S alone", i, h))


NOT_FINITE_TYPES = [F32, BF16]
SHAPES = [(1, 2, 128, 128), (2, 2, 64, 64), (1, 3, 72, 104), (1, 1, 96, 40)]


@pytest.mark.parametrize("dt", NOT_FINITE_TYPES)
@pytest.mark.parametrize("h_k,h_v,d_k,d_v", SHAPES)
@pytest.mark.parametrize("at", [0, 5, 37, 64, 127, 128, 130, 255, 299])
def test_prompt_value_that_is_no_number_reaches_no_earlier_token(dt, h_k, h_v, d_k, d_v, at):
    """An infinite or NaN value reaches the outputs and the state of its own row from its token on."""
    x = _prompt([300, 129], h_k, h_v, d_k, d_v, dt, 1000 + at)
    x["v"][at, h_v - 1, d_v // 3] = INF
    x["v"][at // 2, 0, d_v - 1] = NAN
    x["v"][300 + at % 129, 0, 0] = -INF
    _check_not_finite(x)


@pytest.mark.parametrize("dt", NOT_FINITE_TYPES)
@pytest.mark.parametrize("lens", [[1000], [2049], [40, 3000, 0, 777]])
def test_prompt_values_that_are_no_numbers_in_cut_sequences(dt, lens):
    x = _prompt(lens, 1, 2, 64, 96, dt, 2000 + sum(lens))
    T = sum(lens)
    for j, at in enumerate((0, 130, 514, 900, T - 1)):
        x["v"][at, j % 2, 7 * j] = (INF, NAN, -INF)[j % 3]
    _check_not_finite(x)


@pytest.mark.parametrize("dt", NOT_FINITE_TYPES)
@pytest.mark.parametrize("value", [INF, NAN])
@pytest.mark.parametrize("decay", [0.0, -0.05, -3.0])
def test_prompt_keys_and_queries_that_are_no_numbers(dt, value, decay):
    """A key reaches its column of the state and all outputs from its token on, a query its own outputs."""
    x = _prompt([300, 200], 1, 2, 128, 64, dt, 3000)
    x["log_decay"][:] = decay
    x["k"][141, 0, 3] = value
    x["q"][330, 0, 9] = value
    x["v"][450, 1, 63] = value
    _check_not_finite(x)


@pytest.mark.parametrize("dt", NOT_FINITE_TYPES)
def test_prompt_large_finite_values_stay_finite(dt):
    x = _prompt([300], 1, 1, 128, 128, dt, 3500)
    x["v"] *= 1e19  # (a product of two overflows)
    x["S0"] *= 1e19
    _check_not_finite(x)


@pytest.mark.parametrize("dt", NOT_FINITE_TYPES)
@pytest.mark.parametrize("lens", [[300, 129], [2049]])
def test_prompt_values_that_are_no_numbers_with_the_state_in_place(dt, lens):
    x = _prompt(lens, 1, 2, 128, 72, dt, 3600)
    x["v"][77, 0, 11] = INF
    x["v"][200, 1, 71] = NAN
    x["v"][201, 1, 70] = -INF
    x["S0"][0, 1, 70, 5] = INF  # this row of the state is not finite from its start
    _check_not_finite(x, in_place=True)


@pytest.mark.parametrize("dt", NOT_FINITE_TYPES)
def test_prompt_values_that_are_no_numbers_in_many_sequences(dt):
    """Every one of 600 short sequences (more items than the GPU takes at once), every row of a few."""
    gen = _gen(3700)
    lens = torch.randint(2, 200, (600,), generator=gen).tolist()
    x = _prompt(lens, 1, 1, 64, 64, dt, 3701)
    cu = x["cu_seqlens"].tolist()
    for i, n in enumerate(lens):
        at = cu[i] + int(torch.randint(n, (1,), generator=gen))
        if i % 50 == 0:
            x["v"][at] = INF
        else:
            x["v"][at, 0, i % 64] = (INF, NAN, -INF)[i % 3]
    x["log_decay"][0] = -0.02
    _check_not_finite(x)


@pytest.mark.parametrize("dt", NOT_FINITE_TYPES)
@pytest.mark.parametrize("decay", [-1e-4, -0.5])
def test_prompt_late_value_that_is_no_number_in_a_long_sequence(dt, decay):
    """The outputs computed again carry the state over thousands of tokens."""
    x = _prompt([4000, 3], 1, 160, 8, 16, dt, 3750)  # (more heads than SMs: not cut)
    x["log_decay"][:] = decay
    x["v"][3950, :, 2] = NAN
    x["v"][3960, 7, 15] = INF
    _check_not_finite(x, in_place=True)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("n", [1, 3])
@pytest.mark.parametrize("state_only", [False, True])
def test_prompt_of_no_tokens(dt, n, state_only):
    """Empty prompts return their entering states, or zero."""
    x = _cuda(_prompt([0] * n, 1, 2, 64, 72, dt, 3800))
    O, S = api.gdn_linear_attn(**x, state_only=state_only)
    _, S2 = api.gdn_linear_attn(**dict(x, S0=None), state_only=state_only)
    api.gdn_get_status()
    assert torch.equal(S, x["S0"]) and float(S2.abs().max()) == 0.0
    assert O is None if state_only else O.shape == (0, 2, 72)


# ------------------------------------------------------------------ verification


@pytest.mark.parametrize("vocab", [1 << 19, (1 << 19) - 1, 1000])
def test_verify_rows_of_ones(vocab):
    """Rows that add up to vocab, at most 2^63 in units of 2^-44: entry floor(u vocab 2^44) >> 44 is drawn
    (whole numbers; u vocab 2^44 is exact in fp64 for a power of two, else rounded once)."""
    u = [0.0, 0.5, 0.9979, 0.9984, 0.999, 0.99999994, 1.0, 1.5]
    uniforms = torch.tensor(u, dtype=F32).reshape(-1, 1)
    target = torch.ones((1, 1, vocab), device="cuda").repeat(len(u), 1, 1)
    counts, tokens = api.gdn_verify_draft(target, torch.empty((len(u), 0), dtype=torch.int32, device="cuda"),
                                          uniforms.cuda())
    api.gdn_get_status()
    total = vocab << 44
    want = [min(int(float(x) * float(total)), total - 1) >> 44 for x in uniforms.flatten()]
    assert counts.tolist() == [1] * len(u) and tokens.flatten().tolist() == want
