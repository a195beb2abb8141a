"""gdn_linear_attn, gdn_decode and gdn_verify_draft refuse bad arguments on the host, before any GPU
work (CPU tests: every call below fails its checks, or has nothing to do)."""
import ctypes

import pytest
import torch

from gated_deltanet_state_chunked_gb300 import _lib, api

A = ctypes.c_void_p(1 << 20)  # aligned fake addresses, never dereferenced
B = ctypes.c_void_p((1 << 20) + 4096)
MIS = ctypes.c_void_p((1 << 20) + 8)
ODD = ctypes.c_void_p((1 << 20) + 2)


@pytest.fixture(scope="module")
def lib():
    return _lib.load(build=True)


def _dims(**kw):
    d = dict(n_seqs=2, total_tokens=6, h_k=2, h_v=4, d_k=64, d_v=64, dtype=_lib.GDN_BF16, flags=0, scale=1.0)
    d.update(kw)
    return _lib.GdnDims(**d)


def _linear(lib, dims, q=A, k=A, v=A, g=A, cu=A, S0=None, O=B, S=B):
    return lib.gdn_linear_attn(None if dims is None else ctypes.byref(dims), q, k, v, g, cu, S0, O, S, None)


def _decode(lib, dims, n_slots=4, q=A, k=A, v=A, g=A, beta=A, slots=A, counts=None, S=B, O=B):
    return lib.gdn_decode(None if dims is None else ctypes.byref(dims), n_slots, q, k, v, g, beta, slots, counts, S, O,
                          None)


def _verify(lib, target=A, draft=None, drafted=A, lens=None, uniforms=A, counts=B, tokens=B, null_dims=False, **kw):
    d = dict(n_seqs=2, n_draft=3, vocab=100, dtype=_lib.GDN_F32, target_stride=100, draft_stride=100)
    d.update(kw)
    dims = _lib.GdnVerifyDims(**d)
    return lib.gdn_verify_draft(None if null_dims else ctypes.byref(dims), target, draft, drafted, lens, uniforms, counts,
                                tokens, None)


@pytest.mark.parametrize("dims,code", [
    (dict(h_v=3), _lib.GDN_ERR_SHAPE),
    (dict(h_k=0), _lib.GDN_ERR_ARG),
    (dict(d_k=12), _lib.GDN_ERR_UNSUPPORTED),
    (dict(d_v=136), _lib.GDN_ERR_UNSUPPORTED),
    (dict(dtype=2), _lib.GDN_ERR_UNSUPPORTED),
    (dict(n_seqs=-1), _lib.GDN_ERR_ARG),
    (dict(total_tokens=-1), _lib.GDN_ERR_ARG),
    (dict(h_k=65536, h_v=65536), _lib.GDN_ERR_UNSUPPORTED),
    (dict(flags=1 << 20), _lib.GDN_ERR_ARG),
])
def test_bad_dims(lib, dims, code):
    for call in (_linear, _decode):
        assert call(lib, _dims(**dims)) == code, call
        assert lib.gdn_last_error() != b""


def test_null_dims(lib):
    assert _linear(lib, None) == _lib.GDN_ERR_ARG
    assert _decode(lib, None) == _lib.GDN_ERR_ARG
    assert _verify(lib, null_dims=True) == _lib.GDN_ERR_ARG


@pytest.mark.parametrize("flag", [_lib.GDN_QK_L2NORM, _lib.GDN_PRECISE, _lib.GDN_SCALAR_DECAY, _lib.GDN_HEAD_DECAY,
                                  _lib.GDN_KEEP_STATE])
def test_linear_flags(lib, flag):
    assert _linear(lib, _dims(flags=flag)) == _lib.GDN_ERR_ARG


@pytest.mark.parametrize("kw", [dict(cu=None), dict(S=None), dict(g=None), dict(O=None), dict(q=None), dict(k=None),
                                dict(v=None)])
def test_linear_missing(lib, kw):
    assert _linear(lib, _dims(), **kw) == _lib.GDN_ERR_ARG


@pytest.mark.parametrize("kw", [dict(q=MIS), dict(k=MIS), dict(v=MIS), dict(S0=MIS), dict(O=MIS), dict(S=MIS),
                                dict(g=ODD), dict(cu=ODD)])
def test_linear_misaligned(lib, kw):
    assert _linear(lib, _dims(), **kw) == _lib.GDN_ERR_ALIGN


def test_linear_more_work_than_a_launch_takes(lib):
    for kw in (dict(n_seqs=2**31 - 1), dict(n_seqs=2**31 - 1, total_tokens=2**31 - 1, h_k=1, h_v=1),
               dict(n_seqs=1 << 16, h_k=1 << 15, h_v=1 << 15), dict(n_seqs=0, total_tokens=2**31 - 1, h_k=1, h_v=256)):
        assert _linear(lib, _dims(**kw)) == _lib.GDN_ERR_UNSUPPORTED, kw


def test_replay_takes_no_decode_flags(lib):
    for flag in (_lib.GDN_HEAD_DECAY, _lib.GDN_KEEP_STATE):
        d = _dims(flags=flag)
        assert lib.gdn_replay(ctypes.byref(d), A, A, A, A, A, A, None, B, B, None) == _lib.GDN_ERR_ARG
        assert lib.gdn_chunk_operator(ctypes.byref(d), A, A, A, A, A, B, B, None) == _lib.GDN_ERR_ARG


@pytest.mark.parametrize("kw,code", [
    (dict(dims=dict(total_tokens=7)), _lib.GDN_ERR_SHAPE),
    (dict(dims=dict(flags=_lib.GDN_PRECISE)), _lib.GDN_ERR_ARG),
    (dict(dims=dict(flags=_lib.GDN_STATE_ONLY | _lib.GDN_KEEP_STATE)), _lib.GDN_ERR_ARG),
    (dict(dims=dict(flags=_lib.GDN_HEAD_DECAY | _lib.GDN_SCALAR_DECAY), beta=None), _lib.GDN_ERR_ARG),
    (dict(dims=dict(flags=_lib.GDN_HEAD_DECAY)), _lib.GDN_ERR_ARG),  # beta given
    (dict(beta=None), _lib.GDN_ERR_ARG),
    (dict(n_slots=-1), _lib.GDN_ERR_ARG),
    (dict(n_slots=1, slots=None), _lib.GDN_ERR_SHAPE),
    (dict(S=None), _lib.GDN_ERR_ARG),
    (dict(q=None), _lib.GDN_ERR_ARG),
    (dict(k=None), _lib.GDN_ERR_ARG),
    (dict(v=None), _lib.GDN_ERR_ARG),
    (dict(g=None), _lib.GDN_ERR_ARG),
    (dict(O=None), _lib.GDN_ERR_ARG),
    (dict(q=MIS), _lib.GDN_ERR_ALIGN),
    (dict(k=MIS), _lib.GDN_ERR_ALIGN),
    (dict(v=MIS), _lib.GDN_ERR_ALIGN),
    (dict(S=MIS), _lib.GDN_ERR_ALIGN),
    (dict(O=MIS), _lib.GDN_ERR_ALIGN),
    (dict(g=ODD), _lib.GDN_ERR_ALIGN),
    (dict(beta=ODD), _lib.GDN_ERR_ALIGN),
    (dict(slots=ODD), _lib.GDN_ERR_ALIGN),
    (dict(counts=ODD), _lib.GDN_ERR_ALIGN),
])
def test_decode_refusals(lib, kw, code):
    kw = dict(kw)
    assert _decode(lib, _dims(**kw.pop("dims", {})), **kw) == code
    assert lib.gdn_last_error() != b""


@pytest.mark.parametrize("kw,code", [
    (dict(n_seqs=-1), _lib.GDN_ERR_ARG),
    (dict(n_draft=-1), _lib.GDN_ERR_ARG),
    (dict(vocab=0), _lib.GDN_ERR_ARG),
    (dict(dtype=2), _lib.GDN_ERR_UNSUPPORTED),
    (dict(vocab=(1 << 19) + 1, target_stride=1 << 20), _lib.GDN_ERR_UNSUPPORTED),
    (dict(target_stride=99), _lib.GDN_ERR_SHAPE),
    (dict(draft=A, draft_stride=99), _lib.GDN_ERR_SHAPE),
    (dict(target=None), _lib.GDN_ERR_ARG),
    (dict(drafted=None), _lib.GDN_ERR_ARG),
    (dict(uniforms=None), _lib.GDN_ERR_ARG),
    (dict(counts=None), _lib.GDN_ERR_ARG),
    (dict(tokens=None), _lib.GDN_ERR_ARG),
    (dict(target=ODD), _lib.GDN_ERR_ALIGN),
    (dict(draft=ODD), _lib.GDN_ERR_ALIGN),
    (dict(drafted=ODD), _lib.GDN_ERR_ALIGN),
    (dict(lens=ODD), _lib.GDN_ERR_ALIGN),
    (dict(uniforms=ODD), _lib.GDN_ERR_ALIGN),
    (dict(counts=ODD), _lib.GDN_ERR_ALIGN),
    (dict(tokens=ODD), _lib.GDN_ERR_ALIGN),
])
def test_verify_refusals(lib, kw, code):
    assert _verify(lib, **kw) == code
    assert lib.gdn_last_error() != b""


def test_nothing_to_do(lib):
    assert _linear(lib, _dims(n_seqs=0)) == _lib.GDN_OK
    assert _decode(lib, _dims(n_seqs=0)) == _lib.GDN_OK
    assert _decode(lib, _dims(total_tokens=0)) == _lib.GDN_OK
    assert _verify(lib, n_seqs=0) == _lib.GDN_OK


def test_binding_refuses_cpu_tensors(lib):
    q = torch.zeros(4, 2, 64)
    g = torch.zeros(4, 2)
    with pytest.raises(ValueError, match="CUDA"):
        api.gdn_linear_attn(q, q, q, g[0], torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        api.gdn_decode(q, q, q, g, g, torch.zeros(4, 2, 64, 64))
    with pytest.raises(ValueError, match="CUDA"):
        api.gdn_verify_draft(torch.zeros(1, 3, 9), torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, 3))


def test_binding_refuses_types_and_missing_queries(lib):
    q = torch.zeros(4, 2, 64, dtype=torch.float16)
    g = torch.zeros(4, 2)
    with pytest.raises(ValueError, match="dtype"):
        api.gdn_linear_attn(q, q, q, g[0], torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="dtype"):
        api.gdn_decode(q, q, q, g, g, torch.zeros(4, 2, 64, 64))
    with pytest.raises(ValueError, match="dtype"):
        api.gdn_verify_draft(torch.zeros(1, 3, 9, dtype=torch.float64), torch.zeros(1, 2, dtype=torch.int32),
                             torch.zeros(1, 3))
    f = q.float()
    with pytest.raises(ValueError, match="q may be None"):
        api.gdn_linear_attn(None, f, f, g[0], torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="q may be None"):
        api.gdn_decode(None, f, f, g, g, torch.zeros(4, 2, 64, 64))
    with pytest.raises(ValueError, match="no requests"):
        api.gdn_decode(f, f, f, g, g, torch.zeros(0, 2, 64, 64))
