"""gdn_kv_append, gdn_paged_attn, gdn_beam_select and gdn_beam_reorder refuse bad arguments on the host, before any GPU work
(CPU tests: every call below fails its checks, or has nothing to do)."""
import ctypes

import pytest
import torch

from gated_deltanet_state_chunked_gb300 import _lib, api

A = ctypes.c_void_p(1 << 20)  # aligned fake addresses, never dereferenced
B = ctypes.c_void_p((1 << 20) + 4096)
MIS = ctypes.c_void_p((1 << 20) + 8)
ODD = ctypes.c_void_p((1 << 20) + 2)
ARG, SHAPE, ALIGN, UNSUPPORTED = _lib.GDN_ERR_ARG, _lib.GDN_ERR_SHAPE, _lib.GDN_ERR_ALIGN, _lib.GDN_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    return _lib.load(build=True)


def _dims(**kw):
    d = dict(n_seqs=2, total_tokens=6, max_q=6, h_q=4, h_kv=2, d=64, page_size=16, n_pages=10, table_width=5, dtype=_lib.GDN_BF16,
             window=0, scale=1.0, table_stride=5, q_stride=256, k_stride=128, v_stride=128, k_page=2048, k_token=128, k_head=64,
             v_page=2048, v_token=128, v_head=64)
    d.update(kw)
    return _lib.GdnPagedDims(**d)


def _attn(lib, dims, q=A, k=A, v=A, table=A, lens=A, cu=A, O=B, lse=None):
    return lib.gdn_paged_attn(None if dims is None else ctypes.byref(dims), q, k, v, table, lens, cu, O, lse, None)


def _rotary(**kw):
    d = dict(rotary_dim=64, neighbours=0, n_axes=1)
    sections = kw.pop("sections", ())
    d.update(kw)
    r = _lib.GdnRotary(**d)
    r.sections[:len(sections)] = sections
    return r


def _append(lib, dims, rotary=None, q=A, k=A, v=A, freq=A, pos=None, table=A, lens=A, cu=A, kp=B, vp=B, q_out=B):
    return lib.gdn_kv_append(None if dims is None else ctypes.byref(dims), None if rotary is None else ctypes.byref(rotary), q, k, v,
                             freq, pos, table, lens, cu, kp, vp, q_out, None)


def _select(lib, null_dims=False, logits=A, scores=A, so=B, po=B, to=B, **kw):
    d = dict(n_seqs=2, beams=4, best=4, vocab=100, dtype=_lib.GDN_F32, stride=100)
    d.update(kw)
    return lib.gdn_beam_select(None if null_dims else ctypes.byref(_lib.GdnBeamDims(**d)), logits, scores, so, po, to, None)


def _reorder(lib, null_dims=False, slots=A, parents=A, pool=B, out=B, **kw):
    d = dict(n_seqs=2, beams=4, n_slots=10, layers=1, row_bytes=64, slot_stride=64, layer_stride=640)
    d.update(kw)
    return lib.gdn_beam_reorder(None if null_dims else ctypes.byref(_lib.GdnReorderDims(**d)), slots, parents, pool, out, None)


@pytest.mark.parametrize("kw,code", [
    (dict(n_seqs=-1), ARG), (dict(total_tokens=-1), ARG), (dict(dtype=2), UNSUPPORTED), (dict(h_q=0), ARG), (dict(h_kv=0), ARG),
    (dict(h_q=3), SHAPE), (dict(h_q=129 * 2, q_stride=1 << 20), UNSUPPORTED), (dict(h_q=65536 * 2, h_kv=65536, q_stride=1 << 30), UNSUPPORTED),
    (dict(d=4), UNSUPPORTED), (dict(d=136), UNSUPPORTED), (dict(d=0), UNSUPPORTED), (dict(max_q=0), ARG), (dict(page_size=0), UNSUPPORTED),
    (dict(page_size=24), UNSUPPORTED), (dict(n_pages=-1), ARG), (dict(table_width=-1), ARG), (dict(window=-1), ARG),
    (dict(total_tokens=2**31 - 1000), UNSUPPORTED), (dict(table_width=1 << 30, table_stride=1 << 30), UNSUPPORTED), (dict(table_stride=4), SHAPE),
    (dict(k_page=-8), ARG), (dict(v_token=4), ALIGN), (dict(k_head=60), ALIGN), (dict(q_stride=248), SHAPE), (dict(q_stride=260), ALIGN),
])
def test_paged_dims(lib, kw, code):
    assert _attn(lib, _dims(**kw)) == code
    assert lib.gdn_last_error() != b""
    assert _append(lib, _dims(**kw)) == code


def test_null_dims(lib):
    assert _attn(lib, None) == ARG
    assert _append(lib, None) == ARG
    assert _select(lib, null_dims=True) == ARG
    assert _reorder(lib, null_dims=True) == ARG


def test_windows_of_one_length(lib):
    assert _attn(lib, _dims(total_tokens=7, max_q=7), cu=None) == SHAPE
    assert _attn(lib, _dims(max_q=2), cu=None) == SHAPE
    assert _append(lib, _dims(max_q=2), cu=None) == SHAPE


@pytest.mark.parametrize("kw", [dict(q=None), dict(k=None), dict(v=None), dict(table=None), dict(lens=None), dict(O=None)])
def test_attn_missing(lib, kw):
    assert _attn(lib, _dims(), **kw) == ARG


@pytest.mark.parametrize("kw", [dict(q=MIS), dict(k=MIS), dict(v=MIS), dict(O=MIS), dict(table=ODD), dict(lens=ODD), dict(cu=ODD), dict(lse=ODD)])
def test_attn_misaligned(lib, kw):
    assert _attn(lib, _dims(), **kw) == ALIGN


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), ARG), (dict(v=None), ARG), (dict(kp=None), ARG), (dict(vp=None), ARG), (dict(q=None), ARG), (dict(q_out=None), ARG),
    (dict(lens=None), ARG), (dict(kp=MIS), ALIGN), (dict(q_out=MIS), ALIGN), (dict(rotary=_rotary(), freq=None), ARG),
    (dict(rotary=_rotary(), freq=ODD), ALIGN), (dict(rotary=_rotary(), pos=ODD), ALIGN),
    (dict(rotary=_rotary(rotary_dim=63)), UNSUPPORTED), (dict(rotary=_rotary(rotary_dim=66)), UNSUPPORTED),
    (dict(rotary=_rotary(rotary_dim=-2)), UNSUPPORTED), (dict(rotary=_rotary(n_axes=0)), UNSUPPORTED),
    (dict(rotary=_rotary(n_axes=5)), UNSUPPORTED), (dict(rotary=_rotary(neighbours=2)), ARG),
    (dict(rotary=_rotary(n_axes=2, sections=(16, 15)), pos=A), SHAPE), (dict(rotary=_rotary(n_axes=2, sections=(33, -1)), pos=A), ARG),
    (dict(rotary=_rotary(n_axes=2, sections=(16, 16))), ARG),
])
def test_append_refusals(lib, kw, code):
    assert _append(lib, _dims(), **kw) == code


def test_append_strides(lib):
    assert _append(lib, _dims(k_stride=120)) == SHAPE
    assert _append(lib, _dims(v_stride=132)) == ALIGN
    assert _append(lib, _dims(q_stride=512), q=A, q_out=A) == ARG  # in place only without gaps


@pytest.mark.parametrize("kw,code", [
    (dict(n_seqs=-1), ARG), (dict(beams=0), ARG), (dict(best=0), ARG), (dict(vocab=0), ARG), (dict(dtype=5), UNSUPPORTED),
    (dict(beams=65), UNSUPPORTED), (dict(best=65), UNSUPPORTED), (dict(vocab=524289, stride=524289), UNSUPPORTED),
    (dict(n_seqs=1 << 25, beams=64), UNSUPPORTED), (dict(stride=99), SHAPE), (dict(logits=None), ARG), (dict(scores=None), ARG),
    (dict(so=None), ARG), (dict(po=None), ARG), (dict(to=None), ARG), (dict(logits=ODD), ALIGN), (dict(scores=ODD), ALIGN),
    (dict(to=ODD), ALIGN), (dict(so=A), ARG),
])
def test_select_refusals(lib, kw, code):
    assert _select(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(n_seqs=-1), ARG), (dict(n_slots=-1), ARG), (dict(layers=-1), ARG), (dict(row_bytes=-16), ARG), (dict(beams=0), ARG),
    (dict(beams=65), UNSUPPORTED), (dict(n_seqs=1 << 26, beams=64), UNSUPPORTED), (dict(layers=65536), UNSUPPORTED),
    (dict(row_bytes=1 << 33, slot_stride=1 << 33), UNSUPPORTED), (dict(row_bytes=24), ALIGN), (dict(slot_stride=72), ALIGN),
    (dict(slot_stride=48), SHAPE), (dict(layers=2, layer_stride=48), SHAPE), (dict(slots=None), ARG), (dict(parents=None), ARG),
    (dict(out=None), ARG), (dict(pool=None), ARG), (dict(pool=MIS), ALIGN), (dict(slots=ODD), ALIGN), (dict(out=A), ARG),
])
def test_reorder_refusals(lib, kw, code):
    assert _reorder(lib, **kw) == code


def test_nothing_to_do(lib):
    assert _attn(lib, _dims(n_seqs=0, total_tokens=0), q=None, k=None, v=None, table=None, lens=None, O=None) == 0
    assert _append(lib, _dims(total_tokens=0), q=None, k=None, v=None, table=None, lens=None, kp=None, vp=None, q_out=None) == 0
    assert _select(lib, n_seqs=0, logits=None, scores=None) == 0
    assert _reorder(lib, n_seqs=0, slots=None, parents=None) == 0


def test_binding_refuses_before_the_library():
    t = torch.zeros(4, 2, 64)
    pages, table, lens = torch.zeros(3, 16, 2, 64), torch.zeros(4, 3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    for call in (lambda: api.gdn_paged_attn(t, pages, pages, table, lens), lambda: api.gdn_kv_append(t, t, pages, pages, table, lens),
                 lambda: api.gdn_beam_select(torch.zeros(2, 3, 5), torch.zeros(2, 3)),
                 lambda: api.gdn_beam_reorder(torch.zeros(8, 4), table[:, :2], table[:, :2]),
                 lambda: api.gdn_paged_attn(t.half(), pages.half(), pages.half(), table, lens),
                 lambda: api.gdn_paged_attn(t, pages[0], pages[0], table, lens),
                 lambda: api.gdn_paged_attn(t, pages[..., :32], pages[..., :32], table, lens),
                 lambda: api.gdn_paged_attn(t, pages, pages, table, lens, window=2**31),
                 lambda: api.gdn_beam_select(torch.zeros(2, 5), torch.zeros(2))):
        with pytest.raises(ValueError):
            call()
