"""Python binding of libgdn.so: same names as the C ABI, argument marshalling only.

PyTorch supplies device memory and streams; every step of the computation
runs in the library's CUDA kernels.  There is no CPU fallback: these
functions raise when the library is missing or a tensor is not on a CUDA
device.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib

_DTYPE = {torch.float32: _lib.GDN_F32, torch.bfloat16: _lib.GDN_BF16}


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_handle(stream, device):
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def _need_cuda(name, t, dtype=None, shape=None):
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def gdn_replay(q, k, v, g, beta, cu_seqlens, S0=None, *, O_out=None, S_out=None, l2norm_qk=True,
               scale=1.0, state_only=False, precise=False, scalar_decay=False, stream=None):
    """Rebuild the recurrent state of each packed replay tail (see gdn.h).

    q, k: [T, h_k, d_k]; v: [T, h_v, d_v] (all bf16 or all fp32); g, beta: fp32
    [T, h_v]; cu_seqlens: int32 [n + 1] on the device; S0: fp32 [n, h_v, d_v, d_k]
    or None.  Returns (O, S): O [T, h_v, d_v] in the input dtype (None when
    ``state_only``) and S fp32 [n, h_v, d_v, d_k]."""
    lib = _lib.load()
    T, h_k, d_k = k.shape
    h_v, d_v = v.shape[1], v.shape[2]
    n = cu_seqlens.shape[0] - 1
    dt = q.dtype
    if dt not in _DTYPE:
        raise ValueError(f"unsupported dtype {dt}")
    _need_cuda("q", q, dt, (T, h_k, d_k))
    _need_cuda("k", k, dt)
    _need_cuda("v", v, dt, (T, h_v, d_v))
    _need_cuda("g", g, torch.float32, (T, h_v))
    _need_cuda("beta", beta, torch.float32, (T, h_v))
    _need_cuda("cu_seqlens", cu_seqlens, torch.int32)
    _need_cuda("S0", S0, torch.float32, (n, h_v, d_v, d_k))
    if S_out is None:
        S_out = torch.empty((n, h_v, d_v, d_k), dtype=torch.float32, device=k.device)
    _need_cuda("S_out", S_out, torch.float32, (n, h_v, d_v, d_k))
    if not state_only:
        if O_out is None:
            O_out = torch.empty((T, h_v, d_v), dtype=dt, device=k.device)
        _need_cuda("O_out", O_out, dt, (T, h_v, d_v))
    else:
        O_out = None
    flags = (_lib.GDN_QK_L2NORM if l2norm_qk else 0) | (_lib.GDN_STATE_ONLY if state_only else 0) \
        | (_lib.GDN_PRECISE if precise else 0) | (_lib.GDN_SCALAR_DECAY if scalar_decay else 0)
    dims = _lib.GdnDims(n, T, h_k, h_v, d_k, d_v, _DTYPE[dt], flags, float(scale))
    rc = lib.gdn_replay(ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(cu_seqlens),
                        _ptr(S0), _ptr(O_out), _ptr(S_out), _stream_handle(stream, k.device))
    _lib.check(rc, "gdn_replay")
    return O_out, S_out


def gdn_replay_noalloc(q, k, v, g, beta, cu_seqlens, S0, O_out, S_out, *, l2norm_qk=True, scale=1.0,
                       state_only=False, precise=False, scalar_decay=False, stream=None):
    """gdn_replay for callers that cannot allocate device memory at call time.

    Same arguments and results as gdn_replay, except that the outputs O_out
    (None with ``state_only``) and S_out must be passed in: neither this
    wrapper nor the library allocates anything.  The library's scratch is a
    96 MiB static device array shared by all calls, so calls that overlap on
    the GPU race; larger problems raise GdnError(GDN_ERR_NOMEM)."""
    lib = _lib.load()
    T, h_k, d_k = k.shape
    h_v, d_v = v.shape[1], v.shape[2]
    n = cu_seqlens.shape[0] - 1
    dt = q.dtype
    if dt not in _DTYPE:
        raise ValueError(f"unsupported dtype {dt}")
    _need_cuda("q", q, dt, (T, h_k, d_k))
    _need_cuda("k", k, dt)
    _need_cuda("v", v, dt, (T, h_v, d_v))
    _need_cuda("g", g, torch.float32, (T, h_v))
    _need_cuda("beta", beta, torch.float32, (T, h_v))
    _need_cuda("cu_seqlens", cu_seqlens, torch.int32)
    _need_cuda("S0", S0, torch.float32, (n, h_v, d_v, d_k))
    if S_out is None or (O_out is None and not state_only):
        raise ValueError("gdn_replay_noalloc needs caller-provided outputs")
    _need_cuda("S_out", S_out, torch.float32, (n, h_v, d_v, d_k))
    if not state_only:
        _need_cuda("O_out", O_out, dt, (T, h_v, d_v))
    else:
        O_out = None
    flags = (_lib.GDN_QK_L2NORM if l2norm_qk else 0) | (_lib.GDN_STATE_ONLY if state_only else 0) \
        | (_lib.GDN_PRECISE if precise else 0) | (_lib.GDN_SCALAR_DECAY if scalar_decay else 0)
    dims = _lib.GdnDims(n, T, h_k, h_v, d_k, d_v, _DTYPE[dt], flags, float(scale))
    rc = lib.gdn_replay_noalloc(ctypes.byref(dims), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                _ptr(cu_seqlens), _ptr(S0), _ptr(O_out), _ptr(S_out), _stream_handle(stream, k.device))
    _lib.check(rc, "gdn_replay_noalloc")
    return O_out, S_out


def gdn_chunk_operator(k, g, beta, v, cu_seqlens=None, *, T_out=None, Slocal_out=None, l2norm_qk=True,
                       scalar_decay=False, stream=None):
    """(T_C, S_local) of each chunk (range of cu_seqlens, or all tokens when None).
    ``scalar_decay``: the scalar-transition family (T_C is then a scaled identity).
    Returns T fp32 [n, h_v, d_k, d_k] and S_local fp32 [n, h_v, d_v, d_k]."""
    lib = _lib.load()
    T, h_k, d_k = k.shape
    h_v, d_v = v.shape[1], v.shape[2]
    n = 1 if cu_seqlens is None else cu_seqlens.shape[0] - 1
    dt = k.dtype
    if dt not in _DTYPE:
        raise ValueError(f"unsupported dtype {dt}")
    _need_cuda("k", k, dt)
    _need_cuda("v", v, dt, (T, h_v, d_v))
    _need_cuda("g", g, torch.float32, (T, h_v))
    _need_cuda("beta", beta, torch.float32, (T, h_v))
    _need_cuda("cu_seqlens", cu_seqlens, torch.int32)
    if T_out is None:
        T_out = torch.empty((n, h_v, d_k, d_k), dtype=torch.float32, device=k.device)
    if Slocal_out is None:
        Slocal_out = torch.empty((n, h_v, d_v, d_k), dtype=torch.float32, device=k.device)
    _need_cuda("T_out", T_out, torch.float32, (n, h_v, d_k, d_k))
    _need_cuda("Slocal_out", Slocal_out, torch.float32, (n, h_v, d_v, d_k))
    flags = (_lib.GDN_QK_L2NORM if l2norm_qk else 0) | (_lib.GDN_SCALAR_DECAY if scalar_decay else 0)
    dims = _lib.GdnDims(n, T, h_k, h_v, d_k, d_v, _DTYPE[dt], flags, 1.0)
    rc = lib.gdn_chunk_operator(ctypes.byref(dims), _ptr(k), _ptr(g), _ptr(beta), _ptr(v), _ptr(cu_seqlens),
                                _ptr(T_out), _ptr(Slocal_out), _stream_handle(stream, k.device))
    _lib.check(rc, "gdn_chunk_operator")
    return T_out, Slocal_out


def gdn_compose(T_list, Slocal_list, S_in=None, *, S_out=None, stream=None):
    """S <- S T_j^T + S_local_j for j = 1..K.  T_list[j]: fp32 [h, d_k, d_k];
    Slocal_list[j]: fp32 [h, d_v, d_k]; S_in: [h, d_v, d_k] or None."""
    lib = _lib.load()
    K = len(T_list)
    if len(Slocal_list) != K:
        raise ValueError("T_list and Slocal_list differ in length")
    ref = Slocal_list[0] if K else S_in
    if ref is None:
        raise ValueError("need at least one chunk or an entering state")
    h, d_v, d_k = ref.shape
    for j in range(K):
        _need_cuda(f"T[{j}]", T_list[j], torch.float32, (h, d_k, d_k))
        _need_cuda(f"Slocal[{j}]", Slocal_list[j], torch.float32, (h, d_v, d_k))
    _need_cuda("S_in", S_in, torch.float32, (h, d_v, d_k))
    if S_out is None:
        S_out = torch.empty((h, d_v, d_k), dtype=torch.float32, device=ref.device)
    _need_cuda("S_out", S_out, torch.float32, (h, d_v, d_k))
    Tp = (ctypes.c_void_p * max(K, 1))(*[t.data_ptr() for t in T_list])
    Sp = (ctypes.c_void_p * max(K, 1))(*[s.data_ptr() for s in Slocal_list])
    dims = _lib.GdnDims(1, 0, h, h, d_k, d_v, _lib.GDN_F32, 0, 1.0)
    rc = lib.gdn_compose(ctypes.byref(dims), K, ctypes.cast(Tp, ctypes.c_void_p), ctypes.cast(Sp, ctypes.c_void_p),
                         _ptr(S_in), _ptr(S_out), _stream_handle(stream, ref.device))
    _lib.check(rc, "gdn_compose")
    return S_out


# The serving calls below run once per layer and token, so their checks and launches are kept to a few
# microseconds: one comparison per tensor (the message is made only when it fails), no context manager
# on the current device and stream, pointers as plain integers.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _want(name, t, device, dtype, shape):
    """data_ptr of t, a contiguous tensor of this shape and dtype on CUDA device ``device`` (None for None)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device or not t.is_contiguous():
        _need_cuda(name, t, dtype, shape)
        raise ValueError(f"{name} is on {t.device}, the other tensors on cuda:{device}")
    return t.data_ptr()


def _fits(*sizes):
    """The C structures hold 32 bits, and what is more would be cut off without a word."""
    if max(sizes) > 0x7fffffff:
        raise ValueError(f"a size of {max(sizes)} does not fit in 32 bits")


def _cuda_index(name, t):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.get_device()


def _launch(call, where, ref, stream, outputs, *args):
    """Allocate the missing outputs, given as (shape, dtype), and make the C call on the device of the
    tensor ``ref`` and on ``stream`` (None: the current one).  What is allocated here belongs to the
    stream that the kernels run on.  Returns the outputs."""
    device = ref.get_device()
    if stream is not None:
        if stream.device.index != device:
            raise ValueError(f"stream belongs to {stream.device}, the tensors to cuda:{device}")
        if stream != torch.cuda.current_stream(device) or torch.cuda.current_device() != device:
            with torch.cuda.stream(stream):
                return _launch(call, where, ref, None, outputs, *args)
    elif _current_device() != device:
        with torch.cuda.device(device):
            return _launch(call, where, ref, None, outputs, *args)
    made = [torch.empty(t[0], dtype=t[1], device=ref.device) if type(t) is tuple else t for t in outputs]
    rc = call(*args, *[None if t is None else t.data_ptr() for t in made], _raw_stream(device))
    if rc != _lib.GDN_OK:
        _lib.check(rc, where)
    return made


def gdn_linear_attn(q, k, v, log_decay, cu_seqlens, S0=None, *, O_out=None, S_out=None, scale=1.0,
                    state_only=False, stream=None):
    """Linear attention with a decay for each head over packed prompts (see gdn.h):
    S_t = exp(log_decay[h]) S_{t-1} + v_t k_t^T, o_t = S_t (scale q_t).

    q, k: [T, h_k, d_k]; v: [T, h_v, d_v] (all bf16 or all fp32; q may be None with
    ``state_only``); log_decay: fp32 [h_v]; cu_seqlens: int32 [n + 1] on the device; S0: fp32
    [n, h_v, d_v, d_k] or None.  Returns (O, S) as gdn_replay does;
    bf16 outputs are off by 2.4e-3 of their norm (widened inputs: 3e-7)."""
    lib = _lib.load()
    T, h_k, d_k = k.shape
    h_v, d_v = v.shape[1], v.shape[2]
    n = cu_seqlens.shape[0] - 1
    dt = k.dtype
    if dt not in _DTYPE:
        raise ValueError(f"unsupported dtype {dt}")
    if q is None and not state_only:
        raise ValueError("q may be None only with state_only")
    _fits(n, T, h_k, h_v, d_k, d_v)
    dev = _cuda_index("k", k)
    qk, vo, state = (T, h_k, d_k), (T, h_v, d_v), (n, h_v, d_v, d_k)
    args = (_want("q", q, dev, dt, qk), _want("k", k, dev, dt, qk), _want("v", v, dev, dt, vo),
            _want("log_decay", log_decay, dev, torch.float32, (h_v,)),
            _want("cu_seqlens", cu_seqlens, dev, torch.int32, (n + 1,)), _want("S0", S0, dev, torch.float32, state))
    _want("O_out", O_out, dev, dt, vo)
    _want("S_out", S_out, dev, torch.float32, state)
    dims = _lib.GdnDims(n, T, h_k, h_v, d_k, d_v, _DTYPE[dt], _lib.GDN_STATE_ONLY if state_only else 0, scale)
    O, S = _launch(lib.gdn_linear_attn, "gdn_linear_attn", k, stream,
                   (None if state_only else (vo, dt) if O_out is None else O_out,
                    (state, torch.float32) if S_out is None else S_out), dims, *args)
    return O, S


def gdn_decode(q, k, v, g, beta, S_pool, slots=None, *, counts=None, O_out=None, l2norm_qk=True, scale=1.0,
               state_only=False, keep_state=False, scalar_decay=False, head_decay=False, stream=None):
    """One token, or a window of tokens, for each request on its state in ``S_pool`` (see gdn.h).

    q, k: [n * window, h_k, d_k]; v: [n * window, h_v, d_v], request after request (all bf16 or
    all fp32; q may be None with ``state_only``); g, beta: fp32 [n * window, h_v] (``head_decay``:
    g is the log decay [h_v] and beta None); S_pool: fp32 [n_slots, h_v, d_v, d_k], updated in
    place unless ``keep_state``; slots: int32 [n] on the device (negative: padding) or None, then
    n = n_slots; counts: int32 [n] on the device, the tokens of each window that count, or None.
    Returns O [n * window, h_v, d_v] in the input dtype, None with ``state_only``.  Rows that do
    not count are left as they were (undefined when O is allocated here)."""
    lib = _lib.load()
    T, h_k, d_k = k.shape
    h_v, d_v = v.shape[1], v.shape[2]
    n_slots = S_pool.shape[0]
    n = n_slots if slots is None else slots.shape[0]
    dt = k.dtype
    if dt not in _DTYPE:
        raise ValueError(f"unsupported dtype {dt}")
    if q is None and not state_only:
        raise ValueError("q may be None only with state_only")
    if n == 0 and T:
        raise ValueError(f"{T} tokens of no requests")
    _fits(n, n_slots, T, h_k, h_v, d_k, d_v)
    dev = _cuda_index("k", k)
    qk, vo, per = (T, h_k, d_k), (T, h_v, d_v), (T, h_v)
    args = (n_slots, _want("q", q, dev, dt, qk), _want("k", k, dev, dt, qk), _want("v", v, dev, dt, vo),
            _want("g", g, dev, torch.float32, (h_v,) if head_decay else per),
            _want("beta", beta, dev, torch.float32, per), _want("slots", slots, dev, torch.int32, (n,)),
            _want("counts", counts, dev, torch.int32, (n,)),
            _want("S_pool", S_pool, dev, torch.float32, (n_slots, h_v, d_v, d_k)))
    _want("O_out", O_out, dev, dt, vo)
    flags = (_lib.GDN_QK_L2NORM if l2norm_qk else 0) | (_lib.GDN_STATE_ONLY if state_only else 0) \
        | (_lib.GDN_SCALAR_DECAY if scalar_decay else 0) | (_lib.GDN_HEAD_DECAY if head_decay else 0) \
        | (_lib.GDN_KEEP_STATE if keep_state else 0)
    dims = _lib.GdnDims(n, T, h_k, h_v, d_k, d_v, _DTYPE[dt], flags, scale)
    return _launch(lib.gdn_decode, "gdn_decode", k, stream,
                   (None if state_only else (vo, dt) if O_out is None else O_out,), dims, *args)[0]


def _prob_rows(name, t, shape):
    """Element stride between the rows of probabilities t [n, rows, vocab] (a vocabulary slice of
    padded rows will do; the rows must be evenly spaced)."""
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.is_contiguous():
        return shape[2]
    n, rows, _ = shape
    step = t.stride(1) if rows > 1 else t.stride(0)
    if t.stride(2) != 1 or (n > 1 and t.stride(0) != rows * step):
        raise ValueError(f"{name} must have evenly spaced rows of consecutive entries")
    return step


def gdn_verify_draft(target, drafted, uniforms, draft=None, draft_lens=None, *, counts_out=None, tokens_out=None,
                     stream=None):
    """Drafted tokens against the target's probabilities, from given random numbers (see gdn.h).

    target: [n, n_draft + 1, vocab] fp32 or bf16; draft: [n, n_draft, vocab] of the same dtype, or
    None when the drafts were chosen outright; drafted: int32 [n, n_draft]; uniforms: fp32
    [n, n_draft + 1] in [0, 1); draft_lens: int32 [n] (negative: padding) or None.
    Returns (counts, tokens): counts int32 [n], the emitted tokens of each request (accepted
    drafts + 1), and tokens int32 [n, n_draft + 1], those tokens followed by -1."""
    lib = _lib.load()
    n, n_draft = drafted.shape
    if target.dim() != 3:
        raise ValueError("target must be [n, n_draft + 1, vocab]")
    vocab = target.shape[2]
    dt = target.dtype
    if dt not in _DTYPE:
        raise ValueError(f"unsupported dtype {dt}")
    _fits(n, n_draft, vocab)
    dev = _cuda_index("target", target)
    target_stride = _prob_rows("target", target, (n, n_draft + 1, vocab))
    draft_stride, draft_ptr = 0, None
    if draft is not None:
        if draft.dtype is not dt or draft.get_device() != dev:
            raise ValueError(f"draft must be {dt} on cuda:{dev}, got {draft.dtype} on {draft.device}")
        draft_stride, draft_ptr = _prob_rows("draft", draft, (n, n_draft, vocab)), draft.data_ptr()
    i32, emitted = torch.int32, (n, n_draft + 1)
    args = (target.data_ptr(), draft_ptr, _want("drafted", drafted, dev, i32, (n, n_draft)),
            _want("draft_lens", draft_lens, dev, i32, (n,)), _want("uniforms", uniforms, dev, torch.float32, emitted))
    _want("counts_out", counts_out, dev, i32, (n,))
    _want("tokens_out", tokens_out, dev, i32, emitted)
    dims = _lib.GdnVerifyDims(n, n_draft, vocab, _DTYPE[dt], target_stride, draft_stride)
    counts, tokens = _launch(lib.gdn_verify_draft, "gdn_verify_draft", target, stream,
                             (((n,), i32) if counts_out is None else counts_out,
                              (emitted, i32) if tokens_out is None else tokens_out), dims, *args)
    return counts, tokens


def _placed(name, t, device, dtype, shape):
    """Raise for what _want refuses, strides apart."""
    _need_cuda(name, t[:0], dtype)
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name} is on {t.device}, the other tensors on cuda:{device}")


def _token_rows(name, t, device, dtype, shape):
    """(data_ptr, elements between tokens) of t [T, h, d]: a token's heads lie one after another, the
    tokens may be apart (a slice of a projection's rows)."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device:
        _placed(name, t, device, dtype, shape)
    T, h, d = shape
    step, head, one = t.stride()
    if (one != 1 and d > 1 or head != d and h > 1) and t.numel():
        raise ValueError(f"{name}: a token's heads must lie one after another")
    return t.data_ptr(), step if T > 1 else h * d


def _page_strides(name, t, device, dtype, shape):
    """Elements between the pages, tokens and heads of t [n_pages, page_size, h_kv, d] (0 where there is one)."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device:
        _placed(name, t, device, dtype, shape)
    page, token, head, one = t.stride()
    if one != 1 and shape[3] > 1:
        raise ValueError(f"{name}: the values of a head must lie one after another")
    return page if shape[0] > 1 else 0, token if shape[1] > 1 else 0, head if shape[2] > 1 else 0


def _paged(T, h_q, k_pages, v_pages, page_table, kv_lens, cu_seqlens, max_q, d, window=0, scale=0.0):
    """The parts that gdn_kv_append and gdn_paged_attn share: GdnPagedDims without the tokens' strides, and the
    pointers of page_table, kv_lens and cu_seqlens."""
    dt = k_pages.dtype
    code = _DTYPE.get(dt)
    if code is None:
        raise ValueError(f"unsupported dtype {dt}")
    if k_pages.dim() != 4:
        raise ValueError("k_pages must be [n_pages, page_size, h_kv, d]")
    if page_table.dim() != 2:
        raise ValueError("page_table must be [n, table_width]")
    shape = k_pages.shape
    n_pages, page, h_kv, d_pages = shape
    if d_pages != d:
        raise ValueError(f"heads of {d} values, the pages have heads of {d_pages}")
    n, width = page_table.shape
    if n == 0 and T:
        raise ValueError(f"{T} tokens of no requests")
    if max_q is None:
        max_q = T if cu_seqlens is not None else T // n if n else 0
    _fits(n, T, max_q, h_q, h_kv, d, page, n_pages, width, window)
    dev = _cuda_index("k_pages", k_pages)
    i32 = torch.int32
    if page_table.dtype is not i32 or page_table.get_device() != dev:
        _placed("page_table", page_table, dev, i32, (n, width))
    step, one = page_table.stride()  # (rows of a wider table will do)
    if one != 1 and width > 1:
        raise ValueError("page_table: a request's pages must lie one after another")
    dims = _lib.GdnPagedDims(n, T, max_q or 1, h_q, h_kv, d, page, n_pages, width, code, window, scale,
                             step if n > 1 else width, 0, 0, 0, *_page_strides("k_pages", k_pages, dev, dt, shape),
                             *_page_strides("v_pages", v_pages, dev, dt, shape))
    return dims, page_table.data_ptr(), _want("kv_lens", kv_lens, dev, i32, (n,)), \
        _want("cu_seqlens", cu_seqlens, dev, i32, (n + 1,)), dev, dt


def gdn_kv_append(k, v, k_pages, v_pages, page_table, kv_lens, cu_seqlens=None, *, q=None, q_out=None, inv_freq=None,
                  positions=None, sections=None, neighbours=False, max_q=None, stream=None):
    """New keys and values into a paged cache, keys (and queries) rotated by their positions (see gdn.h).

    k, v: [T, h_kv, d], bf16 or fp32, tokens packed request after request (a slice of wider rows will do);
    k_pages, v_pages: [n_pages, page_size, h_kv, d] of the same dtype, any strides (of multiples of 16 bytes) with the
    values of a head together, written in place; page_table: int32 [n, width]; kv_lens: int32 [n] on the device, the
    tokens in the cache with the new ones (negative: padding); cu_seqlens: int32 [n + 1] on the device, or None: T / n
    new tokens each.  inv_freq: fp32 [rotary_dim / 2] or None (no rotation); positions: int32 [T] or [axes, T], or None
    (the place in the cache); sections: pairs that turn by each axis; neighbours: pairs are values 2i and 2i + 1 instead
    of i and i + rotary_dim / 2; max_q: the most new tokens of a request, where it is known.
    Returns the rotated queries [T, h_q, d], None without q."""
    lib = _lib.load()
    T, h_kv, d = k.shape
    h_q = h_kv if q is None else q.shape[1]
    dims, table, lens, cu, dev, dt = _paged(T, h_q, k_pages, v_pages, page_table, kv_lens, cu_seqlens, max_q, d)
    if k_pages.shape[2] != h_kv:
        raise ValueError(f"k has {h_kv} heads, the pages {k_pages.shape[2]}")
    k_ptr, dims.k_stride = _token_rows("k", k, dev, dt, (T, h_kv, d))
    v_ptr, dims.v_stride = _token_rows("v", v, dev, dt, (T, h_kv, d))
    q_ptr, rotary, freq_ptr, pos_ptr = None, None, None, None
    if q is not None:
        q_ptr, dims.q_stride = _token_rows("q", q, dev, dt, (T, h_q, d))
        _want("q_out", q_out, dev, dt, (T, h_q, d))
    elif q_out is not None:
        raise ValueError("q_out without q")
    if inv_freq is not None:
        axes = 1 if positions is None or positions.dim() == 1 else positions.shape[0]
        if axes > 1 and (sections is None or len(sections) != axes):
            raise ValueError(f"{axes} axes of positions, sections {sections}")
        if axes > _lib.GDN_MAX_AXES:
            raise ValueError(f"at most {_lib.GDN_MAX_AXES} axes of positions, got {axes}")
        freq_ptr = _want("inv_freq", inv_freq, dev, torch.float32, (inv_freq.shape[0],))
        if positions is not None:
            pos_ptr = _want("positions", positions, dev, torch.int32, (T,) if positions.dim() == 1 else (axes, T))
        rotary = _lib.GdnRotary(2 * inv_freq.shape[0], 1 if neighbours else 0, axes)
        if axes > 1:
            _fits(*sections)
            rotary.sections[:axes] = sections
    elif positions is not None or sections is not None:
        raise ValueError("positions and sections need inv_freq")
    return _launch(lib.gdn_kv_append, "gdn_kv_append", k_pages, stream,
                   (None if q is None else ((T, h_q, d), dt) if q_out is None else q_out,), dims, rotary, q_ptr, k_ptr,
                   v_ptr, freq_ptr, pos_ptr, table, lens, cu, k_pages.data_ptr(), v_pages.data_ptr())[0]


def gdn_paged_attn(q, k_pages, v_pages, page_table, kv_lens, cu_seqlens=None, *, max_q=None, scale=None, window=0,
                   O_out=None, lse_out=None, stream=None):
    """Attention of each request's new tokens over its paged cache (see gdn.h): causal, the new tokens the
    last ones of the cache; with ``window`` > 0 a token sees the last ``window`` tokens, itself among them.

    q: [T, h_q, d], bf16 or fp32, tokens packed request after request; k_pages, v_pages, page_table, kv_lens,
    cu_seqlens: as in gdn_kv_append; max_q: the most new tokens of a request (None: T with cu_seqlens, T / n
    without; a close bound chooses the kernel for short windows); scale: None for d ** -0.5; lse_out: fp32 [T, h_q],
    receives the log of each row's sum of exponentials.  Returns O [T, h_q, d] in the input dtype; rows of padding
    and outside every range are left as they were (undefined when O is allocated here)."""
    lib = _lib.load()
    T, h_q, d = q.shape
    dims, table, lens, cu, dev, dt = _paged(T, h_q, k_pages, v_pages, page_table, kv_lens, cu_seqlens, max_q, d, window,
                                            d ** -0.5 if scale is None else scale)
    q_ptr, dims.q_stride = _token_rows("q", q, dev, dt, (T, h_q, d))
    _want("O_out", O_out, dev, dt, (T, h_q, d))
    _want("lse_out", lse_out, dev, torch.float32, (T, h_q))
    return _launch(lib.gdn_paged_attn, "gdn_paged_attn", q, stream,
                   (((T, h_q, d), dt) if O_out is None else O_out, lse_out), dims, q_ptr, k_pages.data_ptr(),
                   v_pages.data_ptr(), table, lens, cu)[0]


def gdn_beam_select(logits, scores, best=None, *, scores_out=None, parents_out=None, tokens_out=None, stream=None):
    """The ``best`` (None: as many as beams) continuations of each request over its beams and the vocabulary (see
    gdn.h): the largest scores + log softmax(logits); of equal ones the lower beam's, then the lower token.

    logits: [n, beams, vocab] fp32 or bf16 (evenly spaced rows; a vocabulary slice of padded rows will do); scores:
    fp32 [n, beams], -inf for a dead beam.  Returns (scores, parents, tokens), [n, best] fp32, int32, int32, largest
    first; -inf, -1, -1 where there are fewer continuations."""
    lib = _lib.load()
    if logits.dim() != 3:
        raise ValueError("logits must be [n, beams, vocab]")
    n, beams, vocab = logits.shape
    dt = logits.dtype
    if dt not in _DTYPE:
        raise ValueError(f"unsupported dtype {dt}")
    best = beams if best is None else best
    _fits(n, vocab, best)
    dev = _cuda_index("logits", logits)
    stride = _prob_rows("logits", logits, (n, beams, vocab))
    out, i32 = (n, best), torch.int32
    s_ptr = _want("scores", scores, dev, torch.float32, (n, beams))
    _want("scores_out", scores_out, dev, torch.float32, out)
    _want("parents_out", parents_out, dev, i32, out)
    _want("tokens_out", tokens_out, dev, i32, out)
    dims = _lib.GdnBeamDims(n, beams, best, vocab, _DTYPE[dt], stride)
    return tuple(_launch(lib.gdn_beam_select, "gdn_beam_select", logits, stream,
                         ((out, torch.float32) if scores_out is None else scores_out,
                          (out, i32) if parents_out is None else parents_out,
                          (out, i32) if tokens_out is None else tokens_out), dims, logits.data_ptr(), s_ptr))


def gdn_beam_reorder(pool, slots, parents, *, layers=False, slots_out=None, stream=None):
    """The rows of ``pool`` follow their beams, in place (see gdn.h): the first child of a beam keeps its parent's
    row, the others get copies in the rows of beams without children.

    pool: [n_slots, ...], or [n_layers, n_slots, ...] with ``layers`` (all layers move alike), any dtype, rows of a
    multiple of 16 bytes, each row contiguous; slots, parents: int32 [n, beams] on the device (a negative first slot:
    padding; a negative parent: the new beam continues none).  Returns the new beams' slots, int32 [n, beams] (-1 for
    padding)."""
    lib = _lib.load()
    lead = 2 if layers else 1
    if pool.dim() < lead or slots.dim() != 2:
        raise ValueError("pool must be [n_slots, ...] ([n_layers, n_slots, ...] with layers) and slots [n, beams]")
    n_layers, n_slots = pool.shape[:2] if layers else (1, pool.shape[0])
    n, beams = slots.shape
    _fits(n, beams, n_slots, n_layers)
    dev = _cuda_index("pool", pool)
    size = pool.element_size()
    if pool.is_contiguous():
        row = pool.numel() // (n_layers * n_slots) if n_layers * n_slots else 0
        slot_step, layer_step = row, row * n_slots
    else:
        row, steps = 1, pool.stride()
        for length, step in zip(reversed(pool.shape[lead:]), reversed(steps[lead:])):
            if length != 1 and step != row:
                raise ValueError("pool: each row must be contiguous")
            row *= length
        slot_step = steps[lead - 1] if n_slots > 1 else row
        layer_step = steps[0] if layers and n_layers > 1 else row
    i32 = torch.int32
    args = (_want("slots", slots, dev, i32, (n, beams)), _want("parents", parents, dev, i32, (n, beams)))
    _want("slots_out", slots_out, dev, i32, (n, beams))
    dims = _lib.GdnReorderDims(n, beams, n_slots, n_layers, row * size, slot_step * size, layer_step * size)
    return _launch(lib.gdn_beam_reorder, "gdn_beam_reorder", pool, stream,
                   (((n, beams), i32) if slots_out is None else slots_out,), dims, *args, pool.data_ptr())[0]


def gdn_get_status(stream=None, device=None):
    """Synchronise the stream; raise GdnError if the device recorded an error."""
    lib = _lib.load()
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    rc = lib.gdn_get_status(_stream_handle(stream, dev))
    _lib.check(rc, "gdn_get_status")


def gdn_workspace_bytes(n_seqs, total_tokens, h_k, h_v, d_k, d_v, dtype=torch.bfloat16, flags=0) -> int:
    lib = _lib.load()
    dims = _lib.GdnDims(n_seqs, total_tokens, h_k, h_v, d_k, d_v, _DTYPE[dtype], flags, 1.0)
    return int(lib.gdn_workspace_bytes(ctypes.byref(dims)))


def gdn_set_stage_event(event) -> None:
    """Have this thread's next tensor-core gdn_replay record ``event`` (a
    torch.cuda.Event) between its prep and scan kernels (measurement hook)."""
    lib = _lib.load()
    if event is not None and event.cuda_event == 0:
        raise ValueError("record-able torch.cuda.Event expected")
    lib.gdn_set_stage_event(ctypes.c_void_p(event.cuda_event if event is not None else 0))


def gdn_set_wait_limit_ns(ns: int) -> None:
    """Bound of the device-side waits of this thread's next gdn_compose call (test hook of the
    timeout path; 0 makes a wait give up unless its event has already happened)."""
    _lib.load().gdn_set_wait_limit_ns(int(ns))
