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
    elif torch.cuda.current_device() != device:
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
