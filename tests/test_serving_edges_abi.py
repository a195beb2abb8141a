"""Sizes that the serving calls refuse on the host (CPU tests: every call below fails its checks)."""
import ctypes

import pytest

from gated_deltanet_state_chunked_gb300 import _lib

A = ctypes.c_void_p(1 << 20)  # aligned fake address, never dereferenced
MOST = 2**31 - 1


@pytest.fixture(scope="module")
def lib():
    return _lib.load(build=True)


@pytest.mark.parametrize("tokens", [MOST, MOST - 64, MOST - 1022])
@pytest.mark.parametrize("dtype", [_lib.GDN_F32, _lib.GDN_BF16])
def test_more_tokens_than_32_bits_step_over(lib, tokens, dtype):
    """A chunk's end, or a window's, behind the last token would pass 2^31."""
    dims = _lib.GdnDims(1, tokens, 1, 1, 8, 8, dtype, _lib.GDN_STATE_ONLY, 1.0)
    assert lib.gdn_linear_attn(ctypes.byref(dims), None, A, A, A, A, None, None, A, None) == _lib.GDN_ERR_UNSUPPORTED
    assert lib.gdn_decode(ctypes.byref(dims), 1, None, A, A, A, A, None, None, A, None, None) == _lib.GDN_ERR_UNSUPPORTED


@pytest.mark.parametrize("n_draft", [MOST, MOST - 1022])
def test_more_drafts_than_32_bits_step_over(lib, n_draft):
    dims = _lib.GdnVerifyDims(2, n_draft, 1, _lib.GDN_BF16, 1, 1)
    assert lib.gdn_verify_draft(ctypes.byref(dims), A, None, A, None, A, A, A, None) == _lib.GDN_ERR_UNSUPPORTED
