"""Sizes that the serving calls refuse on the host (CPU tests: every call below fails its checks)."""
import ctypes

import pytest
import torch

from gated_deltanet_state_chunked_gb300 import _lib, api

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


def test_binding_refuses_what_32_bits_cut_off(lib):
    """2^32 + 4 tokens are not four of them (tensors without storage)."""
    far = 2**32 + 4

    def empty(*shape, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device="meta")

    k, g = empty(far, 1, 8), empty(far, 1, dtype=torch.float32)
    with pytest.raises(ValueError, match="32 bits"):
        api.gdn_linear_attn(k, k, k, g[0], empty(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="32 bits"):
        api.gdn_decode(k, k, k, g, g, empty(1, 1, 8, 8, dtype=torch.float32))
    with pytest.raises(ValueError, match="32 bits"):
        api.gdn_verify_draft(empty(1, 1, far), empty(1, 0, dtype=torch.int32), empty(1, 1, dtype=torch.float32))
