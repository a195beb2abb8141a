"""GPU test: the library in a second driver context of the same device (in a child process, by the
driver's API alone).  What a call looks up on the host belongs to the context it runs in."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu

CHILD = r"""
import ctypes, struct, sys
from gated_deltanet_state_chunked_gb300 import _lib

lib = _lib.load(build=True)
cu = ctypes.CDLL("libcuda.so.1")


def ok(rc):
    assert rc == 0, rc


def device(data):
    p = ctypes.c_uint64()
    ok(cu.cuMemAlloc_v2(ctypes.byref(p), ctypes.c_size_t(len(data))))
    ok(cu.cuMemcpyHtoD_v2(p, data, ctypes.c_size_t(len(data))))
    return ctypes.c_void_p(p.value)


def host(p, n):
    out = ctypes.create_string_buffer(n)
    ok(cu.cuMemcpyDtoH_v2(out, ctypes.c_uint64(p.value), ctypes.c_size_t(n)))
    return out.raw


def bad_draft_length():
    # one request of five drafts where a call has room for two: skipped, and reported
    dims = _lib.GdnVerifyDims(1, 2, 8, _lib.GDN_F32, 8, 8)
    target, ints, floats = device(struct.pack("24f", *[0.125] * 24)), device(struct.pack("4i", 0, 0, 5, 0)), device(bytes(16))
    out = device(struct.pack("4i", 7, 7, 7, 7))
    ok(lib.gdn_verify_draft(ctypes.byref(dims), target, None, ints, ctypes.c_void_p(ints.value + 8), floats, out,
                            ctypes.c_void_p(out.value + 4), None))
    assert lib.gdn_get_status(None) == _lib.GDN_ERR_SHAPE
    assert lib.gdn_get_status(None) == 0
    assert host(out, 16) == struct.pack("4i", 7, 7, 7, 7)


def prompt_of_one_token():
    # S = v k^T and o = (k.q) v, whole numbers in bf16
    d = 64
    dims = _lib.GdnDims(1, 1, 1, 1, d, d, _lib.GDN_BF16, 0, 1.0)
    q, k, v = (device(struct.pack("H", bits) * d) for bits in (0x3F80, 0x3F00, 0x4000))  # 1, 1/2 and 2
    O, S = device(bytes(2 * d)), device(bytes(4 * d * d))
    ok(lib.gdn_linear_attn(ctypes.byref(dims), q, k, v, device(bytes(4)), device(struct.pack("2i", 0, 1)), None, O, S, None))
    ok(lib.gdn_get_status(None))
    assert host(S, 4 * d * d) == struct.pack("f", 1.0) * (d * d)
    assert host(O, 2 * d) == struct.pack("H", 0x4280) * d  # 64


CALLS = [bad_draft_length, prompt_of_one_token]


def main():
    ok(cu.cuInit(0))
    first, second = ctypes.c_void_p(), ctypes.c_void_p()
    ok(cu.cuDevicePrimaryCtxRetain(ctypes.byref(first), 0))
    ok(cu.cuCtxSetCurrent(first))
    for call in CALLS:
        call()
    ok(cu.cuCtxCreate_v2(ctypes.byref(second), 0, 0))
    for call in CALLS:
        call()
    ok(cu.cuCtxSetCurrent(first))
    for call in CALLS:
        call()
    print("both contexts")


main()
"""


def test_second_context():
    run = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and "both contexts" in run.stdout, run.stdout[-2000:] + run.stderr[-2000:]
