"""Refusals of pa_decode_shared, through the C ABI and the binding: no GPU is touched."""
import ctypes

import pytest
import torch

import paged_kv_cache_107_gb300 as pk
from paged_kv_cache_107_gb300 import build as lib_build


@pytest.fixture(scope="module")
def lib():
    return ctypes.CDLL(lib_build.build())


def call(lib, B=4, groups=2, H=16, Hk=8, D=128, dtype=1, starts=16, prefix=16):
    vp = ctypes.c_void_p(16)
    return lib.pa_decode_shared(vp, vp, vp, vp, vp, 4, vp, ctypes.c_void_p(starts),
                                ctypes.c_void_p(prefix), B, groups, H, Hk, D, dtype, 16,
                                ctypes.c_int64(4), ctypes.c_float(0), vp,
                                ctypes.c_size_t(1 << 30), None, None)


def test_c_refusals(lib):
    assert call(lib, groups=0) == 2 and call(lib, groups=-1) == 2
    assert call(lib, groups=5) == 2
    assert call(lib, B=-1) == 2
    assert call(lib, B=8193, groups=1) == 3
    assert call(lib, starts=None) == 1 and call(lib, prefix=None) == 1
    assert call(lib, H=12) == 2
    assert call(lib, H=72) == 3
    assert call(lib, D=96) == 3
    assert call(lib, dtype=0) == 3
    assert call(lib, B=0, groups=0) == 0


def test_workspace_size_of_invalid_sizes(lib):
    fn = lib.pa_decode_shared_workspace_size
    fn.restype = ctypes.c_size_t
    assert fn(-1, 16, 8, 128) == 0 and fn(4, 16, 8, 96) == 0 and fn(4, 0, 8, 128) == 0


def test_binding_refuses_host_tensors():
    q = torch.zeros(2, 16, 128, dtype=torch.bfloat16)
    kc = torch.zeros(2, 16, 8, 128, dtype=torch.bfloat16)
    i32 = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(pk.PagedAttentionError, match="CUDA"):
        pk.pa_decode_shared(q, q, kc, kc, i32.view(2, 1), i32, i32, i32[:1])
