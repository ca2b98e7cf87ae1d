"""Waits of pa_decode_q8 that run out: the launch returns with PA_DEV_ERR_TIMEOUT, writes nothing
but its own rows, and the next call on a zeroed workspace is correct.

As in test_timeout_gpu.py a second copy of the library is built with every wait limit at 2^17
cycles and the producers holding back the copies of a CTA's last key tile for 2^20 cycles; they
issue them late and wait for them, so nothing is left in flight."""
import ctypes

import pytest
import torch

import paged_kv_cache_107_gb300 as pk
from paged_kv_cache_107_gb300 import build as lib_build
from tests.test_decode_q8_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def timeout_lib(tmp_path_factory):
    path = str(tmp_path_factory.mktemp("timeout_build") / "libpagedkv_timeout.so")
    lib_build.build(lib_path=path, extra_flags=("-DPA_WAIT_CYCLES=131072ll",
                                                "-DPA_TEST_DELAY_LAST_TILE_CYCLES=1048576ll"))
    lib = ctypes.CDLL(path)
    vp, i32, i64, f32, sz = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float,
                             ctypes.c_size_t)
    lib.pa_decode_q8.argtypes = [vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32, i32, i64, f32,
                                 i32, vp, sz, vp, vp]
    return lib


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("H,Hk,D,bs", [(16, 8, 128, 16), (8, 1, 128, 16), (32, 8, 64, 16),
                                       (6, 3, 64, 20)])
@pytest.mark.parametrize("n", [5, 40, 1500])
def test_a_late_tile_is_a_timeout(timeout_lib, fmt, H, Hk, D, bs, n):
    """One, a few and many tiles in one CTA of each slab."""
    case = Case([n], H, Hk, D, fmt, "bf16", bs, seed=n)
    ws = pk.DecodeWorkspace(1, H, Hk, D)
    around = torch.full((3, H, D), 7.0, dtype=case.q.dtype, device="cuda")
    torch.cuda.synchronize()
    ptr = lambda t: ctypes.c_void_p(t.data_ptr())
    rc = timeout_lib.pa_decode_q8(
        ptr(around[1]), ptr(case.q), case.cache._arg, ptr(case.bt), case.bt.shape[1],
        ptr(case.ctx), 1, H, Hk, D, 1, bs, case.cache.k.shape[0], 0.0, 1, ptr(ws.buffer), ws.nbytes,
        ptr(case.err), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == 0
    torch.cuda.synchronize()  # raises if the launch faulted
    assert case.err.item() == pk.PA_DEV_ERR["timeout"]
    assert bool((around[0] == 7.0).all() and (around[2] == 7.0).all())
    ws.reset()
    case.err.zero_()
    case.check(grid_ctas=1, workspace=ws)
