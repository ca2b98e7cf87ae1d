"""Waits that run out before a stage of the decode has ever held a tile. The consumers then meet
the stage's first metadata: they must store nothing through it, the call returns with
PA_DEV_ERR_TIMEOUT, and the next call on a zeroed workspace is correct.

As in test_timeout_gpu.py a second copy of the library is built with every wait limit at 2^17
cycles and the producers holding back the copies of a CTA's last key tile for 2^20 cycles; they
issue them late and wait for them, so nothing is left in flight."""
import ctypes

import pytest
import torch

import paged_kv_cache_107_gb300 as pk
from paged_kv_cache_107_gb300 import build as lib_build
from paged_kv_cache_107_gb300 import workloads
from tests.gpu_helpers import DeviceCase, assert_close, from_bits, oracle_after_store, to_f64

import oracle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def timeout_lib(tmp_path_factory):
    path = str(tmp_path_factory.mktemp("timeout_build") / "libpagedkv_timeout.so")
    lib_build.build(lib_path=path, extra_flags=("-DPA_WAIT_CYCLES=131072ll",
                                                "-DPA_TEST_DELAY_LAST_TILE_CYCLES=1048576ll"))
    lib = ctypes.CDLL(path)
    vp, i32, i64, f32, sz = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float,
                             ctypes.c_size_t)
    lib.pa_decode.argtypes = [vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, i32, i32, i64, f32,
                              i32, vp, sz, vp, vp]
    return lib


@pytest.mark.parametrize("H,Hk,D,bs", [(16, 8, 128, 16), (32, 8, 128, 16), (32, 8, 64, 16),
                                       (32, 8, 128, 20)])
@pytest.mark.parametrize("n", [5, 40, 300])
def test_a_late_tile_is_a_timeout_and_no_stray_store(timeout_lib, H, Hk, D, bs, n):
    """One, a few and many tiles of the CUDA-core and the tensor-core decode, in one CTA. The rows
    around the output stay as they were."""
    case = workloads.decode_case([n], H, Hk, D, bs, seed=107810)
    dc = DeviceCase(case)
    dc.store()
    ws = pk.DecodeWorkspace(1, H, Hk, D)
    around = torch.full((3, H, D), 7.0, dtype=dc.q.dtype, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    ptr = lambda t: ctypes.c_void_p(t.data_ptr())
    rc = timeout_lib.pa_decode(
        ptr(around[1]), ptr(dc.q), ptr(dc.k_cache), ptr(dc.v_cache), ptr(dc.bt), dc.bt.shape[1],
        ptr(dc.ctx), 1, H, Hk, D, 1, bs, dc.k_cache.shape[0], 0.0, 1, ptr(ws.buffer), ws.nbytes,
        ptr(err), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == 0
    torch.cuda.synchronize()  # raises if the launch faulted
    assert int(err.item()) == pk.PA_DEV_ERR["timeout"]
    assert torch.all(around[0] == 7.0) and torch.all(around[2] == 7.0)

    ws.reset()
    got = dc.decode(grid_ctas=1, workspace=ws)
    assert dc.dev_err() == 0
    ok, ov = oracle_after_store(case)
    ref = oracle.decode(case.q, from_bits(ok), from_bits(ov), case.block_tables,
                        case.context_lens)
    assert_close(to_f64(got), ref, "decode after a timed-out launch")
