"""Waits of pa_decode_shared that run out, in the prefix part (tensor-core issuer, softmax and the
segments' readers), in the rests (consumers of the decode) and in both: the call returns with
PA_DEV_ERR_TIMEOUT, and the next call on the same workspace is correct, whatever the join found
of the first one's parts.

As in test_timeout_gpu.py a second copy of the library is built with every wait limit at 2^17
cycles. The K warp of a prefix CTA and the producer of a rest hold back the copies of their last
step or tile for 2^20 cycles, issue them late and wait for them, so nothing is left in flight."""
import ctypes

import pytest
import torch

import paged_kv_cache_107_gb300 as pk
from paged_kv_cache_107_gb300 import build as lib_build
from tests.test_decode_shared_gpu import Shared

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def timeout_lib(tmp_path_factory):
    path = str(tmp_path_factory.mktemp("timeout_build") / "libpagedkv_timeout.so")
    lib_build.build(lib_path=path, extra_flags=("-DPA_WAIT_CYCLES=131072ll",
                                                "-DPA_TEST_DELAY_LAST_TILE_CYCLES=1048576ll"))
    lib = ctypes.CDLL(path)
    vp, i32, i64, f32, sz = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float,
                             ctypes.c_size_t)
    lib.pa_decode_shared.argtypes = [vp, vp, vp, vp, vp, i32, vp, vp, vp, i32, i32, i32, i32, i32,
                                     i32, i32, i64, f32, vp, sz, vp, vp]
    return lib


@pytest.mark.parametrize("fill", [0x00, 0xFF, 0x11])
@pytest.mark.parametrize("sizes,prefix,rest", [
    ([4], [256], [0] * 4),                    # nothing but prefixes, one row tile
    ([150], [900], [0] * 150),                # two row tiles and one, several segments a CTA
    ([1, 1, 1], [200, 300, 5], [1, 9, 40]),   # nothing but rests
    ([70, 3, 1], [700, 130, 0], [1 + i % 90 for i in range(74)])])
@pytest.mark.parametrize("D", [64, 128])
def test_late_tiles_are_a_timeout(timeout_lib, sizes, prefix, rest, D, fill):
    c = Shared(sizes, prefix, rest, 16, 8, D, 16, torch.bfloat16, seed=107820)
    q, k, v, bt, ctx, starts, plen = c.device()
    B = len(c.lens)
    ws = pk.SharedDecodeWorkspace(B, 16, 8, D)
    ws.buffer.fill_(fill)
    around = torch.full((B + 2, 16, D), 7.0, dtype=q.dtype, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    ptr = lambda t: ctypes.c_void_p(t.data_ptr())
    rc = timeout_lib.pa_decode_shared(
        ptr(around[1]), ptr(q), ptr(k), ptr(v), ptr(bt), bt.shape[1], ptr(ctx), ptr(starts),
        ptr(plen), B, len(sizes), 16, 8, D, 1, 16, k.shape[0], 0.0, ptr(ws.buffer), ws.nbytes,
        ptr(err), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == 0
    torch.cuda.synchronize()  # raises if a launch faulted
    assert int(err.item()) == pk.PA_DEV_ERR["timeout"], f"error word {int(err.item())}"
    assert torch.all(around[0] == 7.0) and torch.all(around[-1] == 7.0)
    c.check(ws=ws)
