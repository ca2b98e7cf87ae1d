"""The 8-bit cache's and the rotary calls through ctypes, as they go where the Python module is not
built: bit for bit what the module gives."""
import pytest
import torch

import paged_kv_cache_107_gb300 as pk
from paged_kv_cache_107_gb300 import build as lib_build

pytestmark = pytest.mark.gpu
DEV = "cuda"


def chain(fmt):
    g = torch.Generator(device=DEV).manual_seed(3)
    n, h, hk, d, bs = 40, 8, 4, 64, 16
    q, k, v = (torch.randn(n, m, d, generator=g, device=DEV).half() for m in (h, hk, hk))
    cache, other = (pk.Q8Cache(3, bs, hk, d, fmt) for _ in range(2))
    rotary = pk.Rotary(d, sections=(8, 24), amplitude=1.5)
    pos = torch.arange(2 * n, dtype=torch.int32, device=DEV).view(2, n)
    slots = torch.arange(n, dtype=torch.int32, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    k_cache, v_cache = (torch.zeros(3, bs, hk, d, device=DEV).half() for _ in range(2))
    outs = [pk.pa_rotary_store(torch.empty_like(q), q, k, v, pos, rotary, k_cache, v_cache, slots,
                               dev_err=err), k_cache, v_cache,
            pk.pa_rotary_store_q8(torch.empty_like(q), q, k, v, pos, rotary, cache, slots, dev_err=err)]
    pk.pa_store_kvcache_q8(k, v, other, slots, dev_err=err)
    for c in (cache, other):
        blocks = [torch.zeros(3, bs, hk, d, device=DEV).half() for _ in range(2)]
        pk.pa_load_kvcache_q8(*blocks, c, torch.tensor([2, -1, 0], dtype=torch.int32, device=DEV))
        tables = torch.tensor([[0, 1, 2], [1, 0, -1]], dtype=torch.int32, device=DEV)
        lens = torch.tensor([n, 20], dtype=torch.int32, device=DEV)
        outs += [*blocks, c.k.view(torch.uint8), c.v.view(torch.uint8), c.k_scale, c.v_scale,
                 pk.pa_decode_q8(torch.empty_like(q[:2]), q[:2], c, tables, lens, scale=0.2,
                                 dev_err=err)]
    assert err.item() == 0
    return outs


@pytest.mark.parametrize("fmt", [torch.float8_e4m3fn, torch.int8])
def test_through_ctypes(fmt, monkeypatch, tmp_path):
    want = chain(fmt)
    module = pk._call_module
    monkeypatch.setattr(lib_build, "CALL_PATH", str(tmp_path / "absent.so"))
    monkeypatch.setattr(pk, "_call_module", None)
    got = chain(fmt)
    assert pk._call_module is not module
    assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))
