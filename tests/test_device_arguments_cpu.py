"""Objects that allocate on a device take index 0 for device 0, whichever the current one is."""
import pytest
import torch

import paged_kv_cache_107_gb300 as pk
from paged_kv_cache_107_gb300 import build as lib_build

MAKE = {
    "Q8Cache": lambda **kw: pk.Q8Cache(2, 16, 8, 128, **kw),
    "Rotary": lambda **kw: pk.Rotary(64, **kw),
    "DecodeWorkspace": lambda **kw: pk.DecodeWorkspace(2, 16, 8, **kw),
    "SampleWorkspace": lambda **kw: pk.SampleWorkspace(2, **kw),
}


@pytest.mark.parametrize("name", MAKE)
@pytest.mark.parametrize("device,want", [(0, "cuda:0"), (1, "cuda:1"), ("cuda:0", "cuda:0"),
                                         (torch.device("cuda", 2), "cuda:2"), (None, "cuda"),
                                         ("cuda", "cuda"), ("cpu", "cpu")])
def test_device(name, device, want, monkeypatch):
    lib_build.build()
    monkeypatch.setattr(pk, "pa_decode_workspace_size", lambda *a: 256)  # (asks the device)
    asked = []

    def on_the_host(make):
        def wrapped(*args, device=None, **kw):
            asked.append(torch.device(device))
            return make(*args, device="cpu", **kw)
        return wrapped

    for fn in ("zeros", "empty", "tensor"):
        monkeypatch.setattr(torch, fn, on_the_host(getattr(torch, fn)))
    MAKE[name](**({} if device is None else {"device": device}))
    assert asked and set(asked) == {torch.device(want)}
