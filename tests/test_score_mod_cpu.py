"""Refusals of pa_decode_mod and pa_prefill_mod, through the C ABI and the binding: no GPU is
touched (rules out of range are refused before the device is looked at)."""
import ctypes
import math

import pytest
import torch

import paged_kv_cache_107_gb300 as pk
from paged_kv_cache_107_gb300 import build as lib_build


@pytest.fixture(scope="module")
def lib():
    return ctypes.CDLL(lib_build.build())


def rules(softcap=0.0, window=0, sink=0):
    return pk._PaScoreMod(softcap, window, sink, None, None)


def decode(lib, mod, B=2, H=16, D=128, dtype=1, scale=0.0):
    vp = ctypes.c_void_p(16)
    return lib.pa_decode_mod(vp, vp, vp, vp, vp, 1, vp, B, H, 8, D, dtype, 16, ctypes.c_int64(4),
                             ctypes.c_float(scale), ctypes.byref(mod) if mod else None, 0, vp,
                             ctypes.c_size_t(1 << 20), None, None)


def prefill(lib, mod, S=2, H=16, D=128, bs=16, dtype=1, scale=0.0):
    vp = ctypes.c_void_p(16)
    return lib.pa_prefill_mod(vp, vp, vp, vp, vp, 4, vp, vp, S, 10, 20, H, 8, D, dtype, bs,
                              ctypes.c_int64(4), 1, ctypes.c_float(scale),
                              ctypes.byref(mod) if mod else None, None, None)


@pytest.mark.parametrize("call", [decode, prefill])
def test_c_refusals(lib, call):
    assert call(lib, None) == 1
    for bad in (-1.0, math.inf, math.nan):
        assert call(lib, rules(softcap=bad)) == 2
    # factors that leave fp32: scale / softcap, softcap * log2(e)
    assert call(lib, rules(softcap=1e-30), scale=1e30) == 2
    assert call(lib, rules(softcap=3e38)) == 2
    assert call(lib, rules(softcap=1e30), scale=1e-9) == 2
    assert call(lib, rules(window=-1)) == 2
    assert call(lib, rules(sink=-1)) == 2
    assert call(lib, rules(), H=12) == 2
    assert call(lib, rules(), D=96) == 3
    assert call(lib, rules(), dtype=0) == 3
    assert call(lib, rules(softcap=50.0), 0) == 0  # an empty batch


def test_prefill_block_size(lib):
    assert prefill(lib, rules(), bs=20) == 3
    assert prefill(lib, rules(), H=24) == 3


def tensors(B=2, H=16, Hk=8, D=128):
    q = torch.zeros(B, H, D, dtype=torch.bfloat16)
    kc = torch.zeros(2, 16, Hk, D, dtype=torch.bfloat16)
    return q.clone(), q, kc, kc.clone(), torch.zeros(B, 1, dtype=torch.int32), torch.ones(
        B, dtype=torch.int32)


def test_binding_refuses_host_tensors():
    with pytest.raises(pk.PagedAttentionError, match="CUDA"):
        pk.pa_decode_mod(*tensors(), pk.ScoreMod())
    cu = torch.zeros(2, dtype=torch.int32)
    o, q, kc, vc, bt, _ = tensors()
    with pytest.raises(pk.PagedAttentionError, match="CUDA"):
        pk.pa_prefill_mod(o, q, kc, vc, bt[:1], cu, cu, 1, 1, pk.ScoreMod())


@pytest.mark.parametrize("kw", [dict(softcap=-1.0), dict(softcap=math.inf), dict(softcap=math.nan),
                                dict(window=-1), dict(sink=-1), dict(window=1 << 31),
                                dict(slopes=torch.zeros(16)),
                                dict(prefix_lens=torch.zeros(2, dtype=torch.int32))])
def test_binding_refuses_rules(kw):
    with pytest.raises(pk.PagedAttentionError):
        pk.ScoreMod(**kw)._check(16, 2)


@pytest.mark.parametrize("mod", [None, dict(softcap=1.0), 30.0])
def test_binding_wants_a_score_mod(mod):
    cu = torch.zeros(2, dtype=torch.int32)
    o, q, kc, vc, bt, ctx = tensors()
    with pytest.raises(pk.PagedAttentionError, match="ScoreMod"):
        pk.pa_decode_mod(o, q, kc, vc, bt, ctx, mod)
    with pytest.raises(pk.PagedAttentionError, match="ScoreMod"):
        pk.pa_prefill_mod(o, q, kc, vc, bt[:1], cu, cu, 1, 1, mod)
