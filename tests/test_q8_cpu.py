"""The calls around 8-bit caches and rotary positions without a GPU: refusals through the C ABI
and the binding, the frequencies' fractions, and the reference's own roundings."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import paged_kv_cache_107_gb300 as pk
from tests import q8_reference as ref
from paged_kv_cache_107_gb300 import build as lib_build

VP = ctypes.c_void_p
I64 = ctypes.c_int64


@pytest.fixture(scope="module")
def lib():
    return ctypes.CDLL(lib_build.build())


def cache(fmt=1, k=16, v=16, ks=16, vs=16):
    return ctypes.byref(pk._PaQ8Cache(k, v, ks, vs, fmt))


def rotary(rot=128, axes=1, amplitude=1.0, turns=16, ax=16):
    return ctypes.byref(pk._PaRotary(turns, ax, rot, axes, 0, amplitude))


def store(lib, c="default", n=3, hk=8, d=128, bs=16, nb=4, dtype=1, ks=1024, vs=1024, k=16, v=16,
          slots=16):
    return lib.pa_store_kvcache_q8(VP(k), VP(v), I64(ks), I64(vs), dtype,
                                   cache() if c == "default" else c, VP(slots), n, hk, d, bs,
                                   I64(nb), None, None)


def load(lib, c="default", n=3, hk=8, d=128, bs=16, nb=4, dtype=1, k=16, v=16, blocks=16):
    return lib.pa_load_kvcache_q8(VP(k), VP(v), dtype, cache() if c == "default" else c,
                                  VP(blocks), n, hk, d, bs, I64(nb), None, None)


def rotate(lib, r="default", n=3, h=16, hk=8, d=128, dtype=1, qs=2048, qos=2048, ks=1024, vs=1024,
           q=16, qo=16, pos=16, kc=16, q8=None):
    r = rotary() if r == "default" else r
    head = (VP(qo), VP(q), VP(16), VP(16), I64(qos), I64(qs), I64(ks), I64(vs), dtype, VP(pos),
            I64(0), r)
    tail = (VP(16), n, h, hk, d, 16, I64(4), None, None)
    if q8 is not None:
        return lib.pa_rotary_store_q8(*head, q8, *tail)
    return lib.pa_rotary_store(*head, VP(kc), VP(16), *tail)


def decode(lib, c="default", B=2, H=16, D=128, dtype=1, bs=16, q=16, ws=1 << 30):
    return lib.pa_decode_q8(VP(16), VP(q), cache() if c == "default" else c, VP(16), 1, VP(16), B, H,
                            8, D, dtype, bs, I64(4), ctypes.c_float(0), 0, VP(256),
                            ctypes.c_size_t(ws), None, None)


@pytest.mark.parametrize("call", [store, load, decode])
def test_c_refusals_of_a_cache(lib, call):
    assert call(lib, None) == 1
    for fmt in (0, 3, -1):
        assert call(lib, cache(fmt)) == 3
    for missing in ("k", "v", "ks", "vs"):
        assert call(lib, cache(**{missing: None})) == 1
        assert call(lib, cache(**{missing: 8})) == 6
    assert call(lib, dtype=0) == 3


@pytest.mark.parametrize("call", [store, load])
def test_c_refusals_of_shapes(lib, call):
    for kw in (dict(n=-1), dict(hk=0), dict(bs=0), dict(nb=0)):
        assert call(lib, **kw) == 2, kw
    assert call(lib, d=96) == 3
    assert call(lib, n=0) == 0  # nothing to do
    assert call(lib, k=None) == 1 and call(lib, v=None) == 1
    assert load(lib, bs=1 << 20, hk=1 << 12) == 3
    assert load(lib, k=8) == 6 and load(lib, blocks=2) == 6
    assert store(lib, ks=1023) == 2 and store(lib, vs=1023) == 2
    assert store(lib, k=1) == 6 and store(lib, slots=None) == 1


def test_c_refusals_of_rotary(lib):
    for q8 in (None, cache()):
        assert rotate(lib, None, q8=q8) == 1
        for kw in (dict(rot=0), dict(rot=8), dict(rot=24), dict(rot=144), dict(axes=0),
                   dict(axes=17), dict(amplitude=math.inf), dict(amplitude=math.nan)):
            assert rotate(lib, rotary(**kw), q8=q8) == 2, kw
        assert rotate(lib, rotary(turns=None), q8=q8) == 1
        assert rotate(lib, rotary(ax=None), q8=q8) == 1
        assert rotate(lib, rotary(turns=4), q8=q8) == 6
        for kw in (dict(h=0), dict(hk=0), dict(n=-1), dict(qs=2047), dict(qos=2047), dict(ks=1023)):
            assert rotate(lib, q8=q8, **kw) == 2, kw
        assert rotate(lib, q8=q8, d=80) == 3 and rotate(lib, q8=q8, dtype=0) == 3
        assert rotate(lib, q8=q8, q=None) == 1 and rotate(lib, q8=q8, pos=None) == 1
        assert rotate(lib, q8=q8, qo=1) == 6
        assert rotate(lib, q8=q8, n=0) == 0
    assert rotate(lib, kc=8) == 6 and rotate(lib, kc=None) == 1
    assert rotate(lib, q8=cache(7)) == 3
    # rotation only reaches the head's own dims
    assert rotate(lib, rotary(rot=128), d=64) == 2


def test_c_refusals_of_decode(lib):
    assert decode(lib, H=12) == 2 and decode(lib, H=72) == 3 and decode(lib, D=96) == 3
    assert decode(lib, q=8) == 6 and decode(lib, B=-1) == 2 and decode(lib, B=0) == 0


def test_frequencies_as_fractions_of_a_turn():
    bits = 400

    def arctan_inverse(n):  # of 1/n, in 2^-bits
        term = total = (1 << bits) // n
        k, sign = 1, -1
        while term:
            term //= n * n
            k += 2
            total += sign * (term // k)
            sign = -sign
        return total

    two_pi = 8 * (4 * arctan_inverse(5) - arctan_inverse(239))
    freqs = [1.0, 0.5, 1e-6, 0.3, -1.0, 2.0 ** 40, -(2.0 ** 40), 2.0 ** -80, math.pi, 0.0, 5e-324]
    freqs += [1e6 ** (-2 * i / 128) for i in range(64)]
    for f in freqs:
        exact = Fraction(f) * (1 << bits) / two_pi * (1 << 64) % (1 << 64)
        off = (pk.pa_rotary_turns(f) - exact) % (1 << 64)
        assert min(off, (1 << 64) - off) <= Fraction(51, 100), f
    for f in (math.inf, -math.inf, math.nan, 2.0 ** 41):
        assert pk.pa_rotary_turns(f) == 0


def test_reference_rounds_as_torch_does():
    """Every bf16 magnitude below 464 (e4m3), and the int8 ties of a power of two."""
    x = torch.arange(0x43e0, dtype=torch.int16).view(torch.bfloat16).float()
    x = x[x <= 448]
    assert np.array_equal(ref.e4m3_round(x.double().numpy()),
                          x.to(torch.float8_e4m3fn).double().numpy())
    row = torch.tensor([[128.0, 64.0, 0.5, 1.5, 2.5, -2.5]], dtype=torch.float64).numpy()
    codes, scale = ref.quantise("int8", row)
    assert codes.tolist() == [[127, 64, 0, 1, 2, -2]] and scale[0] == np.float32(128 / 127)
    codes, scale = ref.quantise("e4m3", np.array([[448.0, 1.0], [449.0, 1.0], [0.0, 0.0],
                                                  [np.inf, 1.0]]))
    assert scale[:3].tolist() == [1.0, 2.0, 0.0] and np.isnan(scale[3])
    assert codes.tolist() == [[448, 1], [224, 0.5], [0, 0], [0, 0]]


def test_calls_without_ctypes(lib):
    """The compiled binding passes every argument on: the statuses of the C ABI, for each call."""
    calls = pk._calls()
    c = pk._PaQ8Cache(16, 16, 16, 16, 1)
    r = pk._PaRotary(16, 16, 128, 1, 0, 1.0)
    a, ra = ctypes.addressof(c), ctypes.addressof(r)
    store = [16, 16, 1024, 1024, 1, a, 16, 0, 8, 128, 16, 4, None, None]
    load = [16, 16, 1, a, 16, 0, 8, 128, 16, 4, None, None]
    decode = [16, 16, a, 16, 1, 16, 0, 16, 8, 128, 1, 16, 4, 0.0, 0, 256, 1 << 30, None, None]
    head = [16, 16, 16, 16, 2048, 2048, 1024, 1024, 1, 16, 0, ra]
    tail = [16, 0, 16, 8, 128, 16, 4, None, None]
    for name, args, bad in (
            ("pa_store_kvcache_q8", store, {2: 1023, 3: -5, 4: 0, 7: -1, 8: 0, 9: 96, 10: 0, 11: 0}),
            ("pa_load_kvcache_q8", load, {2: 0, 3: None, 5: -1, 6: 0, 7: 96, 8: 0, 9: -1}),
            ("pa_decode_q8", decode, {2: None, 4: -1, 6: -1, 7: 12, 8: 0, 9: 96, 10: 0, 11: 0, 12: 0,
                                      14: -1}),
            ("pa_rotary_store", head + [16, 16] + tail, {4: 2047, 5: 2047, 6: 1023, 7: 1023, 8: 0,
                                                         11: None, 15: -1, 16: 0, 17: 0, 18: 96,
                                                         19: 0, 20: 0}),
            ("pa_rotary_store_q8", head + [a] + tail, {4: 2047, 5: 2047, 6: 1023, 7: 1023, 8: 0,
                                                       11: None, 12: None, 14: -1, 15: 0, 16: 0,
                                                       17: 96, 18: 0, 19: 0})):
        fn = getattr(calls, name)
        assert fn(*args) == 0, name  # nothing to do
        for i, x in bad.items():
            assert fn(*args[:i], x, *args[i + 1:]) in (1, 2, 3), (name, i)
        for wrong in (args[:-1], args + [0], []):
            with pytest.raises(TypeError):
                fn(*wrong)
        with pytest.raises(TypeError):
            fn("x", *args[1:])
    with pytest.raises(TypeError):
        calls.pa_decode_q8(*decode[:13], "x", *decode[14:])


# ---------------------------------------------------------------- the binding
def host_cache(nb=2, bs=16, hk=8, d=128, dtype=torch.int8):
    return pk.Q8Cache(nb, bs, hk, d, dtype, device="cpu")


def host_rotary(**kw):
    return pk.Rotary(device="cpu", **kw)


def test_binding_refuses_host_tensors():
    c = host_cache()
    x, i = torch.zeros(2, 8, 128, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    q = torch.zeros(2, 16, 128, dtype=torch.bfloat16)
    b = torch.zeros(2, 16, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(pk.PagedAttentionError, match="CUDA"):
        pk.pa_store_kvcache_q8(x, x, c, i)
    with pytest.raises(pk.PagedAttentionError, match="CUDA"):
        pk.pa_load_kvcache_q8(b, b, c, i)
    with pytest.raises(pk.PagedAttentionError, match="CUDA"):
        pk.pa_decode_q8(q, q, c, i[:, None], i)
    with pytest.raises(pk.PagedAttentionError, match="CUDA"):
        pk.pa_rotary_store(q, q, x, x, i, host_rotary(), b, b.clone(), i)
    with pytest.raises(pk.PagedAttentionError, match="CUDA"):
        pk.pa_rotary_store_q8(q, q, x, x, i, host_rotary(), c, i)


@pytest.mark.parametrize("name,bad", [
    ("k", torch.zeros(2, 16, 8, 128, dtype=torch.uint8)),
    ("k", torch.zeros(2, 16, 8, 128, dtype=torch.float8_e4m3fn)),  # V is int8
    ("k", torch.zeros(2, 16, 8, 64, dtype=torch.int8)),
    ("k", torch.zeros(16, 8, 128, dtype=torch.int8)),
    ("k", torch.zeros(2, 16, 128, 8, dtype=torch.int8).transpose(2, 3)),
    ("k_scale", torch.zeros(2, 16, 8)),
    ("v_scale", torch.zeros(2, 8, 16, dtype=torch.float64)),
    ("v_scale", torch.zeros(2, 16, 8).transpose(1, 2)),
    ("k_scale", torch.zeros(2, 8, 16, device="meta"))])
def test_binding_refuses_caches(name, bad):
    t = dict(k=torch.zeros(2, 16, 8, 128, dtype=torch.int8),
             v=torch.zeros(2, 16, 8, 128, dtype=torch.int8),
             k_scale=torch.zeros(2, 8, 16), v_scale=torch.zeros(2, 8, 16))
    pk.Q8Cache.of(**t)
    t[name] = bad
    with pytest.raises(pk.PagedAttentionError):
        pk.Q8Cache.of(**t)


@pytest.mark.parametrize("make", [lambda: None, lambda: torch.zeros(2, 16, 8, 128)])
def test_binding_wants_a_q8_cache(make):
    x, i = torch.zeros(2, 8, 128, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    for call in (lambda c: pk.pa_store_kvcache_q8(x, x, c, i),
                 lambda c: pk.pa_load_kvcache_q8(x, x, c, i),
                 lambda c: pk.pa_decode_q8(x, x, c, i, i),
                 lambda c: pk.pa_rotary_store_q8(x, x, x, x, i, host_rotary(), c, i)):
        with pytest.raises(pk.PagedAttentionError, match="Q8Cache"):
            call(make())


def test_row_strides():
    x = torch.zeros(6, 24, 64, dtype=torch.bfloat16)
    assert pk._rows("k", x[:, 16:20], torch.bfloat16, 6, 4, 64) == 24 * 64
    assert pk._rows("k", x[:1, 16:20], torch.bfloat16, 1, 4, 64) == 24 * 64
    assert pk._rows("k", x[:0, :4], torch.bfloat16, 0, 4, 64) == 24 * 64
    one = x.as_strided((1, 24, 64), (7, 64, 1))  # a single token's stride does not matter
    assert pk._rows("k", one, torch.bfloat16, 1, 24, 64) == 24 * 64
    for bad in (x[:, ::2], x[..., :32], x.transpose(0, 1), x[:1].expand(6, 24, 64), x.float(),
                x[:, :3], x.as_strided((2, 24, 64), (64, 64, 1))):
        with pytest.raises(pk.PagedAttentionError):
            pk._rows("k", bad, torch.bfloat16, bad.shape[0], 24, 64)


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=24), dict(rotary_dim=8), dict(rotary_dim=256), dict(base=0.0), dict(base=0.5),
    dict(base=math.nan), dict(base=math.inf), dict(sections=(64, -5)), dict(rotary_dim=0), dict(rotary_dim=-16), dict(inv_freq=[1.0] * 7), dict(inv_freq=[math.inf] * 8),
    dict(inv_freq=[2.0 ** 41] * 8), dict(sections=(16, 24)), dict(sections=(16, 24, 25)),
    dict(axes=[0] * 63), dict(axes=[-1] + [0] * 63), dict(axes=[16] + [0] * 63),
    dict(sections=(16, 24, 24), axes=[0] * 64), dict(amplitude=math.inf),
    dict(rotary_dim=32, inv_freq=[1.0] * 8)])
def test_binding_refuses_frequencies(kw):
    with pytest.raises(pk.PagedAttentionError):
        host_rotary(**kw)


def test_rotary_plans():
    r = host_rotary()
    assert (r.rotary_dim, r.num_axes, r.head_dim) == (128, 1, 128)
    assert r.turns[0].item() == pk.pa_rotary_turns(1.0)
    r = host_rotary(sections=(16, 24, 24), base=1e6)
    assert r.num_axes == 3 and r.axes.tolist() == [0] * 16 + [1] * 24 + [2] * 24
    r = host_rotary(head_dim=64, rotary_dim=32, axes=[0, 1] * 8, adjacent=True)
    assert r.num_axes == 2 and r.axes.tolist() == [0, 1] * 8 and r.rotary_dim == 32
    # a section may be empty: the call still takes its axis
    assert host_rotary(sections=(64, 0, 0)).num_axes == 3
    r = host_rotary(inv_freq=[-1.0] * 64)
    assert r.turns[0].item() % (1 << 64) == pk.pa_rotary_turns(-1.0)
