"""pa_store_kvcache_q8 and pa_load_kvcache_q8 on the GPU: codes and scales equal to the
definition's to the bit, over types, head counts, strides, alignments and block sizes; rows with
zeros, ties, subnormals, the types' largest values, infinities and NaN."""
import numpy as np
import pytest
import torch

import paged_kv_cache_107_gb300 as pk
from tests import q8_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def new_cache(nb, bs, hk, d, fmt):
    """A cache whose every byte is marked, to see what a call leaves alone."""
    codes = [torch.full((nb, bs, hk, d), 0x55, dtype=torch.uint8, device=DEV).view(ref.FORMATS[fmt])
             for _ in range(2)]
    scales = [torch.full((nb, hk, bs), -7.0, device=DEV) for _ in range(2)]
    return pk.Q8Cache.of(*codes, *scales)


def check_store(cache, k, v, slots, fmt):
    nb, bs, hk, d = cache.k.shape
    for codes, scales, x in ((cache.k, cache.k_scale, k), (cache.v, cache.v_scale, v)):
        want_c = torch.full((nb * bs, hk, d), 0x55, dtype=torch.uint8).view(ref.FORMATS[fmt])
        want_s = torch.full((nb * bs, hk), -7.0)
        c, s = ref.quantise(fmt, x.double().cpu().numpy())
        for i, slot in enumerate(slots):
            if 0 <= slot < nb * bs:
                want_c[slot] = torch.from_numpy(c[i]).to(torch.float32).to(ref.FORMATS[fmt])
                want_s[slot] = torch.from_numpy(s[i]).float()
        got_c = codes.cpu().view(nb * bs, hk, d)
        # (e4m3 has two zeros)
        assert torch.equal(got_c.float().nan_to_num(1e9), want_c.float().nan_to_num(1e9))
        got_s = scales.cpu().transpose(1, 2).reshape(nb * bs, hk)
        assert torch.equal(got_s.nan_to_num(1e9), want_s.nan_to_num(1e9))


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d,hk,bs,n", [(128, 8, 16, 1), (128, 8, 256, 700), (64, 8, 16, 333),
                                       (128, 1, 20, 67), (64, 1, 1, 5), (64, 3, 32, 100),
                                       (128, 5, 8, 41), (128, 16, 48, 129), (64, 40, 16, 9),
                                       (128, 2, 16, 500), (128, 3, 8, 1), (64, 7, 16, 1031),
                                       (128, 4, 32, 77), (64, 2, 256, 3000), (128, 1, 64, 2000)])
def test_store_matches_the_definition(fmt, dtype, d, hk, bs, n):
    g = torch.Generator(device=DEV).manual_seed(n * hk)
    # rows of very different sizes
    size = torch.exp2(torch.randint(-12, 12, (n, hk, 1), generator=g, device=DEV).float())
    k = (torch.randn(n, hk, d, generator=g, device=DEV) * size).to(TYPES[dtype])
    v = torch.randn(n, hk, d, generator=g, device=DEV).to(TYPES[dtype])
    nb = -(-n // bs) + 2
    slots = torch.randperm(nb * bs, generator=torch.Generator().manual_seed(n))[:n].int()
    slots[::5] = -1
    cache = new_cache(nb, bs, hk, d, fmt)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pk.pa_store_kvcache_q8(k, v, cache, slots.to(DEV), dev_err=err)
    check_store(cache, k, v, slots.tolist(), fmt)
    assert err.item() == 0


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("d,hk", [(128, 8), (64, 3)])
@pytest.mark.parametrize("shift", [0, 1, 3])
def test_store_of_strided_and_unaligned_rows(fmt, d, hk, shift):
    n, h = 37, 6
    g = torch.Generator(device=DEV).manual_seed(shift)
    width = (h + 2 * hk) * d + (5 if shift == 3 else 0)
    flat = torch.randn(n * width + shift, generator=g, device=DEV).to(torch.bfloat16)
    rows = flat[shift:].as_strided((n, h + 2 * hk, d), (width, d, 1), shift)
    k, v = rows[:, h:h + hk], rows[:, h + hk:]
    cache = new_cache(4, 16, hk, d, fmt)
    slots = torch.arange(n).flip(0).int()
    pk.pa_store_kvcache_q8(k, v, cache, slots.to(DEV))
    check_store(cache, k, v, slots.tolist(), fmt)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
def test_store_of_special_rows(fmt, dtype, d):
    t = TYPES[dtype]
    fin = torch.finfo(t)
    rows = []

    def row(*values):
        x = torch.zeros(d, dtype=torch.float64)
        x[:len(values)] = torch.tensor(values, dtype=torch.float64)
        rows.append(x.to(t).roll(len(rows)))

    row()
    row(-0.0, 0.0)
    for p in range(-6, 8):  # ties of both formats: largest value a power of two, halves below
        row(2.0 ** p, *(2.0 ** p * (2 * i + 1) / 256 for i in range(40)))
        row(1.75 * 2.0 ** p, 2.0 ** p, -1.75 * 2.0 ** p)  # exactly 448 steps
        row((1.75 + fin.eps) * 2.0 ** p, 1.1 * 2.0 ** p)  # just above
    # every odd quotient i / 2 of 127 and the numbers next to it
    for base in (3 * 2.0 ** -5, 127.0 / 64, 254.0 / 256, 1.0, 85.0):
        x = base / 254 * (2 * torch.arange(30, dtype=torch.float64) + 1)
        row(base, *x.to(t).double().tolist())
    row(fin.max, -fin.max, fin.max / 2, 1.0)
    row(fin.tiny, fin.tiny / 2, -fin.tiny)
    row(fin.smallest_normal * fin.eps, -fin.smallest_normal * fin.eps)  # one subnormal step
    row(fin.smallest_normal * fin.eps * 3, fin.smallest_normal * fin.eps * 2)
    row(float("inf"), 1.0)
    row(1.0, -float("inf"), float("nan"))
    row(float("nan"))
    row(2.0, 1e-6, -1e-6, 2.0 ** -9, 2.0 ** -10)  # far below the largest
    # neighbours of every code border: 1 and 1 + eps over a spread of sizes
    for top in (1.0, 1.3, 1.7421875):
        row(top, *(top * (1 + i * fin.eps) * 2.0 ** -(i % 9) for i in range(50)))
    k = torch.stack(rows)[:, None].to(DEV)
    v = k.flip(0).contiguous()
    n = k.shape[0]
    cache = new_cache(-(-n // 8), 8, 1, d, fmt)
    slots = torch.arange(n, dtype=torch.int32)
    pk.pa_store_kvcache_q8(k, v, cache, slots.to(DEV))
    check_store(cache, k, v, slots.tolist(), fmt)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_int8_codes_of_every_pair(dtype):
    """code = round(127 x / t) for t over all significands of the type and x over many: the
    quotient's ties and their neighbours are met, and none may go the wrong way."""
    t = TYPES[dtype]
    m = 2 ** (7 if dtype == "bf16" else 10)
    tops = 1 + torch.arange(m, dtype=torch.float64) / m
    if m > 256:
        tops = tops[torch.randperm(m, generator=torch.Generator().manual_seed(1))[:300]]
    x = torch.arange(2 * m, dtype=torch.float64) / (2 * m)  # [0, 1) in half steps of the top's
    x = torch.cat([x, x * 2.0 ** -4, x * 2.0 ** -7]).to(t).double()
    x = torch.cat([x, torch.zeros(-x.numel() % 127, dtype=torch.float64)]).view(-1, 127)
    rows = torch.cat([tops[:, None, None].expand(-1, x.shape[0], 1),
                      x[None].expand(len(tops), -1, -1)], -1).reshape(-1, 1, 128).to(t).to(DEV)
    n = rows.shape[0]
    cache = pk.Q8Cache(-(-n // 256), 256, 1, 128, torch.int8)
    pk.pa_store_kvcache_q8(rows, rows, cache, torch.arange(n, dtype=torch.int32, device=DEV))
    y = rows.double()
    # 127 x and t are exact in float64, and a tie's quotient is too
    want = torch.round(127 * y / y[..., :1].abs())
    assert torch.equal(cache.k.view(-1, 1, 128)[:n].double(), want)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_store_of_bad_slots(fmt):
    k = torch.randn(6, 8, 128, device=DEV).bfloat16()
    cache = new_cache(2, 16, 8, 128, fmt)
    slots = torch.tensor([3, 32, -2, 31, -1, 2 ** 31 - 1], dtype=torch.int32)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pk.pa_store_kvcache_q8(k, k, cache, slots.to(DEV), dev_err=err)
    check_store(cache, k, k, slots.tolist(), fmt)
    assert err.item() == pk.PA_DEV_ERR["slot"]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d,hk,bs,nb", [(128, 8, 16, 7), (64, 8, 256, 3), (64, 1, 1, 9),
                                        (128, 3, 20, 5), (64, 5, 7, 6), (128, 1, 33, 4)])
def test_load_matches_the_definition(fmt, dtype, d, hk, bs, nb):
    g = torch.Generator(device=DEV).manual_seed(bs)
    raw = [torch.randint(0, 256, (nb, bs, hk, d), dtype=torch.uint8, generator=g, device=DEV)
           for _ in range(2)]
    scales = [torch.exp2(torch.randint(-20, 20, (nb, hk, bs), generator=g, device=DEV).float())
              * (1 + torch.rand(nb, hk, bs, generator=g, device=DEV)) for _ in range(2)]
    cache = pk.Q8Cache.of(*(x.view(ref.FORMATS[fmt]) for x in raw), *scales)
    blocks = [nb - 1, -1, 0, 0, nb, -2, 1, 2 ** 31 - 1]
    out = [torch.full((len(blocks), bs, hk, d), 3.25, dtype=TYPES[dtype], device=DEV)
           for _ in range(2)]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pk.pa_load_kvcache_q8(*out, cache, torch.tensor(blocks, dtype=torch.int32, device=DEV),
                          dev_err=err)
    assert err.item() == pk.PA_DEV_ERR["block_id"]
    for o, c, s in zip(out, (cache.k, cache.v), scales):
        for i, b in enumerate(blocks):
            if 0 <= b < nb:
                # one fp32 product, then one rounding: the product of an 8-bit code and an fp32
                # scale rounded twice is what the definition rounds once, but for half steps
                exact = c[b].float().double() * s[b].double().t()[..., None]
                half = torch.finfo(TYPES[dtype]).eps / 2
                got = o[i].double()
                nan = exact.isnan()
                assert torch.equal(got.isnan(), nan)
                big = exact.abs() >= torch.finfo(TYPES[dtype]).max
                tol = exact.abs() * half * (1 + 2.0 ** -13) + (2.0 ** -25 if dtype == "fp16" else 0)
                ok = (got - exact).abs() <= tol
                assert bool((ok | nan | big).all())
                assert bool((got[big & ~nan].abs() >= 65504).all())
            else:
                assert bool((o[i] == 3.25).all())


def test_what_is_stored_reads_back():
    """Stored rows read back within half a step: 2^-4 relative, or half of the row's least step
    for e4m3; half of scale for int8."""
    k = torch.randn(500, 8, 128, device=DEV).bfloat16()
    v = (torch.randn(500, 8, 128, device=DEV) * 30).bfloat16()
    for fmt, dt in ref.FORMATS.items():
        cache = pk.Q8Cache(32, 16, 8, 128, dt)
        slots = torch.randperm(512, device=DEV)[:500].int()
        pk.pa_store_kvcache_q8(k, v, cache, slots)
        out = [torch.zeros(32, 16, 8, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        pk.pa_load_kvcache_q8(*out, cache, torch.arange(32, dtype=torch.int32, device=DEV))
        for o, x, s in zip(out, (k, v), (cache.k_scale, cache.v_scale)):
            got = o.view(512, 8, 128)[slots.long()].double()
            scale = s.transpose(1, 2).reshape(512, 8)[slots.long()].double()[..., None]
            off = (got - x.double()).abs()
            if fmt == "e4m3":
                bound = torch.maximum(x.double().abs() * 2.0 ** -4, scale * 2.0 ** -10)
            else:
                bound = scale * 0.5 * (1 + 2.0 ** -20) + got.abs() * 2.0 ** -8
            assert bool((off <= bound).all())


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_empty_calls_and_refusals(fmt):
    cache = new_cache(2, 16, 8, 128, fmt)
    k = torch.randn(4, 8, 128, device=DEV).bfloat16()
    i = torch.zeros(4, dtype=torch.int32, device=DEV)
    out = torch.zeros(4, 16, 8, 128, dtype=torch.bfloat16, device=DEV)
    pk.pa_store_kvcache_q8(k[:0], k[:0], cache, i[:0])
    pk.pa_load_kvcache_q8(out[:0], out[:0], cache, i[:0])
    assert bool((cache.k.view(torch.uint8) == 0x55).all())
    for bad in (dict(k=k.float()), dict(v=k.half()), dict(k=k[:, :4]), dict(k=k[:3]),
                dict(slot_mapping=i.long()), dict(slot_mapping=i[:3]), dict(slot_mapping=i.cpu()),
                dict(k=k.cpu()), dict(dev_err=torch.zeros(1, dtype=torch.int32))):
        args = dict(k=k, v=k, cache=cache, slot_mapping=i) | bad
        with pytest.raises(pk.PagedAttentionError):
            pk.pa_store_kvcache_q8(**args)
    for bad in (dict(k_out=out.float()), dict(v_out=out.half()), dict(k_out=out[:3]),
                dict(blocks=i.long()), dict(blocks=i[:3]), dict(v_out=out[:, :8]),
                dict(blocks=i.cpu()), dict(k_out=out.transpose(0, 1).contiguous().transpose(0, 1))):
        args = dict(k_out=out, v_out=out.clone(), cache=cache, blocks=i) | bad
        with pytest.raises(pk.PagedAttentionError):
            pk.pa_load_kvcache_q8(**args)
