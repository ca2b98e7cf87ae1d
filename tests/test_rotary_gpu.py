"""pa_rotary_store and pa_rotary_store_q8 on the GPU against the definition in 64 bits: axes,
pairings, partial heads, strides, far positions; the 8-bit form against the two calls apart.

A turned element a cos - b sin: cos and sin are off by 2^-22 at most (the angle is a fraction of
a turn in fp32, half of 2^-24 of at most half a turn, times 2 pi; sincospi adds 2^-23), the two
products and the sum by 2^-24 each relative, the result is rounded once:
half |exact| + (|a| + |b|) amplitude 2^-21."""
import numpy as np
import pytest
import torch

import paged_kv_cache_107_gb300 as pk
from tests import q8_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def check(got, x, pos, r, inv_freq, axes, adjacent, amplitude=1.0):
    dt = got.dtype
    x = x.double().cpu().numpy()
    exact = ref.rotate(x, pos, inv_freq, axes, adjacent, amplitude)
    rot = 2 * len(inv_freq)
    size = np.zeros_like(x)
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if adjacent else (x[..., :rot // 2],
                                                                x[..., rot // 2:rot])
    s = np.abs(a) + np.abs(b)
    if adjacent:
        size[..., 0:rot:2] = size[..., 1:rot:2] = s
    else:
        size[..., :rot // 2] = size[..., rot // 2:rot] = s
    tol = (torch.finfo(dt).eps / 2 * np.abs(exact) + size * abs(amplitude) * 2.0 ** -21
           + (2.0 ** -25 if dt == torch.float16 else 0.0))
    off = np.abs(got.double().cpu().numpy() - exact)
    assert (off <= tol).all(), (off / np.maximum(tol, 1e-300)).max()
    # what is not turned passes through to the bit
    assert np.array_equal(got.double().cpu().numpy()[..., rot:], x[..., rot:])


def run(n, h, hk, d, dtype, bs, rot, sections, adjacent, base=1e4, pos=None, packed=False,
        shift=0, amplitude=1.0, in_place=False, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed + n)
    t = TYPES[dtype]
    if packed:
        width = (h + 2 * hk) * d
        flat = torch.randn(n * width + shift, generator=g, device=DEV).to(t)
        rows = flat.as_strided((n, h + 2 * hk, d), (width, d, 1), shift)
        q, k, v = rows[:, :h], rows[:, h:h + hk], rows[:, h + hk:]
    else:
        q, k, v = (torch.randn(n, m, d, generator=g, device=DEV).to(t) for m in (h, hk, hk))
    q0, k0, v0 = q.clone(), k.clone(), v.clone()
    inv = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    axes = [a for a, m in enumerate(sections) for _ in range(m)]
    if pos is None:
        pos = np.random.default_rng(n).integers(0, 5000, (len(sections), n)).astype(np.int32)
    r = pk.Rotary(d, rotary_dim=rot, base=base, sections=sections, adjacent=adjacent,
                  amplitude=amplitude)
    nb = -(-n // bs) + 1
    slots = torch.randperm(nb * bs, generator=torch.Generator().manual_seed(n))[:n].int()
    slots[3::7] = -1
    kc, vc = (torch.full((nb, bs, hk, d), 9.0, dtype=t, device=DEV) for _ in range(2))
    q_out = q if in_place else torch.full((n, h, d), float("nan"), dtype=t, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    p = torch.from_numpy(pos).to(DEV)
    got = pk.pa_rotary_store(q_out, q, k, v, p, r, kc, vc, slots.to(DEV), dev_err=err)
    assert got is q_out and err.item() == 0
    if not in_place:
        assert torch.equal(q, q0)
    assert torch.equal(k, k0) and torch.equal(v, v0)
    check(q_out, q0, pos, r, inv, axes, adjacent, amplitude)
    kept = [i for i in range(n) if slots[i] >= 0]
    rows = slots[kept].long().to(DEV)
    if kept:
        check(kc.view(-1, hk, d)[rows], k0[kept], pos[:, kept], r, inv, axes, adjacent, amplitude)
        assert torch.equal(vc.view(-1, hk, d)[rows], v0[kept])
    rest = torch.ones(nb * bs, dtype=torch.bool, device=DEV)
    rest[rows] = False
    assert bool((kc.view(-1, hk, d)[rest] == 9.0).all() and (vc.view(-1, hk, d)[rest] == 9.0).all())
    # the 8-bit form: bit for bit the rotary store and then the quantising store
    for fmt in ref.FORMATS.values():
        one, two = (pk.Q8Cache(nb, bs, hk, d, fmt) for _ in range(2))
        q2 = torch.empty(n, h, d, dtype=t, device=DEV)
        pk.pa_rotary_store_q8(q2, q0, k, v, p, r, one, slots.to(DEV), dev_err=err)
        turned = torch.zeros(n, hk, d, dtype=t, device=DEV)
        if kept:
            turned[kept] = kc.view(-1, hk, d)[rows]
        pk.pa_store_kvcache_q8(turned, v, two, slots.to(DEV))
        assert torch.equal(q2, q_out)
        for x, y in ((one.k, two.k), (one.v, two.v), (one.k_scale, two.k_scale),
                     (one.v_scale, two.v_scale)):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert err.item() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("d,rot,sections", [(128, 128, (64,)), (128, 128, (16, 24, 24)),
                                            (128, 32, (3, 13)), (64, 64, (8, 12, 12)),
                                            (64, 16, (8,)), (64, 48, (1, 2, 21)),
                                            (128, 112, (0, 56)), (128, 16, (2, 2, 2, 2))])
def test_forms(dtype, adjacent, d, rot, sections):
    run(45, 16, 8, d, dtype, 16, rot, sections, adjacent)


@pytest.mark.parametrize("n,h,hk,bs", [(1, 16, 8, 16), (1, 1, 1, 1), (2, 7, 3, 20), (300, 64, 1, 256),
                                       (33, 5, 16, 8), (4000, 4, 2, 64)])
@pytest.mark.parametrize("d", [64, 128])
def test_shapes(n, h, hk, bs, d):
    run(n, h, hk, d, "bf16", bs, d, (d // 4, d // 4), False)


@pytest.mark.parametrize("n", [1, 7, 64, 129, 1500])
@pytest.mark.parametrize("h,hk", [(1, 1), (2, 1), (3, 3), (8, 1), (9, 2), (16, 3), (7, 5), (40, 2),
                                  (12, 7), (2, 8), (1, 16)])
@pytest.mark.parametrize("d,adjacent", [(64, True), (128, False)])
def test_few_heads(n, h, hk, d, adjacent):
    """Head counts below, at and above a work item's, for queries and for keys."""
    run(n, h, hk, d, "fp16" if adjacent else "bf16", 16, d // 2, (3, d // 4 - 3), adjacent)


def test_few_heads_packed_in_place():
    run(300, 3, 2, 64, "bf16", 16, 64, (32,), False, packed=True, shift=1, in_place=True)
    run(300, 1, 1, 128, "fp16", 16, 128, (30, 34), True, packed=True, shift=0, in_place=True)


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("shift,d", [(0, 128), (8, 64), (1, 128), (3, 64)])
@pytest.mark.parametrize("in_place", [False, True])
def test_packed_projections(adjacent, shift, d, in_place):
    run(50, 12, 4, d, "bf16", 16, d // 2, (d // 8, d // 8), adjacent, packed=True, shift=shift,
        in_place=in_place)


def test_far_positions():
    pos = np.array([[0, 1, -1, 2 ** 31 - 1, -2 ** 31, 10 ** 9, 123456789, -987654321, 1 << 30,
                     (1 << 30) + 1]], dtype=np.int32)
    for base in (1e4, 1e6):
        run(10, 16, 8, 128, "fp16", 16, 128, (64,), False, base=base, pos=pos)
        run(10, 16, 8, 128, "bf16", 16, 128, (64,), True, base=base, pos=pos, amplitude=-1.25)


def test_amplitude():
    run(20, 8, 8, 64, "fp16", 16, 64, (32,), False, amplitude=0.5)
    run(20, 8, 8, 64, "bf16", 16, 64, (32,), False, amplitude=1.4142)


def test_positions_as_views():
    """One axis as [N], an axis stride above N, and one row for every axis (stride 0)."""
    n, h, hk, d = 30, 8, 4, 64
    q, k = torch.randn(n, h, d, device=DEV).bfloat16(), torch.randn(n, hk, d, device=DEV).bfloat16()
    slots = torch.arange(n, dtype=torch.int32, device=DEV)
    pos = torch.randint(0, 1000, (n,), dtype=torch.int32, device=DEV)
    wide = torch.randint(0, 1000, (3, n + 11), dtype=torch.int32, device=DEV)

    def call(r, p):
        kc, vc = (torch.zeros(2, 16, hk, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        out = pk.pa_rotary_store(torch.empty_like(q), q, k, k, p, r, kc, vc, slots)
        return torch.cat([out.flatten(), kc.flatten(), vc.flatten()])

    one, three = pk.Rotary(d), pk.Rotary(d, sections=(8, 12, 12))
    assert torch.equal(call(one, pos), call(one, pos[None]))
    assert torch.equal(call(one, pos), call(three, pos.expand(3, n)))
    assert torch.equal(call(three, wide[:, :n]), call(three, wide[:, :n].contiguous()))


def test_bad_axes_and_slots():
    n, h, hk, d = 5, 4, 2, 64
    q, k = torch.randn(n, h, d, device=DEV).bfloat16(), torch.randn(n, hk, d, device=DEV).bfloat16()
    kc, vc = (torch.zeros(2, 16, hk, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    slots = torch.tensor([0, 32, 1, -1, -5], dtype=torch.int32, device=DEV)
    pos = torch.arange(2 * n, dtype=torch.int32, device=DEV).view(2, n)
    r = pk.Rotary(d, sections=(16, 16))
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pk.pa_rotary_store(torch.empty_like(q), q, k, k, pos, r, kc, vc, slots, dev_err=err)
    assert err.item() == pk.PA_DEV_ERR["slot"]
    assert torch.equal(vc.view(-1, hk, d)[:2], k[[0, 2]]) and not bool(vc.view(-1, hk, d)[2:].any())
    r.axes[3], r.axes[9] = 2, -1  # such pairs turn by axis 0
    err.zero_()
    out = pk.pa_rotary_store(torch.empty_like(q), q, k, k, pos, r, kc, vc, slots, dev_err=err)
    assert err.item() == pk.PA_DEV_ERR["slot"] | pk.PA_DEV_ERR["axis"]
    r.axes[3] = r.axes[9] = 0
    assert torch.equal(out, pk.pa_rotary_store(torch.empty_like(q), q, k, k, pos, r, kc, vc, slots))


def test_refusals():
    n, h, hk, d = 4, 8, 4, 64
    t = dict(q_out=torch.empty(n, h, d, device=DEV).bfloat16(),
             q=torch.randn(n, h, d, device=DEV).bfloat16(),
             k=torch.randn(n, hk, d, device=DEV).bfloat16(),
             v=torch.randn(n, hk, d, device=DEV).bfloat16(),
             positions=torch.zeros(1, n, dtype=torch.int32, device=DEV), rotary=pk.Rotary(d),
             slot_mapping=torch.zeros(n, dtype=torch.int32, device=DEV))
    cache = dict(k_cache=torch.zeros(2, 16, hk, d, device=DEV).bfloat16(),
                 v_cache=torch.zeros(2, 16, hk, d, device=DEV).bfloat16())
    q8 = dict(cache=pk.Q8Cache(2, 16, hk, d))
    for bad in (dict(q=t["q"].half()), dict(q_out=t["q_out"][:, :4]), dict(k=t["k"][:3]),
                dict(v=t["v"].float()), dict(positions=t["positions"].long()),
                dict(positions=t["positions"].expand(2, n)), dict(positions=t["positions"][:, :3]),
                dict(positions=torch.zeros(1, 2 * n, dtype=torch.int32, device=DEV)[:, ::2]),
                dict(rotary=pk.Rotary(128)), dict(rotary=None), dict(rotary=pk.Rotary(d, device="cpu")),
                dict(slot_mapping=t["slot_mapping"][:3]), dict(slot_mapping=t["slot_mapping"].cpu()),
                dict(q=t["q"].cpu()), dict(q_out=t["q_out"][:1].expand(n, h, d))):
        with pytest.raises(pk.PagedAttentionError):
            pk.pa_rotary_store(**(t | cache | bad))
        with pytest.raises(pk.PagedAttentionError):
            pk.pa_rotary_store_q8(**(t | q8 | bad))
    for bad in (dict(k_cache=cache["k_cache"].half()), dict(v_cache=cache["v_cache"][:1]),
                dict(k_cache=cache["k_cache"].cpu()), dict(v_cache=cache["v_cache"].float())):
        with pytest.raises(pk.PagedAttentionError):
            pk.pa_rotary_store(**(t | cache | bad))
