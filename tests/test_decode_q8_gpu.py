"""pa_decode_q8 on the GPU against attention in 64 bits over the values that the cache stands for,
within the bound of its roundings (q8_reference.decode)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_107_gb300 as pk
from tests import attention_reference as att
from tests import q8_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
CODE_MAX = {"e4m3": 448.0, "int8": 127.0}


class Case:
    """A batch over a shuffled pool. Everything that no sequence holds is poison: e4m3 NaN codes
    (int8: -128), NaN scales."""

    def __init__(self, lens, H, Hk, D, fmt, dtype, bs, seed=0, spread=0):
        self.g = torch.Generator(device=DEV).manual_seed(seed)
        self.lens, self.bs, self.fmt, self.dtype = lens, bs, fmt, TYPES[dtype]
        self.Hk, self.D = Hk, D
        need = [-(-n // bs) for n in lens]
        nb = sum(need) + 3
        order = np.random.default_rng(seed).permutation(nb).tolist()
        self.tables, at = [], 0
        width = max(need) + 2
        for k in need:
            self.tables.append(order[at:at + k] + [-1] * (width - k))
            at += k
        poison = 0x7f if fmt == "e4m3" else 0x80
        codes = [torch.full((nb * bs, Hk, D), poison, dtype=torch.uint8, device=DEV)
                 for _ in range(2)]
        scales = [torch.full((nb * bs, Hk), float("nan"), device=DEV) for _ in range(2)]
        rows = np.concatenate([np.asarray(self.tables[b])[np.arange(n) // bs] * bs
                               + np.arange(n) % bs for b, n in enumerate(lens)]).astype(np.int64)
        rows = torch.from_numpy(rows).to(DEV)
        for c, s in zip(codes, scales):
            x = torch.randn(len(rows), Hk, D, generator=self.g, device=DEV).double()
            if spread:  # rows of very different sizes
                x *= torch.exp2(torch.randint(-spread, spread + 1, (len(rows), Hk, 1),
                                              generator=self.g, device=DEV).double())
            y, z = ref.quantise(fmt, x.cpu().numpy())
            c[rows] = torch.from_numpy(y).float().to(ref.FORMATS[fmt]).view(torch.uint8).to(DEV)
            s[rows] = torch.from_numpy(z).float().to(DEV)
        self.cache = pk.Q8Cache.of(
            *(c.view(ref.FORMATS[fmt]).view(nb, bs, Hk, D) for c in codes),
            *(s.view(nb, bs, Hk).transpose(1, 2).contiguous() for s in scales))
        self.q = torch.randn(len(lens), H, D, generator=self.g, device=DEV).to(self.dtype)
        self.bt = torch.tensor(self.tables, dtype=torch.int32, device=DEV)
        self.ctx = torch.tensor(lens, dtype=torch.int32, device=DEV)
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)

    def run(self, **kw):
        out = torch.full_like(self.q, float("nan"))
        assert pk.pa_decode_q8(out, self.q, self.cache, self.bt, self.ctx, dev_err=self.err,
                               **kw) is out
        return out

    def reference(self, scale=None):
        k = ref.dequantised(self.cache.k, self.cache.k_scale)
        v = ref.dequantised(self.cache.v, self.cache.v_scale)
        top = float(self.cache.v_scale.nan_to_num(0.0).max())
        return ref.decode(self.q, k, v, top, self.tables, self.lens, self.bs, self.dtype, scale,
                          CODE_MAX[self.fmt], float(self.cache.k_scale.nan_to_num(0.0).max()))

    def check(self, what="", **kw):
        out = self.run(**kw)
        att.assert_within(out.double().cpu().numpy(), *self.reference(kw.get("scale")), what)
        assert self.err.item() == 0
        return out


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hk,G", [(8, 2), (8, 1), (4, 4), (2, 8), (1, 6), (3, 3), (16, 1), (12, 5),
                                  (1, 1)])
def test_heads(fmt, dtype, D, Hk, G):
    Case([1, 31, 32, 33, 0, 257, 600], Hk * G, Hk, D, fmt, dtype, 16, seed=Hk * G).check()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("D,Hk", [(128, 8), (64, 8), (64, 1), (128, 2)])
@pytest.mark.parametrize("bs", [1, 4, 8, 16, 20, 24, 48, 100, 256, 512])
def test_block_sizes(fmt, D, Hk, bs):
    Case([5, 64, 511, 1025, 100], Hk * 2, Hk, D, fmt, "bf16", bs, seed=bs).check()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("D", [64, 128])
def test_every_length_around_a_tile(fmt, D):
    T = 32 if D == 128 else 64  # tokens of a tile at 8 KV heads
    Case(list(range(2 * T + 2)), 16, 8, D, fmt, "fp16", 16, seed=T).check()
    Case([8 * T - 1, 8 * T, 8 * T + 1, 1], 2, 1, D, fmt, "bf16", 16, seed=T).check()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_long_contexts(fmt, dtype):
    Case([20000, 1, 4097], 16, 4, 128, fmt, dtype, 64, seed=3).check()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("Hk", [1, 8])
def test_rows_of_very_different_sizes(fmt, dtype, Hk):
    case = Case([300, 1000, 77], Hk * 4, Hk, 128, fmt, dtype, 16, seed=5, spread=8)
    case.check(scale=1e-4)  # scores near each other, values of sizes 2^-8 .. 2^8
    case.check(scale=0.05)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_scales_at_the_ends(fmt):
    """Zero rows, the least scales, and values near fp32's largest."""
    case = Case([40, 70], 16, 8, 64, fmt, "bf16", 16, seed=6)
    c = case.cache
    c.v_scale[case.tables[0][0]] = 0.0
    c.k_scale[case.tables[0][1]] = 0.0
    c.v_scale[case.tables[1][:2]] = 2.0 ** -126
    case.check()
    for b in case.tables[1][:5]:
        c.v_scale[b] = 2.0 ** 110  # (poison behind the context stays NaN below)
    c.v_scale[case.tables[1][4], :, 70 - 64:] = float("nan")
    case.check()
    for b in range(2):
        for i in range(-(-case.lens[b] // 16)):
            c.v_scale[case.tables[b][i]] = 0.0
    out = case.run()
    assert not bool(out.any())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_queries_of_any_size(dtype):
    for size in (2.0 ** -14, 1.0, 2.0 ** 10):
        case = Case([100, 33], 16, 8, 128, "e4m3", dtype, 16, seed=7)
        case.q *= size
        case.check(scale=0.02 / size)
    case = Case([50], 16, 8, 128, "int8", dtype, 16, seed=8)
    case.q[0, 3] = 0.0
    case.q[0, 5, 1:] = 0.0
    case.check()
    if dtype == "bf16":
        case.q *= 2.0 ** 100
        case.check(scale=2.0 ** -104)
        case.q *= 2.0 ** -100
        case.q *= 2.0 ** -120
        case.check(scale=2.0 ** 117)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("D", [64, 128])
def test_grids_and_repeats(fmt, D):
    case = Case([700, 3, 1500, 64, 0, 2100], 32, 8, D, fmt, "bf16", 16, seed=9)
    ws = pk.DecodeWorkspace(6, 32, 8, D)
    first = case.check(workspace=ws)
    for _ in range(3):
        assert torch.equal(case.run(workspace=ws), first)
    for grid in (1, 2, 7, 150, 301, 600):
        case.check(f"grid {grid}", grid_ctas=grid, workspace=ws)
    assert not bool(ws.buffer[-6 * 8 * 4:].any())  # the counters are zero again
    # a workspace for more sequences serves fewer
    big = pk.DecodeWorkspace(64, 32, 8, D)
    assert torch.equal(case.run(workspace=big), first)


@pytest.mark.parametrize("B", [255, 256, 257, 513, 900])
def test_many_sequences(B):
    """More sequences than the prologue scans at once, some of them empty."""
    rng = np.random.default_rng(B)
    lens = [int(n) if n % 7 else 0 for n in rng.integers(0, 90, B)]
    lens[0], lens[-1] = 0, 33
    case = Case(lens, 8, 4, 64, "int8", "bf16", 16, seed=B)
    case.check()
    case.check("one CTA", grid_ctas=1)
    case = Case([0] * (B - 1) + [200], 2, 1, 64, "e4m3", "fp16", 16, seed=B)  # the last alone
    case.check()


@pytest.mark.parametrize("D", [64, 128])
def test_many_heads(D):
    """More slabs (of one head) than SMs, and twenty slabs of eight."""
    Case([70, 0, 300], 153, 153, D, "e4m3", "bf16", 16, seed=153).check()
    Case([70, 1], 320, 160, D, "int8", "fp16", 16, seed=160).check()


def test_nan_in_a_held_row_reaches_its_sequence_only():
    case = Case([40, 600, 50], 16, 8, 128, "e4m3", "bf16", 16, seed=10)
    clean = case.run()
    c = case.cache
    c.k_scale[case.tables[1][3], 2, 5] = float("nan")
    out = case.run()
    assert bool(out[1, 4:6].isnan().all())
    out[1, 4:6] = clean[1, 4:6]
    assert torch.equal(out, clean)
    c.k_scale[case.tables[1][3], 2, 5] = 1.0
    c.v_scale[case.tables[0][0], 1, 0] = float("nan")
    out = case.run()
    assert bool(out[0, 2:4].isnan().all()) and not bool(out[2].isnan().any())
    # a row stored from a NaN reads back as NaN: one key, one sequence
    one = Case([1], 16, 8, 128, "int8", "bf16", 16, seed=11)
    x = torch.randn(1, 8, 128, device=DEV).bfloat16()
    x[0, 6, 9] = float("nan")
    slot = torch.tensor([one.tables[0][0] * 16], dtype=torch.int32, device=DEV)
    pk.pa_store_kvcache_q8(x, x, one.cache, slot)
    out = one.run()
    assert bool(out[0, 12:14].isnan().all()) and not bool(out[0, :12].isnan().any())


def test_bad_tables_and_lengths():
    case = Case([40, 100, 50], 16, 8, 128, "e4m3", "bf16", 16, seed=12)
    clean = case.run()
    case.bt[1, 2] = case.cache.k.shape[0]
    out = case.run()
    assert case.err.item() == pk.PA_DEV_ERR["block_id"]
    assert torch.equal(out[[0, 2]], clean[[0, 2]])
    case.bt[1, 2] = case.tables[1][2]
    for bad in (-1, case.bt.shape[1] * 16 + 1):
        case.err.zero_()
        case.ctx[1] = bad
        out = case.run()
        assert case.err.item() == pk.PA_DEV_ERR["context"]
        assert torch.equal(out[[0, 2]], clean[[0, 2]]) and not bool(out[1].any())


def test_empty_batches():
    case = Case([0, 0, 0], 16, 8, 64, "int8", "fp16", 16, seed=13)
    assert not bool(case.check().any())
    pk.pa_decode_q8(case.q[:0], case.q[:0], case.cache, case.bt[:0], case.ctx[:0])


def test_refusals():
    case = Case([20, 30], 16, 8, 64, "int8", "fp16", 16, seed=14)
    t = dict(out=torch.empty_like(case.q), q=case.q, cache=case.cache, block_tables=case.bt,
             context_lens=case.ctx)
    small = pk.DecodeWorkspace(1, 8, 8, 64)
    small.nbytes = 256
    for bad in (dict(q=case.q.float()), dict(out=case.q.bfloat16()), dict(q=case.q[:, :12]),
                dict(out=t["out"][:1]), dict(block_tables=case.bt.long()),
                dict(block_tables=case.bt[:1]), dict(context_lens=case.ctx[:1]),
                dict(context_lens=case.ctx.cpu()), dict(q=case.q.transpose(0, 1)),
                dict(cache=pk.Q8Cache(2, 16, 8, 128, torch.int8)),
                dict(cache=pk.Q8Cache(2, 16, 1, 64, torch.int8)), dict(cache=case.cache.k),
                dict(workspace=small), dict(grid_ctas=-1), dict(grid_ctas=100000),
                dict(cache=pk.Q8Cache(2, 16, 8, 64, torch.int8, device="cpu"))):
        with pytest.raises(pk.PagedAttentionError):
            pk.pa_decode_q8(**(t | bad))
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(pk.PagedAttentionError, match="workspace"):
        with torch.cuda.graph(graph):
            pk.pa_decode_q8(**t)


def test_large_pools():
    """Blocks whose codes start past 2^32 bytes, and slots near 2^31 / the head count."""
    hk, d, bs = 8, 128, 256
    nb = (1 << 32) // (bs * hk * d) + 40
    codes = [torch.empty(nb, bs, hk, d, dtype=torch.uint8, device=DEV).view(torch.int8)
             for _ in range(2)]
    scales = [torch.full((nb, hk, bs), float("nan"), device=DEV) for _ in range(2)]
    cache = pk.Q8Cache.of(*codes, *scales)
    n = 700
    table = [nb - 1, 3, nb - 30]
    slots = torch.tensor([table[i // bs] * bs + i % bs for i in range(n)], dtype=torch.int32,
                         device=DEV)
    k, v = (torch.randn(n, hk, d, device=DEV).bfloat16() for _ in range(2))
    pk.pa_store_kvcache_q8(k, v, cache, slots)
    small = pk.Q8Cache(3, bs, hk, d, torch.int8)
    pk.pa_store_kvcache_q8(k, v, small, torch.arange(n, dtype=torch.int32, device=DEV))
    q = torch.randn(1, 16, d, device=DEV).bfloat16()
    ctx = torch.tensor([n], dtype=torch.int32, device=DEV)
    a = pk.pa_decode_q8(torch.empty_like(q), q, cache,
                        torch.tensor([table], dtype=torch.int32, device=DEV), ctx)
    b = pk.pa_decode_q8(torch.empty_like(q), q, small,
                        torch.tensor([[0, 1, 2]], dtype=torch.int32, device=DEV), ctx)
    assert torch.equal(a, b)
    out = [torch.zeros(2, 3, bs, hk, d, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    pk.pa_load_kvcache_q8(out[0][0], out[0][1], cache,
                          torch.tensor(table, dtype=torch.int32, device=DEV))
    pk.pa_load_kvcache_q8(out[1][0], out[1][1], small,
                          torch.arange(3, dtype=torch.int32, device=DEV))
    assert torch.equal(out[0].view(2, -1, hk, d)[:, :n], out[1].view(2, -1, hk, d)[:, :n])
    del cache, codes, scales
    torch.cuda.empty_cache()
