"""Seeded random shapes of the 8-bit cache's and the rotary calls against their definitions."""
import random

import pytest
import torch

import paged_kv_cache_107_gb300 as pk
from tests import q8_reference as ref
from tests import test_rotary_gpu as rotary
from tests.test_decode_q8_gpu import Case
from tests.test_q8_store_gpu import TYPES, check_store, new_cache

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("seed", range(30))
def test_decode(seed):
    rng = random.Random(seed)
    hk = rng.choice([1, 2, 3, 4, 5, 6, 8, 8, 10, 12, 16, 24])
    g = rng.randint(1, 8)
    d = rng.choice([64, 128])
    lens = [rng.choice([0, 1, rng.randint(1, 70), rng.randint(1, 3000 // hk + 50)])
            for _ in range(rng.randint(1, 40))]
    case = Case(lens, hk * g, hk, d, rng.choice(["e4m3", "int8"]), rng.choice(["bf16", "fp16"]),
                rng.choice([1, 2, 8, 12, 16, 24, 32, 64, 100, 128, 256, 1024]), seed=seed,
                spread=rng.choice([0, 0, 4]))
    case.check(grid_ctas=rng.choice([0, 0, 1, rng.randint(2, 400)]),
               scale=rng.choice([None, 0.05, 0.2]))


@pytest.mark.parametrize("seed", range(30))
def test_store(seed):
    rng = random.Random(100 + seed)
    hk, d = rng.randint(1, 20), rng.choice([64, 128])
    n, bs = rng.randint(1, 300), rng.choice([1, 3, 8, 16, 48, 256])
    fmt, t = rng.choice(["e4m3", "int8"]), TYPES[rng.choice(["bf16", "fp16"])]
    g = torch.Generator(device=DEV).manual_seed(seed)
    lead, tail, shift = rng.randint(0, 3), rng.choice([0, 0, 1, 8]), rng.choice([0, 0, 1, 8])
    width = (lead + 2 * hk) * d + tail
    flat = (torch.randn(n * width + shift, generator=g, device=DEV)
            * 2.0 ** rng.randint(-10, 10)).to(t)
    rows = flat.as_strided((n, lead + 2 * hk, d), (width, d, 1), shift)
    k, v = rows[:, lead:lead + hk], rows[:, lead + hk:]
    nb = -(-n // bs) + rng.randint(0, 3)
    slots = torch.randperm(nb * bs, generator=torch.Generator().manual_seed(seed))[:n].int()
    for i in range(n):
        if rng.random() < 0.1:
            slots[i] = rng.choice([-1, -1, nb * bs, -5])
    cache = new_cache(nb, bs, hk, d, fmt)
    pk.pa_store_kvcache_q8(k, v, cache, slots.to(DEV))
    check_store(cache, k, v, slots.tolist(), fmt)


@pytest.mark.parametrize("seed", range(30))
def test_rotary(seed):
    rng = random.Random(200 + seed)
    d = rng.choice([64, 128])
    rot = rng.choice(range(16, d + 1, 16))
    sections, left = [], rot // 2
    for _ in range(rng.randint(0, 4)):
        sections.append(rng.randint(0, left))
        left -= sections[-1]
    packed = rng.random() < 0.5
    rotary.run(rng.randint(1, 400), rng.randint(1, 40), rng.randint(1, 20), d,
               rng.choice(["bf16", "fp16"]), rng.choice([1, 5, 16, 256]), rot,
               (*sections, left), rng.random() < 0.5, base=rng.choice([1e4, 1e6, 10.0]),
               packed=packed, shift=rng.choice([0, 1, 8]) if packed else 0,
               amplitude=rng.choice([1.0, 1.0, 0.7]), in_place=rng.random() < 0.3, seed=seed)
