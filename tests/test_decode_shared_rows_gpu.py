"""Every row of pa_decode_shared on the batches whose cuts between CTAs are most varied: the 64-bit
attention of all sequences, computed on the device, within the bound of attention_reference.py."""
import numpy as np
import pytest
import torch

import paged_kv_cache_107_gb300 as pk
from tests import attention_reference as ar
from tests.test_decode_shared_gpu import Shared

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


def expected(c, d):
    """(reference, bound) of all rows, as attention_reference.attend and bound make them."""
    q, k, v, tables = d[:4]
    G, (B, H, D) = c.H // c.Hk, q.shape
    out = torch.zeros(B, H, D, dtype=torch.float64, device="cuda")
    A, dev = torch.zeros_like(out), torch.zeros(B, H, 1, dtype=torch.float64, device="cuda")
    for b, n in enumerate(c.lens):
        if n == 0:
            continue
        t = torch.arange(n, device="cuda")
        rows = tables[b].long()[t // c.bs] * c.bs + t % c.bs
        kk = k.view(-1, c.Hk, D)[rows].double().permute(1, 2, 0)  # [Hk, D, n]
        vv = v.view(-1, c.Hk, D)[rows].double().permute(1, 0, 2)
        qq = q[b].double().view(c.Hk, G, D)
        x = qq @ kk * D ** -0.5
        mag = (qq.abs() @ kk.abs() * D ** -0.5).amax(-1, keepdim=True)
        top = x.abs().amax(-1, keepdim=True)
        dev[b] = (D * 2.0 ** -23 * mag + 2.0 ** -21 * (top + 1)).view(H, 1)
        w = torch.softmax(x, -1)
        out[b], A[b] = (w @ vv).view(H, D), (w @ vv.abs()).view(H, D)
    ref, A, dev = (x.cpu().numpy() for x in (out, A, dev))
    return ref, ar.bound(ref, A, dev, c.dtype)


def check(c):
    d = c.device()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = pk.pa_decode_shared(torch.full_like(d[0], float("nan")), *d, dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0, f"device error bits {int(err.item())}"
    ref, tol = expected(c, d)
    ar.assert_within(out.double().cpu().numpy(), ref, tol, f"{c.lens[:8]}")


def test_the_reference_is_the_plain_one():
    c = Shared([3, 2], [130, 40], [5, 1, 77, 9, 60], 6, 2, 64, 16, BF, seed=7000)
    for x, y in zip(expected(c, c.device()), c.reference()):
        np.testing.assert_allclose(x, y, rtol=1e-9, atol=1e-12)


@pytest.mark.parametrize("G", range(1, 9))
def test_row_tiles_of_every_group_size(G):
    P = 128 // G
    for n in (2, P - 1, P, P + 1, 2 * P + 3, 4 * P):
        check(Shared([n], [390 + n], [1 + (i * 7) % 40 for i in range(n)], 2 * G, 2,
                     64 if G % 2 else 128, 16, BF if n % 2 else FP, seed=7100 + 10 * G + n))


def test_hundreds_of_small_groups():
    rng = np.random.default_rng(7200)
    sizes = [2] * 400 + [3] * 30
    prefix = [int(x) for x in rng.integers(0, 300, len(sizes))]
    rest = [None if i % 97 == 96 else int(x)
            for i, x in enumerate(rng.integers(1, 30, sum(sizes)))]
    for g, at in enumerate(np.cumsum([0] + sizes[:-1])):  # a padding row may not lead a group
        rest[at] = rest[at] or 1
    check(Shared(sizes, prefix, rest, 8, 4, 64, 16, FP, seed=7201))


@pytest.mark.parametrize("sizes,prefix,H,Hk,D,bs", [
    ([9], [20000], 8, 2, 128, 64), ([150], [3000], 16, 8, 128, 16),
    ([130, 70, 2], [2600, 900, 5000], 16, 4, 64, 32), ([33, 64, 65], [4096, 128, 1111], 8, 8, 128, 16)])
def test_long_prefixes_cut_anywhere(sizes, prefix, H, Hk, D, bs):
    rest = [1 + i * 11 % 300 for i in range(sum(sizes))]
    check(Shared(sizes, prefix, rest, H, Hk, D, bs, BF, seed=7300 + sizes[0]))


@pytest.mark.parametrize("Hk", [155, 160])
def test_more_kv_heads_than_sms(Hk):
    check(Shared([5, 1], [400, 0], [3, 40, 1, 9, 100, 60], Hk, Hk, 64, 16, BF, seed=7400 + Hk))
