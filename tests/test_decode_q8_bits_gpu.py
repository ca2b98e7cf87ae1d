"""pa_decode_q8 where few bits decide: bounds of each sequence and head alone, without the slack of
test_decode_q8_gpu (whose value and key scales are the batch's largest)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_107_gb300 as pk
from tests import attention_reference as att
from tests import q8_reference as ref
from tests.test_decode_q8_gpu import CODE_MAX, DEV, Case

pytestmark = pytest.mark.gpu


def reference(case, scale=None):
    """(out, tolerance). attention_reference's deviation of the scores (their products are exact,
    the sums fp32); each weight is held in two fp16 numbers, 2^-22 relative or 2^-39 of the largest
    value scale that the sequence holds for the head, times a code; the fp32 sums over the keys
    take two MMAs for every 16 keys, and the parts of a sequence, at most 2^-23 of A each
    (16 of them here); the output is rounded once to its type."""
    k = ref.dequantised(case.cache.k, case.cache.k_scale)
    v = ref.dequantised(case.cache.v, case.cache.v_scale)
    vs = case.cache.v_scale.cpu().double().transpose(1, 2).reshape(-1, case.Hk).numpy()
    q = case.q.double().cpu().numpy()
    least = 2.0 ** -25 if case.dtype == torch.float16 else 2.0 ** -134  # half a subnormal's step
    out, tol = np.zeros(q.shape), np.full(q.shape, least)
    half = torch.finfo(case.dtype).eps / 2
    for b, n in enumerate(case.lens):
        if n == 0:
            continue
        t = np.arange(n)
        rows = np.asarray(case.tables[b])[t // case.bs].astype(np.int64) * case.bs + t % case.bs
        o, A, dev = att.attend(q[b:b + 1], k[rows], v[rows], [n - 1], np.ones((1, n), bool),
                               scale=scale)
        top = np.repeat(vs[rows].max(0), q.shape[1] // case.Hk)[None, :, None]
        weights = (2.0 ** -22 + (n / 8 + 16) * 2.0 ** -23) * A
        weights = weights + n * CODE_MAX[case.fmt] * 2.0 ** -39 * top
        out[b] = o[0]
        tol[b] += (half * np.abs(o) + (1 + half) * (weights + np.expm1(2 * dev) * A))[0]
    return out, tol


def check(case, scale=None):
    out = case.run(scale=scale)
    att.assert_within(out.double().cpu().numpy(), *reference(case, scale))
    assert case.err.item() == 0
    return out


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D,Hk", [(128, 8), (64, 8), (64, 1), (128, 2)])
def test_int8_scores_of_queries_with_a_mean(dtype, D, Hk):
    """Queries far from zero mean over keys with one large element, which the query ignores, and
    small ones: sums of code times query are a thousandth of what 128 times the query's sum is."""
    case = Case([1 + b % 7 for b in range(48)], Hk * 2, Hk, D, "int8", dtype, 16, seed=D)
    codes = torch.randint(-1, 2, case.cache.k.shape, generator=case.g, device=DEV)
    codes[..., 0] = 127
    case.cache.k.copy_(codes)
    case.cache.k_scale.fill_(0.125)
    case.q.copy_(8 + torch.randn(case.q.shape, generator=case.g, device=DEV))
    case.q[..., 0] = 0.0
    check(case, scale=0.125)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D,Hk,G", [(128, 8, 2), (64, 8, 4), (64, 1, 8), (128, 3, 1)])
def test_results_are_rounded_once(fmt, dtype, D, Hk, G):
    """Scores near each other: nothing but the output's rounding is seen."""
    check(Case([1 + 3 * b for b in range(20)], Hk * G, Hk, D, fmt, dtype, 16, seed=G), scale=1e-3)
    check(Case([700, 33], Hk * G, Hk, D, fmt, dtype, 16, seed=G), scale=1e-3)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D,Hk", [(128, 8), (64, 8), (64, 1)])
@pytest.mark.parametrize("scale", [2.0 ** 18, 2.0 ** 22 * 1.3, 2.0 ** 30, 2.0 ** 60])
def test_scores_beyond_their_own_precision(fmt, dtype, D, Hk, scale):
    """A sequence of equal keys weighs them equally, whatever the size of their score and however
    coarse an fp32 number of that size is. Where CTAs share a sequence, each one's log-sum-exp
    m + log2 l is rounded at m's size: half a unit u of the last place, so that the weights of two of
    them move by up to 2^u against each other and the result by (2^u - 1) A, or at most from
    one value to another."""
    case = Case([1 + b % 40 for b in range(60)], Hk * 2, Hk, D, fmt, dtype, 16, seed=Hk)
    case.cache.k.view(torch.uint8).copy_(torch.randint(
        1, 100, (1, 1, Hk, D), generator=case.g, device=DEV).to(torch.uint8))
    case.cache.k_scale.fill_(0.01)
    out, alone = case.run(scale=scale), case.run(scale=scale, grid_ctas=1)
    key = np.repeat(ref.dequantised(case.cache.k, case.cache.k_scale)[0], 2, axis=0)
    m = np.abs((case.q.double().cpu().numpy() * key).sum(-1, keepdims=True)) * scale * np.log2(np.e)
    u = np.spacing((m + 6.0).astype(np.float32)).astype(np.float64)  # log2 40 < 6
    case.q.zero_()  # what equal weights give
    want, tol = reference(case)
    att.assert_within(alone.double().cpu().numpy(), want, tol)
    v = ref.dequantised(case.cache.v, case.cache.v_scale)
    far = 2.0 * np.nanmax(np.abs(v))
    att.assert_within(out.double().cpu().numpy(), want,
                      tol + np.minimum(np.exp2(np.minimum(u, 64.0)) - 1.0, 1.0) * far)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("D,Hk", [(128, 8), (64, 1)])
@pytest.mark.parametrize("up", [60, 100, 112])
def test_large_keys_under_small_queries(fmt, D, Hk, up):
    """bf16 keys 2^up times the usual size under queries as much smaller: ordinary scores."""
    case = Case([40, 7, 300], Hk * 2, Hk, D, fmt, "bf16", 16, seed=up)
    case.cache.k_scale.mul_(2.0 ** up)
    case.q *= 2.0 ** -up
    check(case, scale=0.25)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_a_sequence_is_not_bound_by_anothers_scales(fmt, dtype):
    """One sequence's value scales near fp32's largest leave the others' bits as they were."""
    case = Case([40, 70, 0, 33], 16, 8, 64, fmt, dtype, 16, seed=6)
    clean = check(case)
    for i, n in enumerate((16, 16, 16, 16, 6)):
        case.cache.v_scale[case.tables[1][i], :, :n] = 2.0 ** 110
    out = case.run()
    assert torch.equal(out[[0, 2, 3]], clean[[0, 2, 3]])
    if dtype == "bf16":
        att.assert_within(out.double().cpu().numpy(), *reference(case))
    for grid in (1, 2, 5):
        got, want = (case.run(grid_ctas=grid), reference(case))
        keep = [0, 2, 3]
        att.assert_within(got[keep].double().cpu().numpy(), want[0][keep], want[1][keep])


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D,Hk", [(128, 8), (64, 2)])
def test_rows_of_very_different_sizes(fmt, dtype, D, Hk):
    check(Case([300, 1, 77, 500], Hk * 4, Hk, D, fmt, dtype, 16, seed=5, spread=8), scale=1e-4)
