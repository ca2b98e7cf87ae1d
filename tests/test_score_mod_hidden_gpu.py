"""What pa_prefill_mod must not look at, and windows so long that they hide nothing, against the
plain 64-bit attention within the bound that its arithmetic implies (attention_reference.py)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_107_gb300 as pk
from paged_kv_cache_107_gb300 import workloads
from tests import attention_reference as ar
from tests import test_score_mod_gpu as base

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


def stored_case(cached, new, H, Hk, D, bs, dtype, seed):
    """A prefill case whose new tokens are in the caches."""
    case = workloads.prefill_case(cached, new, H, Hk, D, bs, seed=seed, dtype=dtype)
    slots = torch.from_numpy(case.slot_mapping.astype(np.int64))
    case.k_cache.view(-1, Hk, D)[slots] = case.k_new
    case.v_cache.view(-1, Hk, D)[slots] = case.v_new
    return case


def run(case, rule, causal=True, mod=None):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(case.q, float("nan"), device="cuda")
    pk.pa_prefill_mod(out, case.q.cuda(), case.k_cache.cuda(), case.v_cache.cuda(),
                      torch.from_numpy(case.block_tables).cuda(),
                      torch.from_numpy(case.cu_seqlens_q).cuda(),
                      torch.from_numpy(case.cu_seqlens_k).cuda(), case.max_seqlen_q,
                      case.max_seqlen_k,
                      mod or base.make_mod(rule, case.num_heads, case.num_seqs), causal=causal,
                      dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0, f"device error bits {int(err.item())}"
    return out.float().cpu().double().numpy()


def expected(case, s, pos, rule, causal=True):
    """(reference, bound) of the queries of sequence s at positions pos."""
    c0, n = int(case.cu_seqlens_q[s]), int(np.diff(case.cu_seqlens_q)[s])
    total = int(np.diff(case.cu_seqlens_k)[s])
    rows = c0 + np.asarray(pos) - (total - n)
    see = ar.visible(pos, total, causal, rule.get("window", 0), rule.get("sink", 0),
                     rule.get("prefix") or 0)
    r, A, dev = ar.attend(case.q[rows].double().numpy(),
                          ar.gather(case.k_cache, case.block_tables[s], total),
                          ar.gather(case.v_cache, case.block_tables[s], total), pos, see,
                          softcap=rule.get("softcap", 0.0),
                          slopes=base.slopes_of(case.num_heads, rule.get("bias")))
    return rows, r, ar.bound(r, A, dev, case.q.dtype)


@pytest.mark.parametrize("rule", ["none", "cap", "bias", "sink", "prefix", "all"])
@pytest.mark.parametrize("H,Hk,D,bs,dtype", [(4, 2, 128, 16, BF), (8, 1, 64, 64, FP),
                                             (2, 2, 128, 128, FP), (4, 1, 64, 8, BF)])
def test_keys_after_a_units_last_query_may_hold_anything(rule, H, Hk, D, bs, dtype):
    """A unit is 256 / G positions (G heads per KV head). NaN and infinities in every key and
    value that comes after one unit's last query (and behind the prefix) must not reach the
    queries up to there, although the unit's last key tile holds some of them."""
    rule = base.RULES[rule]
    per_unit, cached, new = 2 * (128 // (H // Hk)), 101, 400
    for last in range(per_unit, new, per_unit):  # new tokens of the units up to this one
        case = stored_case([cached], [new], H, Hk, D, bs, dtype, seed=3000 + last)
        end = max(cached + last, rule.get("prefix") or 0)
        for i, t in enumerate(range(end, cached + new)):
            blk = int(case.block_tables[0, t // bs])
            case.k_cache[blk, t % bs] = float("nan")
            case.v_cache[blk, t % bs] = (float("nan"), float("inf"), -float("inf"))[i % 3]
        rows, ref, tol = expected(case, 0, np.arange(cached, cached + last), rule)
        ar.assert_within(run(case, rule)[rows], ref, tol, f"{rule}, first {last} queries")


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 100, 2 ** 31 - 400])
@pytest.mark.parametrize("rule", ["none", "cap", "bias", "all"])
@pytest.mark.parametrize("H,Hk,D,dtype", [(4, 2, 128, BF), (8, 1, 64, FP)])
def test_the_longest_windows_hide_nothing_after_the_query(window, rule, H, Hk, D, dtype):
    """Keys after the query, seen because the call is not causal or through the prefix, under a
    window that reaches back past the start of every sequence."""
    cached, new = [0, 50], [140, 300]
    case = stored_case(cached, new, H, Hk, D, 16, dtype, seed=3100)
    for causal, prefix in ((False, 0), (True, 120)):
        r = dict(base.RULES[rule], window=window, sink=0, prefix=prefix)
        got = run(case, r, causal)
        for s, (c, n) in enumerate(zip(cached, new)):
            rows, ref, tol = expected(case, s, np.arange(c, c + n), r, causal)
            ar.assert_within(got[rows], ref, tol, f"{r} causal {causal}")


@pytest.mark.parametrize("rule", ["none", "cap", "bias", "sink", "prefix", "all"])
@pytest.mark.parametrize("D,dtype", [(128, BF), (64, FP)])
def test_short_units_after_long_ones_with_one_row_tile(rule, D, dtype):
    """Several units for each CTA, the heaviest first: 16 key tiles for the first row tile alone, so
    that the second one's rows sit out many phases of the V ring, then units of both row tiles
    whose first key tile already holds rows to be left out."""
    H, Hk, bs, rule = 16, 8, 16, base.RULES[rule]
    rng = np.random.default_rng(3200)
    n = 30
    new = rng.integers(1, 6, n).tolist() + rng.integers(65, 128, n).tolist()
    case = stored_case([2000] * n + [0] * n, new, H, Hk, D, bs, dtype, seed=3201)
    got = run(case, rule)
    for s in [0, 7, n - 1] + list(range(n, 2 * n)):
        total = int(np.diff(case.cu_seqlens_k)[s])
        rows, ref, tol = expected(case, s, np.arange(total - new[s], total), rule)
        ar.assert_within(got[rows], ref, tol, f"{rule} sequence {s}")
