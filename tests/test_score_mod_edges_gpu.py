"""The ends of what pa_decode_mod, pa_prefill_mod and pa_decode_shared accept: caps and windows
at the limits of their types, biases that grow with the distance, pools past 2^31 elements,
replayed captures, empty batches, and views that the calls refuse."""
import numpy as np
import pytest
import torch

import paged_kv_cache_107_gb300 as pk
from paged_kv_cache_107_gb300 import workloads
from tests import attention_reference as ar
from tests import test_score_mod_gpu as base
from tests.gpu_helpers import DeviceCase
from tests.test_large_pool_gpu import relocate

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cap", [1e-6, 1e-3, 1e30])
@pytest.mark.parametrize("gain", [0.0, 3.0])
def test_caps_near_the_ends_of_fp32(cap, gain, monkeypatch):
    """A tiny cap brings every score near 0; a huge one changes nothing, and the results are held
    against the formula without one."""
    make = base.make_mod
    monkeypatch.setattr(base, "make_mod", lambda r, H, S: make(dict(r, softcap=cap), H, S))
    rule = dict(softcap=cap) if cap < 1 else dict()
    base.decode_check([1, 40, 300], 16, 8, 128, 16, torch.bfloat16, rule, seed=2000, q_gain=gain)
    base.prefill_check([0, 50], [140, 200], 8, 2, 64, 16, torch.float16, rule, seed=2001,
                       q_gain=gain)
    base.prefill_check([0, 50], [140, 200], 8, 2, 128, 16, torch.bfloat16, dict(rule, bias=True),
                       seed=2002, q_gain=gain)


def test_bias_that_grows_with_the_distance(monkeypatch):
    """Slopes of either sign, and of 0: the far keys weigh most, and the running maximum moves at
    nearly every tile."""
    monkeypatch.setattr(base, "slopes_of", lambda H, bias: np.linspace(-0.5, 0.5, H + 1)[:H]
                        .astype(np.float32))
    base.decode_check([1, 130, 900], 16, 8, 128, 16, torch.bfloat16, dict(bias=True), seed=2010)
    base.prefill_check([0, 300], [400, 260], 8, 2, 128, 16, torch.bfloat16, dict(bias=True),
                       seed=2011)
    base.prefill_check([0, 300], [400, 260], 8, 2, 64, 16, torch.float16, dict(bias=True),
                       seed=2012, causal=False)


@pytest.mark.parametrize("rule", [dict(window=2 ** 31 - 1), dict(window=1, sink=2 ** 31 - 1),
                                  dict(window=5, prefix=2 ** 31 - 1), dict(prefix=-(2 ** 31))])
def test_rules_at_the_ends_of_int32(rule, monkeypatch):
    """Windows, sinks and prefixes beyond every sequence hide nothing; a negative prefix is 0."""
    seen = dict(rule, prefix=max(0, rule.get("prefix", 0)))  # what the rules come to
    make = base.make_mod
    monkeypatch.setattr(base, "make_mod", lambda r, H, S: make(rule, H, S))
    base.decode_check([1, 40, 300], 16, 8, 128, 16, torch.bfloat16, seen, 2020)
    base.prefill_check([0, 50], [140, 300], 8, 2, 128, 16, torch.bfloat16, seen, 2021)


def test_pools_past_2_31_elements():
    """The same bits as with the blocks at the start of the pool."""
    H, Hk, D, bs = 16, 8, 128, 256
    mod = base.make_mod(base.RULES["all"], H, 4)
    case = workloads.decode_case([1, 257, 2048, 3000], H, Hk, D, bs, seed=2030)
    starts = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    outs = []
    for far in (False, True):
        dc, first = relocate(case) if far else (DeviceCase(case), 0)
        dc.store()
        if not far:
            # one group that shares real blocks: sequence 2's first six are sequence 3's too
            case.block_tables[3, :6] = case.block_tables[2, :6]
        bt = torch.from_numpy(case.block_tables).cuda()
        bt[bt >= 0] += first
        prefix = torch.tensor([0, 1536], dtype=torch.int32, device="cuda")
        a = pk.pa_decode_mod(torch.empty_like(dc.q), dc.q, dc.k_cache, dc.v_cache, bt, dc.ctx, mod,
                             dev_err=dc.err)
        s = pk.pa_decode_shared(torch.empty_like(dc.q), dc.q, dc.k_cache, dc.v_cache, bt, dc.ctx,
                                starts, prefix, dev_err=dc.err)
        assert dc.dev_err() == 0
        outs.append((a, s))
        del dc
    for x, y in zip(*outs):
        assert torch.isfinite(x.float()).all()
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))
    case = workloads.prefill_case([0, 300, 1000], [129, 77, 260], H, Hk, D, bs, seed=2031)
    mod = base.make_mod(base.RULES["all"], H, 3)
    outs = []
    for far in (False, True):
        dc, _ = relocate(case) if far else (DeviceCase(case), 0)
        dc.store()
        outs.append(pk.pa_prefill_mod(
            torch.empty_like(dc.q), dc.q, dc.k_cache, dc.v_cache, dc.bt,
            torch.from_numpy(case.cu_seqlens_q).cuda(), torch.from_numpy(case.cu_seqlens_k).cuda(),
            case.max_seqlen_q, case.max_seqlen_k, mod, dev_err=dc.err))
        assert dc.dev_err() == 0
        del dc
    assert torch.isfinite(outs[0].float()).all()
    assert torch.equal(outs[0].view(torch.int16), outs[1].view(torch.int16))


@pytest.mark.parametrize("rule", ["cap", "bias", "prefix_window"])
def test_prefill_capture_and_replay(rule):
    """A captured prefill replayed after its lengths, prefixes and queries have changed."""
    H, Hk, D, bs = 8, 2, 128, 16
    case = workloads.prefill_case([200, 200], [128, 128], H, Hk, D, bs, seed=2040, poison=False)
    mod = base.make_mod(dict(base.RULES[rule], prefix=0), H, 2)
    k, v, q = case.k_cache.cuda(), case.v_cache.cuda(), case.q.cuda()
    slots = torch.from_numpy(case.slot_mapping.astype(np.int64)).cuda()
    k.view(-1, Hk, D)[slots], v.view(-1, Hk, D)[slots] = case.k_new.cuda(), case.v_new.cuda()
    bt = torch.from_numpy(case.block_tables).cuda()
    cq = torch.tensor([0, 128, 256], dtype=torch.int32, device="cuda")
    ck = torch.tensor([0, 328, 656], dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)

    def call(o):
        return pk.pa_prefill_mod(o, q, k, v, bt, cq, ck, 256, 328, mod)

    call(out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(out)
    for lens_q, lens_k, prefix in (([128, 128], [328, 328], [0, 0]), ([1, 255], [130, 300], [100, 7]),
                                   ([256, 0], [256, 0], [0, 40])):
        cq.copy_(torch.tensor([0] + list(np.cumsum(lens_q)), dtype=torch.int32))
        ck.copy_(torch.tensor([0] + list(np.cumsum(lens_k)), dtype=torch.int32))
        mod.prefix_lens.copy_(torch.tensor(prefix, dtype=torch.int32))
        q.mul_(-1)
        g.replay()
        want = call(torch.empty_like(q))
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))
        at = 0
        for s, (n, total) in enumerate(zip(lens_q, lens_k)):
            if n == 0:
                continue
            pos = np.arange(total - n, total)
            r = base.RULES[rule]
            see = ar.visible(pos, total, True, r.get("window", 0), r.get("sink", 0), prefix[s])
            ref, A, dev = ar.attend(q[at:at + n].cpu().double().numpy(),
                                    ar.gather(k.cpu(), case.block_tables[s], total),
                                    ar.gather(v.cpu(), case.block_tables[s], total), pos, see,
                                    softcap=r.get("softcap", 0.0),
                                    slopes=base.slopes_of(H, r.get("bias")))
            ar.assert_within(out[at:at + n].float().cpu().double().numpy(), ref,
                             ar.bound(ref, A, dev, torch.bfloat16), f"{rule} {lens_q} {s}")
            at += n


def test_empty_batches_and_views():
    H, Hk, D, bs = 8, 2, 128, 16
    case = workloads.decode_case([40, 300], H, Hk, D, bs, seed=2050, poison=False)
    q, k, v = case.q.cuda(), case.k_cache.cuda(), case.v_cache.cuda()
    bt = torch.from_numpy(case.block_tables).cuda()
    ctx = torch.from_numpy(case.context_lens).cuda()
    ints = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 2], [16])]
    mod = pk.ScoreMod(softcap=30.0)
    calls = {
        "decode_mod": lambda o, q, bt=bt, ctx=ctx: pk.pa_decode_mod(o, q, k, v, bt, ctx, mod),
        "shared": lambda o, q, bt=bt, ctx=ctx: pk.pa_decode_shared(o, q, k, v, bt, ctx, *ints),
        "prefill_mod": lambda o, q, bt=bt, ctx=ctx: pk.pa_prefill_mod(
            o, q, k, v, bt, torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda"),
            torch.tensor([0, 40, 340], dtype=torch.int32, device="cuda"), 1, 300, mod),
    }
    wide = torch.zeros(2, 2 * H, D, dtype=q.dtype, device="cuda")
    for name, call in calls.items():
        call(torch.empty_like(q), q)
        with pytest.raises(pk.PagedAttentionError):  # every other head of a wider tensor
            call(torch.empty_like(q), wide[:, ::2])
        with pytest.raises(pk.PagedAttentionError):
            call(wide[:, :H], q)
        with pytest.raises(pk.PagedAttentionError):
            call(torch.empty_like(q), q.float())
        with pytest.raises(pk.PagedAttentionError):
            call(torch.empty_like(q), q, bt=bt.t().contiguous().t())
        with pytest.raises(pk.PagedAttentionError):
            call(torch.empty_like(q), q, bt=bt.long())
    none = q[:0]
    assert pk.pa_decode_mod(none, none, k, v, bt[:0], ctx[:0], mod).shape[0] == 0
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert pk.pa_prefill_mod(none, none, k, v, bt[:0], zero, zero, 0, 0, mod).shape[0] == 0
    assert pk.pa_decode_shared(none, none, k, v, bt[:0], ctx[:0], zero, zero[:0]).shape[0] == 0
    torch.cuda.synchronize()
