"""pa_decode_mod and pa_prefill_mod against the plain 64-bit attention, within the bound that
their arithmetic implies (attention_reference.py)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_107_gb300 as pk
from paged_kv_cache_107_gb300 import workloads
from tests import attention_reference as ar

pytestmark = pytest.mark.gpu

RULES = {
    "none": dict(),
    "cap": dict(softcap=5.0),
    "bias": dict(bias=True),
    "window1": dict(window=1),
    "window": dict(window=100),
    "sink": dict(window=37, sink=5),
    "prefix": dict(prefix=70),
    "prefix_window": dict(prefix=20, window=33, sink=3),
    "all": dict(softcap=30.0, bias=True, window=150, sink=130, prefix=3),
}


def slopes_of(H, bias):
    return np.array([2.0 ** (-8 * (h + 1) / H) for h in range(H)], np.float32) if bias else None


def make_mod(rule, H, S, dev="cuda"):
    sl = slopes_of(H, rule.get("bias"))
    prefix = rule.get("prefix")
    return pk.ScoreMod(
        softcap=rule.get("softcap", 0.0), window=rule.get("window", 0), sink=rule.get("sink", 0),
        slopes=None if sl is None else torch.from_numpy(sl).to(dev),
        prefix_lens=None if prefix is None else torch.full((S,), prefix, dtype=torch.int32,
                                                           device=dev))


def hide_rows(case, first_pos, rule):
    """Poison what no query from position first_pos[b] on sees: NaN rows, and -1 for blocks
    that hold nothing else."""
    if not rule.get("window"):
        return
    bs = case.block_size
    keep = max(rule.get("sink", 0), rule.get("prefix") or 0)
    for b in range(case.num_seqs):
        low = max(0, first_pos[b] - rule["window"] + 1)
        for t in range(min(keep, low), low):
            blk = int(case.block_tables[b, t // bs])
            case.k_cache[blk, t % bs] = float("nan")
            case.v_cache[blk, t % bs] = float("nan")
        for j in range(case.max_blocks):
            if j * bs >= keep and (j + 1) * bs <= low:
                case.block_tables[b, j] = -1


def decode_check(lens, H, Hk, D, bs, dtype, rule, seed, grid_ctas=0, q_gain=3.0):
    case = workloads.decode_case(lens, H, Hk, D, bs, seed=seed, dtype=dtype)
    for b, n in enumerate(lens):  # the newest token is in the cache
        if n:
            blk = int(case.block_tables[b, (n - 1) // bs])
            case.k_cache[blk, (n - 1) % bs] = case.k_new[b]
            case.v_cache[blk, (n - 1) % bs] = case.v_new[b]
    q = (case.q.float() * q_gain).to(dtype)
    tables = case.block_tables.copy()
    hide_rows(case, [n - 1 for n in lens], rule)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, float("nan"), device="cuda")
    pk.pa_decode_mod(out, q.cuda(), case.k_cache.cuda(), case.v_cache.cuda(),
                     torch.from_numpy(case.block_tables).cuda(),
                     torch.from_numpy(case.context_lens).cuda(), make_mod(rule, H, len(lens)),
                     grid_ctas=grid_ctas, dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0, f"device error bits {int(err.item())}"
    got = out.float().cpu().double().numpy()
    ref, tol = np.zeros(got.shape), np.zeros(got.shape)
    for b, n in enumerate(lens):
        see = ar.visible([n - 1], n, window=rule.get("window", 0), sink=rule.get("sink", 0),
                         prefix=rule.get("prefix") or 0) if n else np.zeros((1, 0), bool)
        r, A, dev = ar.attend(q[b:b + 1].double().numpy(), ar.gather(case.k_cache, tables[b], n),
                              ar.gather(case.v_cache, tables[b], n), [n - 1], see,
                              softcap=rule.get("softcap", 0.0),
                              slopes=slopes_of(H, rule.get("bias")))
        ref[b], tol[b] = r[0], ar.bound(r, A, dev, dtype)[0]
        if n == 0:
            assert np.all(got[b] == 0.0)
    ar.assert_within(got, ref, tol, f"{lens} {rule}")


LENS = [1, 2, 15, 16, 17, 0, 127, 128, 129, 300, 1000, 33]


@pytest.mark.parametrize("rule", list(RULES))
@pytest.mark.parametrize("H,Hk,D,bs,dtype", [
    (16, 8, 128, 16, torch.bfloat16), (32, 8, 64, 16, torch.float16),
    (16, 2, 128, 256, torch.float16), (4, 4, 64, 20, torch.bfloat16)])
def test_decode_rules(rule, H, Hk, D, bs, dtype):
    decode_check(LENS, H, Hk, D, bs, dtype, RULES[rule], seed=400 + len(rule) + H + D)


@pytest.mark.parametrize("G", range(1, 9))
def test_decode_group_sizes(G):
    decode_check([77, 1, 260, 513], 2 * G, 2, 128 if G % 2 else 64, 32, torch.bfloat16,
                 RULES["all"], seed=500 + G)


@pytest.mark.parametrize("Hk", [1, 3, 4, 6])
@pytest.mark.parametrize("bs", [5, 48, 128])
def test_decode_slabs_and_block_sizes(Hk, bs):
    decode_check([9, 130, 700], 3 * Hk, Hk, 128, bs, torch.float16, RULES["sink"],
                 seed=600 + Hk + bs)


@pytest.mark.parametrize("grid", [1, 7, 300, 601])
@pytest.mark.parametrize("rule", ["sink", "all"])
def test_decode_splits(grid, rule):
    """Sequences cut between CTAs, the kept and the window part included."""
    decode_check([2000, 40, 900, 1, 3000 - 1], 16, 8, 128, 16, torch.bfloat16, RULES[rule],
                 seed=700 + grid, grid_ctas=grid)


@pytest.mark.parametrize("gain", [0.2, 4.0, 40.0])
@pytest.mark.parametrize("cap", [1.0, 50.0, 1000.0])
def test_decode_cap_range(gain, cap):
    """Scores from far below the cap to far above it."""
    decode_check([50, 333], 16, 8, 128, 16, torch.float16, dict(softcap=cap), seed=800,
                 q_gain=gain)


def prefill_check(cached, new, H, Hk, D, bs, dtype, rule, seed, causal=True, q_gain=3.0):
    case = workloads.prefill_case(cached, new, H, Hk, D, bs, seed=seed, dtype=dtype,
                                  causal=causal)
    flat_k = case.k_cache.view(-1, Hk, D)
    flat_v = case.v_cache.view(-1, Hk, D)
    slots = torch.from_numpy(case.slot_mapping.astype(np.int64))
    flat_k[slots], flat_v[slots] = case.k_new, case.v_new
    q = (case.q.float() * q_gain).to(dtype)
    tables = case.block_tables.copy()
    hide_rows(case, list(cached), rule)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    # rows behind the last sequence stay as they were
    out = torch.full((q.shape[0] + 3, H, D), 7.0, dtype=dtype, device="cuda")
    q_dev = torch.cat([q, torch.full((3, H, D), float("nan"), dtype=dtype)]).cuda()
    pk.pa_prefill_mod(out, q_dev, case.k_cache.cuda(), case.v_cache.cuda(),
                      torch.from_numpy(case.block_tables).cuda(),
                      torch.from_numpy(case.cu_seqlens_q).cuda(),
                      torch.from_numpy(case.cu_seqlens_k).cuda(), case.max_seqlen_q,
                      case.max_seqlen_k, make_mod(rule, H, len(new)), causal=causal, dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0, f"device error bits {int(err.item())}"
    assert torch.all(out[q.shape[0]:] == 7.0)
    got = out[:q.shape[0]].float().cpu().double().numpy()
    ref, tol = np.zeros(got.shape), np.zeros(got.shape)
    at = 0
    for s, (c, n) in enumerate(zip(cached, new)):
        pos = np.arange(c, c + n)
        see = ar.visible(pos, c + n, causal, rule.get("window", 0), rule.get("sink", 0),
                         rule.get("prefix") or 0)
        r, A, dev = ar.attend(q[at:at + n].double().numpy(),
                              ar.gather(case.k_cache, tables[s], c + n),
                              ar.gather(case.v_cache, tables[s], c + n), pos, see,
                              softcap=rule.get("softcap", 0.0),
                              slopes=slopes_of(H, rule.get("bias")))
        ref[at:at + n], tol[at:at + n] = r, ar.bound(r, A, dev, dtype)
        at += n
    ar.assert_within(got, ref, tol, f"{cached} {new} {rule}")


CACHED, NEW = [0, 17, 256, 1000, 0, 90], [70, 300, 1, 257, 1, 128]


@pytest.mark.parametrize("rule", list(RULES))
@pytest.mark.parametrize("H,Hk,D,bs,dtype", [
    (16, 8, 128, 16, torch.bfloat16), (8, 2, 64, 64, torch.float16),
    (8, 1, 128, 256, torch.float16), (2, 2, 64, 128, torch.bfloat16)])
def test_prefill_rules(rule, H, Hk, D, bs, dtype):
    prefill_check(CACHED, NEW, H, Hk, D, bs, dtype, RULES[rule], seed=900 + len(rule) + H + D)


@pytest.mark.parametrize("rule", ["cap", "bias", "window", "all"])
def test_prefill_not_causal(rule):
    prefill_check([0, 37, 256], [50, 91, 300], 16, 8, 128, 32, torch.bfloat16, RULES[rule],
                  seed=1000, causal=False)


@pytest.mark.parametrize("rule", ["sink", "all"])
def test_prefill_many_sequences(rule):
    """More sequences than the in-kernel sort takes: one unit per CTA."""
    rng = np.random.default_rng(1001)
    prefill_check(rng.integers(0, 60, 1100).tolist(), rng.integers(1, 5, 1100).tolist(), 4, 2, 64,
                  16, torch.bfloat16, RULES[rule], seed=1002)


def test_prefill_long_window():
    """Key tiles left out in the middle of long sequences, for every tile of the unit."""
    prefill_check([1500, 0], [700, 2100], 8, 2, 128, 16, torch.bfloat16,
                  dict(window=200, sink=140), seed=1003)


@pytest.mark.parametrize("gain", [0.2, 40.0])
def test_prefill_cap_range(gain):
    prefill_check([30], [200], 4, 2, 128, 16, torch.float16, dict(softcap=50.0), seed=1004,
                  q_gain=gain)


def test_decode_graph_replay():
    """Captured with its own workspace, replayed on other lengths; without one the capture is
    refused."""
    H, Hk, D, bs, B, maxb = 16, 8, 64, 16, 6, 30
    rule = RULES["sink"]
    mod = make_mod(rule, H, B)
    ws = pk.DecodeWorkspace(B, H, Hk, D)
    big = workloads.decode_case([maxb * bs] * B, H, Hk, D, bs, seed=1100)
    k, v, q = big.k_cache.cuda(), big.v_cache.cuda(), big.q.cuda()
    last = torch.from_numpy(big.slot_mapping.astype(np.int64)).cuda()
    k.view(-1, Hk, D)[last], v.view(-1, Hk, D)[last] = big.k_new.cuda(), big.v_new.cuda()
    bt = torch.from_numpy(big.block_tables).cuda()
    ctx = torch.ones(B, dtype=torch.int32, device="cuda")
    out = torch.zeros_like(q)
    pk.pa_decode_mod(out, q, k, v, bt, ctx, mod, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        with pytest.raises(pk.PagedAttentionError, match="workspace"):
            pk.pa_decode_mod(out, q, k, v, bt, ctx, mod)
        pk.pa_decode_mod(out, q, k, v, bt, ctx, mod, workspace=ws)
    for lens in ([480, 1, 200, 0, 37, 38], [0] * 6, [5, 480, 480, 480, 480, 41]):
        ctx.copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        want = torch.empty_like(q)
        pk.pa_decode_mod(want, q, k, v, bt, ctx, mod)
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))
        for b, n in enumerate(lens):
            see = ar.visible([n - 1], n, window=37, sink=5) if n else np.zeros((1, 0), bool)
            r, A, dev = ar.attend(big.q[b:b + 1].double().numpy(),
                                  ar.gather(k.cpu(), big.block_tables[b], n),
                                  ar.gather(v.cpu(), big.block_tables[b], n), [n - 1], see)
            ar.assert_within(out[b:b + 1].float().cpu().double().numpy(), r,
                             ar.bound(r, A, dev, torch.bfloat16), f"{lens} {b}")


def test_decode_on_two_streams():
    """Two calls in flight at once on streams of their own, each with the default workspace."""
    H, Hk, D, bs = 16, 8, 128, 16
    cases = [workloads.decode_case([700 + i, 90, 1800], H, Hk, D, bs, seed=1200 + i, poison=False)
             for i in range(2)]
    mod = make_mod(RULES["all"], H, 3)
    dev = [[t.cuda() for t in (c.q, c.k_cache, c.v_cache)] +
           [torch.from_numpy(c.block_tables).cuda(), torch.from_numpy(c.context_lens).cuda()]
           for c in cases]
    want = [pk.pa_decode_mod(torch.empty_like(d[0]), *d, mod) for d in dev]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in dev]
    outs = [[torch.empty_like(d[0]) for _ in range(20)] for d in dev]
    for i in range(20):
        for d, s, o in zip(dev, streams, outs):
            pk.pa_decode_mod(o[i], *d, mod, stream=s)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        for x in o:
            assert torch.equal(x.view(torch.int16), w.view(torch.int16))


def test_a_windowed_capped_model_step_by_step():
    """A prompt through pa_prefill_mod, then tokens through pa_store_kvcache and
    pa_decode_mod; blocks that leave the window are given back as it moves."""
    H, Hk, D, bs, n0, steps = 8, 2, 128, 16, 75, 40
    rule = dict(softcap=20.0, bias=True, window=40, sink=4)
    total = n0 + steps
    case = workloads.prefill_case([0], [total], H, Hk, D, bs, seed=1300)
    mod = make_mod(rule, H, 1)
    k, v = case.k_cache.cuda(), case.v_cache.cuda()
    q, kn, vn = case.q.cuda(), case.k_new.cuda(), case.v_new.cuda()
    slots = torch.from_numpy(case.slot_mapping).cuda()
    bt = torch.from_numpy(case.block_tables).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    pk.pa_store_kvcache(kn[:n0], vn[:n0], k, v, slots[:n0], dev_err=err)
    cu = torch.tensor([0, n0], dtype=torch.int32, device="cuda")
    pk.pa_prefill_mod(out[:n0], q[:n0], k, v, bt, cu, cu, n0, n0, mod, dev_err=err)
    for p in range(n0, total):
        gone = (p - rule["window"] + 1) // bs  # blocks 1..gone-1 hold nothing visible
        for j in range(1, gone):
            if int(bt[0, j]) >= 0:
                k[int(bt[0, j])], v[int(bt[0, j])] = float("nan"), float("nan")
                bt[0, j] = -1
        pk.pa_store_kvcache(kn[p:p + 1], vn[p:p + 1], k, v, slots[p:p + 1], dev_err=err)
        pk.pa_decode_mod(out[p:p + 1], q[p:p + 1], k, v, bt,
                         torch.tensor([p + 1], dtype=torch.int32, device="cuda"), mod,
                         dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    pos = np.arange(total)
    r, A, dev = ar.attend(case.q.double().numpy(), case.k_new.double().numpy(),
                          case.v_new.double().numpy(), pos,
                          ar.visible(pos, total, window=40, sink=4), softcap=20.0,
                          slopes=slopes_of(H, True))
    ar.assert_within(out.float().cpu().double().numpy(), r, ar.bound(r, A, dev, torch.bfloat16))
