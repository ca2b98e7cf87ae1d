"""pa_decode_shared against the plain 64-bit attention, within the bound that its arithmetic
implies (attention_reference.py): one rounding of the probabilities in either part, none in
the fp32 join."""
import numpy as np
import pytest
import torch

import paged_kv_cache_107_gb300 as pk
from paged_kv_cache_107_gb300 import workloads
from tests import attention_reference as ar

pytestmark = pytest.mark.gpu


class Shared:
    """Groups of sizes[g] sequences over prefix[g] common positions, then rest[b] of their own
    (rest None: a padding row of length 0)."""

    def __init__(self, sizes, prefix, rest, H, Hk, D, bs, dtype, seed, maxb_extra=0):
        self.H, self.Hk, self.D, self.bs, self.dtype = H, Hk, D, bs, dtype
        rng = np.random.default_rng(seed)
        lens = []
        at = 0
        for n, p in zip(sizes, prefix):
            lens += [0 if rest[at + i] is None else p + rest[at + i] for i in range(n)]
            at += n
        self.lens = lens
        self.starts = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
        self.prefix = np.asarray(prefix, np.int32)
        need = [-(-n // bs) for n in lens]
        nb = sum(need) + 3
        maxb = max(max(need, default=1), 1) + maxb_extra
        order = rng.permutation(nb)
        self.tables = np.full((len(lens), maxb), -1, np.int32)
        used = 0
        for g, p in enumerate(prefix):
            for b in range(self.starts[g], self.starts[g + 1]):
                lead = self.starts[g]
                share = p // bs if b > lead and lens[b] else 0  # whole blocks
                self.tables[b, :share] = self.tables[lead, :share]
                own = need[b] - share
                self.tables[b, share:need[b]] = order[used:used + own]
                used += own
        gen = torch.Generator().manual_seed(seed)
        self.k = torch.full((nb, bs, Hk, D), float("nan"), dtype=dtype)
        self.v = torch.full((nb, bs, Hk, D), float("nan"), dtype=dtype)
        kf, vf = self.k.view(-1, Hk, D), self.v.view(-1, Hk, D)
        for g, p in enumerate(prefix):
            for b in range(self.starts[g], self.starts[g + 1]):
                n, lead = lens[b], self.starts[g]
                if n == 0:
                    continue
                t = np.arange(n)
                rows = torch.from_numpy(self.tables[b, t // bs].astype(np.int64) * bs + t % bs)
                kn = torch.randn(n, Hk, D, generator=gen).to(dtype)
                vn = torch.randn(n, Hk, D, generator=gen).to(dtype)
                if b > lead and p:  # the same values at the shared positions
                    r0 = torch.from_numpy(self.tables[lead, t[:p] // bs].astype(np.int64) * bs
                                          + t[:p] % bs)
                    kn[:p], vn[:p] = kf[r0], vf[r0]
                kf[rows], vf[rows] = kn, vn
        self.q = (torch.randn(len(lens), H, D, generator=gen) * 2).to(dtype)

    def device(self):
        return (self.q.cuda(), self.k.cuda(), self.v.cuda(), torch.from_numpy(self.tables).cuda(),
                torch.tensor(self.lens, dtype=torch.int32, device="cuda"),
                torch.from_numpy(self.starts).cuda(), torch.from_numpy(self.prefix).cuda())

    def reference(self, rows=None):
        rows = range(len(self.lens)) if rows is None else rows
        ref, tol = [], []
        for b in rows:
            n = self.lens[b]
            r, A, dev = ar.attend(self.q[b:b + 1].double().numpy(),
                                  ar.gather(self.k, self.tables[b], n),
                                  ar.gather(self.v, self.tables[b], n), [n - 1],
                                  np.ones((1, n), bool))
            ref.append(r[0])
            tol.append(ar.bound(r, A, dev, self.dtype)[0])
        return np.array(ref), np.array(tol)

    def check(self, rows=None, ws=None):
        d = self.device()
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full_like(d[0], float("nan"))
        pk.pa_decode_shared(out, *d, workspace=ws, dev_err=err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0, f"device error bits {int(err.item())}"
        got = out.float().cpu().double().numpy()
        ref, tol = self.reference(rows)
        ar.assert_within(got if rows is None else got[list(rows)], ref, tol, f"{self.lens[:8]}")
        return out


BF, FP = torch.bfloat16, torch.float16


@pytest.mark.parametrize("prefix", [0, 1, 127, 128, 129, 255, 256, 300, 640, 1000])
@pytest.mark.parametrize("D,dtype", [(128, BF), (64, FP)])
def test_prefix_lengths(prefix, D, dtype):
    """Prefixes that end anywhere in a block and a tile; suffixes of 0, 1 and a few tiles."""
    Shared([5], [prefix], [1, 0 if prefix else 1, 17, 130, 300], 16, 8, D, 16, dtype,
           seed=100 + prefix).check()


@pytest.mark.parametrize("G", range(1, 9))
def test_group_sizes(G):
    """Row tiles of 128/G sequences, whole or not, one to three of them."""
    P = 128 // G
    for n in (2, P, P + 1, 2 * P + 3):
        rest = [1 + (i * 7) % 40 for i in range(n)]
        Shared([n], [400], rest, 2 * G, 2, 64 if G % 2 else 128, 16, BF,
               seed=200 + 10 * G + n).check(rows=sorted({0, 1, n // 2, P - 1, min(P, n - 1), n - 1}
                                                        & set(range(n))))


@pytest.mark.parametrize("bs", [5, 8, 24, 48, 64, 128, 192, 256])
def test_block_sizes(bs):
    Shared([3, 4], [bs * (600 // bs), 333], [1, 50, 200, 9, 1, 70, 33], 32, 8, 128, bs, FP,
           seed=300 + bs).check()


@pytest.mark.parametrize("Hk", [1, 2, 3, 4, 12])
def test_kv_heads(Hk):
    Shared([6, 2], [500, 129], [4, 1, 90, 33, 2, 1, 61, 7], 2 * Hk, Hk, 128, 16, BF,
           seed=400 + Hk).check()


def test_many_groups_of_all_kinds():
    """Uneven, lone, empty and prefix-free groups, padding rows; more units than CTAs."""
    rng = np.random.default_rng(500)
    sizes = [64, 1, 0, 17, 2, 33, 1, 0, 5, 40]
    prefix = [512, 700, 128, 0, 1300, 144, 0, 9, 2000, 256]
    rest = [int(x) for x in rng.integers(1, 300, sum(sizes))]
    rest[5] = rest[70] = None
    rest[66] = 0
    Shared(sizes, prefix, rest, 16, 8, 64, 16, BF, seed=501).check()


def test_prefixes_of_empty_groups_do_not_matter():
    c = Shared([0, 5, 0, 0, 2], [0, 300, 0, 0, 129], [1, 4, 70, 9, 2, 33, 1], 8, 2, 128, 16, BF,
               seed=505)
    c.prefix[[0, 2, 3]] = [1 << 30, -5, 100000]
    c.check()


def test_hundreds_of_small_groups():
    rng = np.random.default_rng(510)
    sizes = [2] * 400 + [3] * 30
    prefix = [int(x) for x in rng.integers(0, 300, len(sizes))]
    rest = [int(x) for x in rng.integers(1, 30, sum(sizes))]
    Shared(sizes, prefix, rest, 8, 4, 64, 16, FP, seed=511).check(rows=range(0, 890, 7))


def test_long_prefix_is_split_over_every_sm():
    Shared([9], [20000], [1 + i for i in range(9)], 8, 2, 128, 64, BF, seed=520).check(
        rows=[0, 4, 8])


def test_two_row_tiles_and_a_single_one():
    """Units of both kinds in one group, cut between CTAs."""
    Shared([150], [3000], [1 + i % 5 for i in range(150)], 16, 8, 128, 16, BF, seed=530).check(
        rows=[0, 63, 64, 127, 128, 149])


def test_equals_the_plain_decode():
    c = Shared([20, 3], [900, 400], [1 + 3 * i for i in range(23)], 32, 8, 128, 16, BF, seed=540)
    d = c.device()
    a = pk.pa_decode_shared(torch.empty_like(d[0]), *d)
    b = pk.pa_decode(torch.empty_like(d[0]), *d[:5])
    torch.cuda.synchronize()
    ref, tol = c.reference()
    for x in (a, b):
        ar.assert_within(x.float().cpu().double().numpy(), ref, tol)


def test_is_deterministic():
    c = Shared([70, 9], [2500, 333], [1 + (i * 13) % 200 for i in range(79)], 16, 8, 128, 16, BF,
               seed=550)
    d = c.device()
    outs = [pk.pa_decode_shared(torch.empty_like(d[0]), *d) for _ in range(30)]
    torch.cuda.synchronize()
    for o in outs[1:]:
        assert torch.equal(o.view(torch.int16), outs[0].view(torch.int16))


def test_a_workspace_serves_smaller_batches_and_needs_no_clearing():
    ws = pk.SharedDecodeWorkspace(80, 16, 8, 128)
    ws.buffer.fill_(0xFF)
    for seed, sizes in ((560, [60, 20]), (561, [3]), (562, [1, 79]), (563, [2, 2])):
        rng = np.random.default_rng(seed)
        Shared(sizes, [int(x) for x in rng.integers(100, 900, len(sizes))],
               [int(x) for x in rng.integers(1, 200, sum(sizes))], 16, 8, 128, 16, BF,
               seed=seed).check(ws=ws)


def test_scale():
    c = Shared([4], [300], [5, 6, 7, 8], 16, 8, 64, 16, BF, seed=570)
    d = c.device()
    out = pk.pa_decode_shared(torch.empty_like(d[0]), *d, scale=0.03)
    c.q = (c.q.double() * 0.03 * 8).to(torch.float64)  # 1/sqrt(64) = 1/8
    ref, tol = c.reference()
    ar.assert_within(out.float().cpu().double().numpy(), ref, tol)


def test_bad_groups_still_decode():
    """Arrays that do not describe groups of the batch are flagged and nothing is shared."""
    c = Shared([4, 3], [256, 130], [1, 20, 33, 4, 5, 6, 70], 16, 8, 128, 16, BF, seed=580)
    d = c.device()
    ref, tol = c.reference()
    for starts, prefix in (([0, 5, 4], [256, 130]), ([1, 4, 7], [256, 130]),
                           ([0, 4, 6], [256, 130]), ([0, 4, 8], [256, 130]),
                           ([-3, 4, 7], [256, 130]), ([0, 4, 7], [-1, 130]),
                           ([0, 4, 7], [256, 1 << 30])):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = pk.pa_decode_shared(torch.empty_like(d[0]), *d[:5],
                                  torch.tensor(starts, dtype=torch.int32, device="cuda"),
                                  torch.tensor(prefix, dtype=torch.int32, device="cuda"),
                                  dev_err=err)
        torch.cuda.synchronize()
        assert int(err.item()) == pk.PA_DEV_ERR["seqlens"]
        ar.assert_within(out.float().cpu().double().numpy(), ref, tol)


def test_context_inside_the_prefix_is_flagged():
    c = Shared([4], [256], [1, 20, 33, 4], 16, 8, 128, 16, BF, seed=590)
    d = list(c.device())
    d[4] = torch.tensor([257, 100, 289, 260], dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = pk.pa_decode_shared(torch.empty_like(d[0]), *d, dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == pk.PA_DEV_ERR["context"]
    ref, tol = c.reference()
    ok = [0, 2, 3]
    ar.assert_within(out.float().cpu().double().numpy()[ok], ref[ok], tol[ok])


def test_block_outside_the_pool_is_flagged():
    c = Shared([4, 2], [256, 128], [1, 20, 33, 4, 3, 9], 16, 8, 128, 16, BF, seed=595)
    d = list(c.device())
    d[3] = d[3].clone()
    d[3][0, 3] = 1 << 20
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = pk.pa_decode_shared(torch.empty_like(d[0]), *d, dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == pk.PA_DEV_ERR["block_id"]
    ref, tol = c.reference([4, 5])
    ar.assert_within(out.float().cpu().double().numpy()[4:], ref, tol)


def test_graph_replay_with_other_groups():
    """One capture serves batches with other groups, lengths and padding rows; a capture
    without a workspace is refused."""
    H, Hk, D, bs, B, groups, maxb = 16, 8, 128, 16, 12, 4, 60
    ws = pk.SharedDecodeWorkspace(B, H, Hk, D)
    cases = [Shared([6, 0, 6, 0], [500, 0, 129, 0], [3 * i for i in range(1, 13)], H, Hk, D, bs,
                    BF, 600),
             Shared([12, 0, 0, 0], [800, 0, 0, 0], [1] * 9 + [None] * 3, H, Hk, D, bs, BF, 601),
             Shared([1, 4, 4, 3], [300, 200, 400, 0], [9] * 9 + [None] * 3, H, Hk, D, bs, BF, 602)]
    nb = max(c.k.shape[0] for c in cases)
    k = torch.zeros(nb, bs, Hk, D, dtype=BF, device="cuda")
    v, q = torch.zeros_like(k), torch.zeros(B, H, D, dtype=BF, device="cuda")
    bt = torch.full((B, maxb), -1, dtype=torch.int32, device="cuda")
    ctx = torch.zeros(B, dtype=torch.int32, device="cuda")
    st = torch.full((groups + 1,), B, dtype=torch.int32, device="cuda")
    st[0] = 0
    pl = torch.zeros(groups, dtype=torch.int32, device="cuda")
    out, err = torch.zeros_like(q), torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (out, q, k, v, bt, ctx, st, pl)
    pk.pa_decode_shared(*args, workspace=ws, dev_err=err)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        with pytest.raises(pk.PagedAttentionError, match="workspace"):
            pk.pa_decode_shared(*args)
        for _ in range(3):
            pk.pa_decode_shared(*args, workspace=ws, dev_err=err)
    for c in cases + cases[:1]:
        k[:c.k.shape[0]], v[:c.k.shape[0]] = c.k.cuda(), c.v.cuda()
        q.copy_(c.q)
        bt.fill_(-1)
        bt[:, :c.tables.shape[1]] = torch.from_numpy(c.tables).cuda()
        ctx.copy_(torch.tensor(c.lens, dtype=torch.int32))
        st.copy_(torch.from_numpy(c.starts))
        pl.copy_(torch.from_numpy(c.prefix))
        g.replay()
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        ref, tol = c.reference()
        ar.assert_within(out.float().cpu().double().numpy(), ref, tol)


def test_on_two_streams():
    cases = [Shared([30, 2], [1500 + 100 * i, 300], [1 + (j * 5) % 60 for j in range(32)], 16, 8,
                    128, 16, BF, seed=620 + i) for i in range(2)]
    dev = [c.device() for c in cases]
    want = [pk.pa_decode_shared(torch.empty_like(d[0]), *d) for d in dev]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in dev]
    outs = [[torch.empty_like(d[0]) for _ in range(20)] for d in dev]
    for i in range(20):
        for d, s, o in zip(dev, streams, outs):
            pk.pa_decode_shared(o[i], *d, stream=s)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        for x in o:
            assert torch.equal(x.view(torch.int16), w.view(torch.int16))


def test_decoding_a_group_step_by_step():
    """A prompt through the prefill, then every member's tokens through the store and
    pa_decode_shared, the members' first blocks being the prompt's."""
    H, Hk, D, bs, n, P, steps = 8, 2, 128, 16, 5, 160, 20
    prompt = workloads.prefill_case([0], [P], H, Hk, D, bs, num_blocks=64, seed=630)
    k, v = prompt.k_cache.cuda(), prompt.v_cache.cuda()
    pk.pa_store_kvcache(prompt.k_new.cuda(), prompt.v_new.cuda(), k, v,
                        torch.from_numpy(prompt.slot_mapping).cuda())
    free = sorted(set(range(64)) - set(prompt.block_tables[0].tolist()))
    tables = np.full((n, 12), -1, np.int32)
    tables[:, :P // bs] = prompt.block_tables[0, :P // bs]
    gen = torch.Generator().manual_seed(631)
    new = [torch.randn(steps, n, x, D, generator=gen).bfloat16() for x in (H, Hk, Hk)]
    starts = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    plen = torch.tensor([P], dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for i in range(steps):
        pos = P + i
        if pos % bs == 0:
            tables[:, pos // bs] = [free.pop() for _ in range(n)]
        slots = torch.from_numpy(tables[:, pos // bs] * bs + pos % bs).cuda()
        q, kn, vn = (x[i].cuda() for x in new)
        pk.pa_store_kvcache(kn, vn, k, v, slots, dev_err=err)
        out = pk.pa_decode_shared(torch.empty_like(q), q, k, v, torch.from_numpy(tables).cuda(),
                                  torch.full((n,), pos + 1, dtype=torch.int32, device="cuda"),
                                  starts, plen, dev_err=err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        for b in range(n):
            keys = torch.cat([prompt.k_new, new[1][:i + 1, b]]).double().numpy()
            vals = torch.cat([prompt.v_new, new[2][:i + 1, b]]).double().numpy()
            r, A, dev = ar.attend(new[0][i, b:b + 1].double().numpy(), keys, vals, [pos],
                                  np.ones((1, pos + 1), bool))
            ar.assert_within(out[b:b + 1].float().cpu().double().numpy(), r,
                             ar.bound(r, A, dev, BF), f"step {i}")


def test_shares_that_end_one_step_into_the_next_unit():
    """Prefixes whose cut into equal shares leaves some CTAs a single step of a second unit: the
    warps of one half may then be a segment behind the other's. No wait runs out and every call
    gives the same bits."""
    B, H, Hk, D, bs = 128, 32, 8, 128, 128
    gen = torch.Generator("cuda").manual_seed(5000)
    k, v = (torch.randn(64 + B, bs, Hk, D, dtype=BF, device="cuda", generator=gen)
            for _ in range(2))
    q = torch.randn(B, H, D, dtype=BF, device="cuda", generator=gen)
    starts = torch.tensor([0, B], dtype=torch.int32, device="cuda")
    for tiles in (16, 24, 31, 32, 40, 48, 63, 64):
        table = torch.arange(tiles, dtype=torch.int32, device="cuda").repeat(B, 1)
        table = torch.cat([table, 64 + torch.arange(B, dtype=torch.int32, device="cuda")[:, None]], 1)
        ctx = tiles * bs + torch.arange(B, dtype=torch.int32, device="cuda") % 7
        d = (q, k, v, table, ctx, starts, starts.new_tensor([tiles * bs]))
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        outs = [pk.pa_decode_shared(torch.empty_like(q), *d, dev_err=err) for _ in range(100)]
        torch.cuda.synchronize()
        assert int(err.item()) == 0, f"device error bits {int(err.item())} at {tiles} tiles"
        for o in outs[1:]:
            assert torch.equal(o.view(torch.int16), outs[0].view(torch.int16))
        for b in (0, 77):
            n = int(ctx[b])
            rows = [c[table[b].long()].reshape(-1, Hk, D)[:n].cpu().double().numpy()
                    for c in (k, v)]
            r, A, dev = ar.attend(q[b:b + 1].cpu().double().numpy(), *rows, [n - 1],
                                  np.ones((1, n), bool))
            ar.assert_within(outs[0][b:b + 1].float().cpu().double().numpy(), r,
                             ar.bound(r, A, dev, BF), f"{tiles} tiles, {b}")


@pytest.mark.parametrize("per_group,prefix", [(1, 200), (2, 130), (300, 144), (8192, 300)])
def test_most_sequences(per_group, prefix):
    """8192 sequences, in groups of one, two, a few hundred, or all together."""
    B, H, Hk, D, bs = 8192, 2, 1, 64, 16
    gen = torch.Generator("cuda").manual_seed(6000 + per_group)
    starts = list(range(0, B, per_group)) + [B]
    groups, lead = len(starts) - 1, -(-prefix // bs)
    k, v = (torch.randn(groups * lead + B, bs, Hk, D, dtype=BF, device="cuda", generator=gen)
            for _ in range(2))
    q = torch.randn(B, H, D, dtype=BF, device="cuda", generator=gen) * 2
    # whole blocks are shared; the block that holds the prefix's end is copied to each sequence
    group = torch.arange(B, device="cuda") // per_group
    table = group[:, None] * lead + torch.arange(lead, device="cuda")
    own = groups * lead + torch.arange(B, device="cuda")
    part = prefix % bs
    if part:
        for c in (k, v):
            c[own, :part] = c[table[:, -1], :part]
        table[:, -1] = own
        first = torch.tensor(starts[:-1], device="cuda")
        k[first * 0 + group[first] * lead + lead - 1] = float("nan")  # no table names it
    else:
        table = torch.cat([table, own[:, None]], 1)
    ctx = (prefix + 1 + torch.arange(B, device="cuda") % (bs - part)).int()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    table = table.int().contiguous()
    out = pk.pa_decode_shared(
        torch.full_like(q, float("nan")), q, k, v, table, ctx,
        torch.tensor(starts, dtype=torch.int32, device="cuda"),
        torch.full((groups,), prefix, dtype=torch.int32, device="cuda"), dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0, f"device error bits {int(err.item())}"
    assert torch.isfinite(out.float()).all()
    for b in (0, 1, 299, 300, 4095, 4096, 8000, 8191):
        n = int(ctx[b])
        rows = [c[table[b].long()].reshape(-1, Hk, D)[:n].cpu().double().numpy() for c in (k, v)]
        r, A, dev = ar.attend(q[b:b + 1].cpu().double().numpy(), *rows, [n - 1],
                              np.ones((1, n), bool))
        ar.assert_within(out[b:b + 1].float().cpu().double().numpy(), r, ar.bound(r, A, dev, BF),
                         f"sequence {b}")


@pytest.mark.parametrize("Hk", [155, 160])
def test_more_kv_heads_than_sms(Hk):
    """A CTA for every slab of KV heads, more than fit the SMs at once."""
    Shared([5, 1], [400, 0], [3, 40, 1, 9, 100, 60], Hk, Hk, 64, 16, BF, seed=6100 + Hk).check(
        rows=[0, 2, 4, 5])
