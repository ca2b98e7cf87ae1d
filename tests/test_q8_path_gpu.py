"""The 8-bit cache's calls together, as a serving step makes them: rotary and quantising store,
then decode; a chunk's prefix read back and prefilled; under graphs, on other streams, two at a
time."""
import numpy as np
import pytest
import torch

import paged_kv_cache_107_gb300 as pk
from tests import attention_reference as att
from tests import q8_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Server:
    """Sequences that grow by tokens through the 8-bit cache; the host keeps the 16-bit rows that
    the definition needs."""

    def __init__(self, fmt, H=16, Hk=8, D=128, bs=16, nb=64, seed=0):
        self.fmt, self.H, self.Hk, self.D, self.bs = fmt, H, Hk, D, bs
        self.cache = pk.Q8Cache(nb, bs, Hk, D, ref.FORMATS[fmt])
        self.rotary = pk.Rotary(D, sections=(D // 8, D // 8, D // 4), base=1e6)
        self.g = torch.Generator(device=DEV).manual_seed(seed)
        self.free = np.random.default_rng(seed).permutation(nb).tolist()
        self.tables = [[], [], []]
        self.lens = [0, 0, 0]
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)

    def new(self, counts):
        """Inputs of counts[s] new tokens for each sequence, slots allocated."""
        n = sum(counts)
        x = [torch.randn(n, h, self.D, generator=self.g, device=DEV).bfloat16()
             for h in (self.H, self.Hk, self.Hk)]
        slots, pos = [], []
        for s, m in enumerate(counts):
            for p in range(self.lens[s], self.lens[s] + m):
                if p // self.bs == len(self.tables[s]):
                    self.tables[s].append(self.free.pop())
                slots.append(self.tables[s][p // self.bs] * self.bs + p % self.bs)
                pos.append((p, p // 7, p % 7))
            self.lens[s] += m
        return (*x, ints(pos).t().contiguous(), ints(slots))

    def padded(self, width=None):
        width = width or max(map(len, self.tables))
        return ints([t + [-1] * (width - len(t)) for t in self.tables])

    def rows(self):
        return (ref.dequantised(self.cache.k, self.cache.k_scale),
                ref.dequantised(self.cache.v, self.cache.v_scale))

    def check_decode(self, q, out):
        k, v = self.rows()
        o, tol = ref.decode(q, k, v, float(self.cache.v_scale.max()), self.tables, self.lens,
                            self.bs, torch.bfloat16, None, 448.0 if self.fmt == "e4m3" else 127.0,
                            float(self.cache.k_scale.max()))
        att.assert_within(out.double().cpu().numpy(), o, tol)
        assert self.err.item() == 0


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("D", [64, 128])
def test_prefill_then_decode(fmt, D):
    s = Server(fmt, D=D, seed=D)
    for counts in ([40, 7, 129], [100, 64, 1]):  # two chunks: the second sees the first's prefix
        before = list(s.lens)
        q, k, v, pos, slots = s.new(counts)
        pk.pa_rotary_store_q8(q, q, k, v, pos, s.rotary, s.cache, slots, dev_err=s.err)
        # the sequences' blocks, read back side by side; the scratch's tables number them
        tables = s.padded()
        scratch = [torch.full((tables.numel(), s.bs, s.Hk, D), float("nan"), dtype=torch.bfloat16,
                              device=DEV) for _ in range(2)]
        pk.pa_load_kvcache_q8(*scratch, s.cache, tables.flatten(), dev_err=s.err)
        numbers = torch.arange(tables.numel(), dtype=torch.int32, device=DEV).view_as(tables)
        cu_q = np.concatenate([[0], np.cumsum(counts)])
        cu_k = np.concatenate([[0], np.cumsum(s.lens)])
        out = pk.pa_prefill_varlen(torch.empty_like(q), q, *scratch, numbers.contiguous(),
                                   ints(cu_q.tolist()), ints(cu_k.tolist()), max(counts),
                                   max(s.lens), dev_err=s.err)
        assert s.err.item() == 0
        kr, vr = (x.reshape(-1, s.Hk, D).double().cpu().numpy() for x in scratch)
        width = tables.shape[1]
        for i, n in enumerate(counts):
            total = s.lens[i]
            rows = i * width * s.bs + np.arange(total)
            p = np.arange(before[i], total)
            o, A, dev = att.attend(q[cu_q[i]:cu_q[i + 1]].double().cpu().numpy(), kr[rows], vr[rows],
                                   p, att.visible(p, total))
            att.assert_within(out[cu_q[i]:cu_q[i + 1]].double().cpu().numpy(), o,
                              att.bound(o, A, dev, torch.bfloat16))
    for _ in range(20):
        q, k, v, pos, slots = s.new([1, 1, 1])
        q = pk.pa_rotary_store_q8(torch.empty_like(q), q, k, v, pos, s.rotary, s.cache, slots,
                                  dev_err=s.err)
        out = pk.pa_decode_q8(torch.empty_like(q), q, s.cache, s.padded(), ints(s.lens),
                              dev_err=s.err)
        s.check_decode(q, out)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_steps_replayed_from_a_graph(fmt):
    """A captured step of rotary store and decode in a padded bucket, replayed over growing
    sequences while an eager step of its own runs between the replays."""
    s = Server(fmt, seed=3)
    s.tables, s.lens = [[], [], []], [0, 0, 0]
    q, k, v, pos, slots = s.new([30, 1, 15])
    pk.pa_rotary_store_q8(q, q, k, v, pos, s.rotary, s.cache, slots)
    B, width = 8, 8  # three sequences in a bucket of eight
    buf = dict(q=torch.zeros(B, 16, 128, device=DEV).bfloat16(),
               k=torch.zeros(B, 8, 128, device=DEV).bfloat16(),
               v=torch.zeros(B, 8, 128, device=DEV).bfloat16(),
               pos=torch.zeros(3, B, dtype=torch.int32, device=DEV),
               slots=torch.full((B,), -1, dtype=torch.int32, device=DEV),
               bt=torch.full((B, width), -1, dtype=torch.int32, device=DEV),
               ctx=torch.zeros(B, dtype=torch.int32, device=DEV))
    qo, out = torch.empty_like(buf["q"]), torch.empty_like(buf["q"])
    ws = pk.DecodeWorkspace(B, 16, 8, 128)

    def step():
        pk.pa_rotary_store_q8(qo, buf["q"], buf["k"], buf["v"], buf["pos"], s.rotary, s.cache,
                              buf["slots"], dev_err=s.err)
        pk.pa_decode_q8(out, qo, s.cache, buf["bt"], buf["ctx"], workspace=ws, dev_err=s.err)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(6):
        q, k, v, pos, slots = s.new([1, 1, 1])
        for name, x in (("q", q), ("k", k), ("v", v), ("slots", slots), ("ctx", ints(s.lens))):
            buf[name][:3] = x
        buf["pos"][:, :3] = pos
        buf["bt"][:3] = s.padded(width)
        graph.replay()
        assert not bool(out[3:].any())
        s.check_decode(qo[:3], out[:3])
        again = pk.pa_decode_q8(torch.empty_like(q), qo[:3].contiguous(), s.cache, buf["bt"][:3],
                                buf["ctx"][:3])
        s.check_decode(qo[:3], again)


def test_calls_on_other_streams_two_at_a_time():
    servers = [Server("e4m3", seed=5), Server("int8", seed=6)]
    streams = [torch.cuda.Stream() for _ in servers]
    want, state = [], []
    for s in servers:
        x = s.new([200, 333, 70])
        pk.pa_rotary_store_q8(x[0], *x[:4], s.rotary, s.cache, x[4])
        x = s.new([1, 1, 1])
        state.append((x, s.padded(), ints(s.lens)))
    torch.cuda.synchronize()
    for _ in range(10):
        outs = []
        for s, st, ((q, k, v, pos, slots), bt, ctx) in zip(servers, streams, state):
            out, qo = torch.empty_like(q), torch.empty_like(q)
            st.wait_stream(torch.cuda.current_stream())
            pk.pa_rotary_store_q8(qo, q, k, v, pos, s.rotary, s.cache, slots, stream=st)
            pk.pa_decode_q8(out, qo, s.cache, bt, ctx, stream=st)
            outs.append((qo, out))
        torch.cuda.synchronize()
        for s, (qo, out) in zip(servers, outs):
            s.check_decode(qo, out)


def test_two_graphs_with_their_own_workspaces():
    s = Server("e4m3", seed=8)
    x = s.new([500, 60, 411])
    pk.pa_rotary_store_q8(x[0], *x[:4], s.rotary, s.cache, x[4])
    bt, ctx = s.padded(), ints(s.lens)
    q = [torch.randn(3, 16, 128, device=DEV).bfloat16() for _ in range(2)]
    out = [torch.empty_like(t) for t in q]
    graphs = []
    for i in range(2):
        ws = pk.DecodeWorkspace(3, 16, 8, 128)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pk.pa_decode_q8(out[i], q[i], s.cache, bt, ctx, workspace=ws)
        graphs.append((g, ws))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for st, (g, _) in zip(streams, graphs):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for i in range(2):
        s.check_decode(q[i], out[i])


def test_a_block_read_by_two_sequences_and_loaded_twice():
    s = Server("int8", seed=9)
    x = s.new([64, 0, 0])
    pk.pa_rotary_store_q8(x[0], *x[:4], s.rotary, s.cache, x[4])
    s.tables = [s.tables[0], s.tables[0], s.tables[0][:2]]
    s.lens = [64, 50, 17]
    q = torch.randn(3, 16, 128, device=DEV).bfloat16()
    s.check_decode(q, pk.pa_decode_q8(torch.empty_like(q), q, s.cache, s.padded(), ints(s.lens)))
    t = s.tables[0]
    out = [torch.zeros(2, s.bs, 8, 128, dtype=torch.float16, device=DEV) for _ in range(2)]
    pk.pa_load_kvcache_q8(*out, s.cache, ints([t[1], t[1]]))
    assert torch.equal(out[0][0], out[0][1]) and torch.equal(out[1][0], out[1][1])
