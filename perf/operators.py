"""Timed cases of the attention calls beyond plain decode and prefill, each in two forms: the
plain one (elementary torch operations in fp32) and the library's own call.

- ``shared``: decode of a batch whose groups of sequences hold the same leading positions
  (``pa_decode_shared``);
- ``decode``: decode with modified scores: tanh cap, bias by distance, window, kept leading
  positions (``pa_decode_mod``);
- ``prefill``: chunked prefill with the same rules and a bidirectional prefix
  (``pa_prefill_mod``).

The caches are paged: ``[num_blocks, block_size, kv_heads, head_dim]`` behind int32 block
tables padded with -1. Lengths come from the case alone, values from the seed alone.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # four requests of one chat template, a few tokens each: the latency of one small call
        dict(name="shared_small", op="shared", dtype="bf16", heads=16, kv_heads=8, head_dim=128,
             block_size=16, groups="4", prefix="512", suffix_lo=1, suffix_hi=64, lens_seed=1),
        # a batch behind one few-shot prompt
        dict(name="shared_prompt", op="shared", dtype="bf16", heads=16, kv_heads=8, head_dim=128,
             block_size=256, groups="64", prefix="8192", suffix_lo=16, suffix_hi=1024,
             lens_seed=2),
        # several system prompts of different lengths with uneven groups, some alone
        dict(name="shared_groups", op="shared", dtype="fp16", heads=32, kv_heads=8, head_dim=64,
             block_size=16, groups="64 17 1 96 5 1 33 40", prefix="1008 2048 0 4096 304 700 1536 2000",
             suffix_lo=1, suffix_hi=700, lens_seed=3),
        # many requests over one long document, the largest: products, not bytes, bound it
        dict(name="shared_document", op="shared", dtype="bf16", heads=32, kv_heads=8, head_dim=128,
             block_size=256, groups="128", prefix="32768", suffix_lo=1, suffix_hi=1024,
             lens_seed=4),
        # one request of a model that caps its scores
        dict(name="decode_cap_one", op="decode", dtype="bf16", heads=16, kv_heads=8, head_dim=128,
             block_size=256, batch=1, ctx_lo=1000, ctx_hi=1000, cap=50.0, bias=False, window=0,
             sink=0, lens_seed=5),
        # the benchmark's decode batch under a cap
        dict(name="decode_cap", op="decode", dtype="bf16", heads=16, kv_heads=8, head_dim=128,
             block_size=256, batch=256, ctx_lo=100, ctx_hi=2048, cap=50.0, bias=False, window=0,
             sink=0, lens_seed=6),
        # a sliding-window layer with kept leading tokens, contexts far past the window
        dict(name="decode_window", op="decode", dtype="fp16", heads=32, kv_heads=8, head_dim=64,
             block_size=16, batch=200, ctx_lo=500, ctx_hi=32768, cap=0.0, bias=False, window=1000,
             sink=4, lens_seed=7),
        # long contexts with a bias by distance
        dict(name="decode_bias_long", op="decode", dtype="bf16", heads=32, kv_heads=8, head_dim=128,
             block_size=256, batch=8, ctx_lo=32768, ctx_hi=131072, cap=0.0, bias=True, window=0,
             sink=0, lens_seed=8),
        # two short prompts under a cap
        dict(name="prefill_cap_small", op="prefill", dtype="bf16", heads=16, kv_heads=8,
             head_dim=128, block_size=256, seqs=2, cached_lo=0, cached_hi=300, new_lo=17,
             new_hi=130, cap=50.0, bias=False, window=0, sink=0, prefix=0, causal=True,
             lens_seed=9),
        # the benchmark's chunked prefill under a cap
        dict(name="prefill_cap", op="prefill", dtype="bf16", heads=16, kv_heads=8, head_dim=128,
             block_size=256, seqs=32, cached_lo=0, cached_hi=2048, new_lo=100, new_hi=1024,
             cap=50.0, bias=False, window=0, sink=0, prefix=0, causal=True, lens_seed=10),
        # long prompts of a sliding-window layer with kept leading tokens
        dict(name="prefill_window", op="prefill", dtype="fp16", heads=32, kv_heads=8, head_dim=64,
             block_size=64, seqs=3, cached_lo=0, cached_hi=4096, new_lo=4000, new_hi=8192,
             cap=0.0, bias=False, window=1024, sink=16, prefix=0, causal=True, lens_seed=11),
        # a bidirectional prompt before causal text, with a bias by distance
        dict(name="prefill_prefix_bias", op="prefill", dtype="bf16", heads=32, kv_heads=4,
             head_dim=128, block_size=128, seqs=6, cached_lo=0, cached_hi=777, new_lo=600,
             new_hi=4096, cap=0.0, bias=True, window=0, sink=0, prefix=500, causal=True,
             lens_seed=12),
    ]


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["shared", "decode", "prefill"])
    c = dict(op=op, dtype=rng.choice(["bf16", "fp16"]), head_dim=rng.choice([64, 128]),
             lens_seed=rng.randrange(1 << 30))
    kv = c["kv_heads"] = rng.choice([1, 2, 4, 8, 8, 8])
    if op == "shared":
        c["heads"] = kv * rng.choice([1, 2, 3, 4, 5, 8])
        c["block_size"] = bs = rng.choice([16, 16, 32, 48, 128, 256])
        sizes = [_log_int(rng, 1, 96) for _ in range(_log_int(rng, 1, 8))]
        prefix = [_log_int(rng, 64, 16384) // bs * bs for _ in sizes]
        c["groups"] = " ".join(map(str, sizes))
        c["prefix"] = " ".join(map(str, prefix))
        c["suffix_lo"] = 1
        c["suffix_hi"] = _log_int(rng, 1, 1024)
        return c
    rule = rng.choice(["cap", "bias", "window", "cap bias", "bias window", "cap window"])
    c["cap"] = rng.choice([20.0, 30.0, 50.0]) if "cap" in rule else 0.0
    c["bias"] = "bias" in rule
    c["window"] = _log_int(rng, 1, 4096) if "window" in rule else 0
    c["sink"] = rng.choice([0, 1, 4, 64]) if c["window"] else 0
    if op == "decode":
        c["heads"] = kv * rng.choice([1, 2, 3, 4, 6, 8])
        c["block_size"] = rng.choice([16, 16, 20, 64, 256])
        c["batch"] = _log_int(rng, 1, 256)
        c["ctx_hi"] = min(_log_int(rng, 16, 65536), 400000 // c["batch"])
        c["ctx_lo"] = rng.randint(1, c["ctx_hi"])
    else:
        c["heads"] = kv * rng.choice([1, 2, 4, 8])
        c["block_size"] = rng.choice([16, 32, 128, 256])
        c["seqs"] = _log_int(rng, 1, 16)
        c["new_hi"] = min(_log_int(rng, 8, 4096), 12000 // c["seqs"])
        c["new_lo"] = rng.randint(1, c["new_hi"])
        c["cached_lo"], c["cached_hi"] = 0, _log_int(rng, 1, 2048) - 1
        c["causal"] = rng.random() < 0.85
        c["prefix"] = rng.choice([0, 0, _log_int(rng, 1, 1000)])
    return c


# ---------------------------------------------------------------------------- the lengths
def _ints(text):
    return [int(w) for w in text.split()]


def _lengths(case):
    """Per sequence (cached, new) tokens; the decode calls have one new token each."""
    rng = random.Random(case["lens_seed"])
    if case["op"] == "shared":
        return [(p + rng.randint(case["suffix_lo"], case["suffix_hi"]) - 1, 1)
                for n, p in zip(_ints(case["groups"]), _ints(case["prefix"])) for _ in range(n)]
    if case["op"] == "decode":
        return [(rng.randint(case["ctx_lo"], case["ctx_hi"]) - 1, 1) for _ in range(case["batch"])]
    return [(rng.randint(case["cached_lo"], case["cached_hi"]),
             rng.randint(case["new_lo"], case["new_hi"])) for _ in range(case["seqs"])]


def _visible(case, c, n):
    """(query, key) pairs that the rules let through, and the keys that any query sees, of a
    sequence with c cached and n new tokens."""
    if case["op"] == "shared":
        return c + n, c + n
    total, window = c + n, case["window"]
    prefix = case.get("prefix", 0)
    keep = max(case["sink"], prefix)
    pairs = 0
    for p in range(c, c + n):
        hi = min(total, max(p + 1, prefix)) if case.get("causal", True) else total
        low = max(0, p - window + 1) if window else 0
        pairs += min(keep, hi) + max(0, hi - max(low, keep)) if low > keep else hi
    low0 = max(0, c - window + 1) if window else 0
    keys = total if low0 <= keep else min(keep, total) + total - low0
    return pairs, keys


def work(case):
    lens = _lengths(case)
    h, d = case["heads"], case["head_dim"]
    row = 2 * case["kv_heads"] * d * 2  # K and V of one position
    new = sum(n for _, n in lens)
    pairs = keys = 0
    for c, n in lens:
        a, b = _visible(case, c, n)
        pairs += a
        keys += b
    if case["op"] == "shared":  # shared positions count once for each group
        keys -= sum((n - 1) * p for n, p in zip(_ints(case["groups"]), _ints(case["prefix"])))
    blocks = sum(-(-(c + n) // case["block_size"]) for c, n in lens)
    return {"bytes": keys * row + 2 * new * h * d * 2 + 4 * blocks + 4 * len(lens),
            "flops": 4 * h * d * pairs}


# ---------------------------------------------------------------------------- the inputs
def _tables(case, lens):
    """Block tables over shuffled physical blocks; the members of a group share the blocks
    that lie wholly inside its prefix. Returns (rows, number of blocks)."""
    bs = case["block_size"]
    shared = {}
    if case["op"] == "shared":
        first = 0
        for n, p in zip(_ints(case["groups"]), _ints(case["prefix"])):
            for b in range(first + 1, first + n):
                shared[b] = (first, p // bs)
            first += n
    rows, used = [], 0
    for b, (c, n) in enumerate(lens):
        need = -(-(c + n) // bs)
        lead, k = shared.get(b, (b, 0))
        row = rows[lead][:k] if k else []
        rows.append(row + list(range(used, used + need - len(row))))
        used += need - len(row)
    order = list(range(used + 3))
    random.Random(case["lens_seed"] + 1).shuffle(order)
    return [[order[i] for i in row] for row in rows], used + 3


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = _TYPES[case["dtype"]]
    lens = _lengths(case)
    rows, nb = _tables(case, lens)
    h, hk, d, bs = case["heads"], case["kv_heads"], case["head_dim"], case["block_size"]
    total = [c + n for c, n in lens]
    new = [n for _, n in lens]
    width = max(len(r) for r in rows)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev, dtype=dt)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    st = dict(case=case, lens=lens, rows=rows)
    st["k"], st["v"] = normal(nb, bs, hk, d), normal(nb, bs, hk, d)
    # queries of a capped model reach into the cap's bend
    st["q"] = normal(sum(new), h, d) * (4.0 if case.get("cap") else 1.0)
    st["tables"] = ints([r + [-1] * (width - len(r)) for r in rows])
    st["total"] = ints(total)
    st["out"] = torch.empty_like(st["q"])
    if case.get("bias"):
        st["slopes"] = torch.tensor([2.0 ** (-8.0 * (i + 1) / h) for i in range(h)], device=dev)
    if case["op"] == "shared":
        starts = [0]
        for n in _ints(case["groups"]):
            starts.append(starts[-1] + n)
        st["starts"], st["prefix"] = ints(starts), ints(_ints(case["prefix"]))
    if case["op"] == "prefill":
        cu_q, cu_k = [0], [0]
        for c, n in lens:
            cu_q.append(cu_q[-1] + n)
            cu_k.append(cu_k[-1] + c + n)
        st["cu_q"], st["cu_k"] = ints(cu_q), ints(cu_k)
        st["max_q"], st["max_k"] = max(new), max(total)
        if case["prefix"]:
            st["prefix"] = ints([case["prefix"]] * len(lens))
    if own:
        import paged_kv_cache_107_gb300 as pk
        if case["op"] == "shared":
            st["ws"] = pk.SharedDecodeWorkspace(len(lens), h, hk, d)
        else:
            st["mod"] = pk.ScoreMod(softcap=case["cap"], slopes=st.get("slopes"),
                                    window=case["window"], sink=case["sink"],
                                    prefix_lens=st.get("prefix"))
            if case["op"] == "decode":
                st["ws"] = pk.DecodeWorkspace(len(lens), h, hk, d)
    return st


# ---------------------------------------------------------------------------- the calls
def _own(st):
    import paged_kv_cache_107_gb300 as pk
    op = st["case"]["op"]
    if op == "shared":
        return pk.pa_decode_shared(st["out"], st["q"], st["k"], st["v"], st["tables"], st["total"],
                                   st["starts"], st["prefix"], workspace=st["ws"])
    if op == "decode":
        return pk.pa_decode_mod(st["out"], st["q"], st["k"], st["v"], st["tables"], st["total"],
                                st["mod"], workspace=st["ws"])
    return pk.pa_prefill_mod(st["out"], st["q"], st["k"], st["v"], st["tables"], st["cu_q"],
                             st["cu_k"], st["max_q"], st["max_k"], st["mod"],
                             causal=st["case"]["causal"])


def _rows(st, b, total):
    """The cache rows of sequence b's positions."""
    bs = st["case"]["block_size"]
    t = torch.arange(total, device="cuda")
    return st["tables"][b].long()[t // bs] * bs + t % bs


def run(state):
    if own:
        return _own(state)
    st, case = state, state["case"]
    h, hk, d = case["heads"], case["kv_heads"], case["head_dim"]
    g = h // hk
    k_rows, v_rows = st["k"].view(-1, hk, d), st["v"].view(-1, hk, d)
    out = torch.empty_like(st["q"])
    first = 0
    for b, (c, n) in enumerate(st["lens"]):
        total = c + n
        rows = _rows(st, b, total)
        # [kv_heads, n * g, head_dim] against [kv_heads, total, head_dim]
        q = (st["q"][first:first + n].float() / math.sqrt(d)).view(n, hk, g, d).transpose(0, 1)
        k, v = k_rows[rows].float().transpose(0, 1), v_rows[rows].float().transpose(0, 1)
        s = torch.matmul(q.reshape(hk, n * g, d), k.transpose(1, 2)).view(hk, n, g, total)
        if case.get("cap"):
            s = case["cap"] * torch.tanh(s / case["cap"])
        if case["op"] != "shared":
            p = torch.arange(c, total, device="cuda")[:, None]
            t = torch.arange(total, device="cuda")[None, :]
            if case["bias"]:
                s = s - st["slopes"].view(hk, 1, g, 1) * (p - t).abs()[:, None, :]
            prefix = case.get("prefix", 0)
            hide = torch.zeros(n, total, dtype=torch.bool, device="cuda")
            if case.get("causal", True):
                hide |= (t > p) & (t >= prefix)
            if case["window"]:
                hide |= (t <= p - case["window"]) & (t >= max(case["sink"], prefix))
            s = s.masked_fill(hide[:, None, :], -math.inf)
        e = torch.exp(s - s.amax(-1, keepdim=True))
        o = torch.matmul(e.view(hk, n * g, total), v) / e.sum(-1).view(hk, n * g, 1)
        out[first:first + n] = o.view(hk, n, g, d).transpose(0, 1).reshape(n, h, d).to(out.dtype)
        first += n
    return out


def exact(case, seed):
    """The same attention in 64 bits, one query head at a time over the keys it may see."""
    st = prepare(case, seed)
    h, hk, d, bs = case["heads"], case["kv_heads"], case["head_dim"], case["block_size"]
    dev = st["q"].device
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=dev)
    at = 0
    for b, (c, n) in enumerate(st["lens"]):
        total = c + n
        blocks = torch.tensor(st["rows"][b], device=dev)
        keys = st["k"][blocks].reshape(-1, hk, d)[:total].permute(1, 0, 2).double()
        vals = st["v"][blocks].reshape(-1, hk, d)[:total].permute(1, 0, 2).double()
        dist = torch.arange(c, total, device=dev).view(n, 1) - torch.arange(total, device=dev)
        pos = torch.arange(total, device=dev).expand(n, total)
        see = torch.ones(n, total, dtype=torch.bool, device=dev)
        if case["op"] != "shared":
            lead = case.get("prefix", 0)
            if case.get("causal", True):
                see &= (dist >= 0) | (pos < lead)
            if case["window"] > 0:
                see &= (dist < case["window"]) | (pos < lead) | (pos < case["sink"])
        for i in range(h):
            j = i * hk // h
            x = st["q"][at:at + n, i].double() @ keys[j].transpose(0, 1) * d ** -0.5
            if case.get("cap"):
                x = torch.tanh(x / case["cap"]) * case["cap"]
            if case.get("bias"):
                x = x - st["slopes"][i].double() * dist.abs()
            x = torch.where(see, x, torch.full((), -math.inf, dtype=torch.float64, device=dev))
            out[at:at + n, i] = torch.softmax(x, dim=-1) @ vals[j]
        at += n
    return out
