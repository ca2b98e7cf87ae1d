"""Timed cases of the calls around an 8-bit cache and of rotary positions, each in two forms: the
plain one (elementary torch operations in fp32) and the library's own call.

- ``rotary``: rotary positions with several axes applied to new queries and keys, keys and
  values written to the 16-bit cache (``pa_rotary_store``);
- ``store``: new keys and values written to an 8-bit cache, one scale for each token and KV
  head, and read back (``pa_store_kvcache_q8``, ``pa_load_kvcache_q8``);
- ``load``: listed blocks of an 8-bit cache read back as 16-bit blocks (``pa_load_kvcache_q8``);
- ``decode``: one query token per sequence over the 8-bit cache (``pa_decode_q8``).

The caches are paged: ``[num_blocks, block_size, kv_heads, head_dim]``; an 8-bit cache has its
scales beside it, ``[num_blocks, kv_heads, block_size]`` in fp32. ``e4m3`` scales are powers of
two, the least for which the row's largest value stays within 448; ``int8`` scales are the row's
largest value / 127. Lengths and positions come from the case alone, values from the seed alone.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
_CODES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def listed():
    return [
        # the next token of one request, at a far position: the latency of one small call
        dict(name="rotary_one", op="rotary", dtype="bf16", heads=16, kv_heads=8, head_dim=128,
             block_size=256, tokens=1, rotary_dim=128, axes="16 24 24", adjacent=False,
             base=1000000.0, packed=False, text=1, grid_h=0, grid_w=0, pos0=100000, pad=0,
             lens_seed=1),
        # an image prompt of odd size: queries, keys and values in one packed projection,
        # half of each head rotated, pairs side by side, two axes
        dict(name="rotary_image", op="rotary", dtype="fp16", heads=32, kv_heads=8, head_dim=64,
             block_size=16, tokens=4095, rotary_dim=32, axes="8 8", adjacent=True, base=10000.0,
             packed=True, text=37, grid_h=45, grid_w=61, pos0=0, pad=0, lens_seed=2),
        # the benchmark's chunked prefill with video frames between the text
        dict(name="rotary_video", op="rotary", dtype="bf16", heads=16, kv_heads=8, head_dim=128,
             block_size=256, tokens=17556, rotary_dim=128, axes="16 24 24", adjacent=False,
             base=1000000.0, packed=False, text=500, grid_h=26, grid_w=37, pos0=4096, pad=0,
             lens_seed=3),
        # the benchmark's decode batch, padded by a graph's empty rows
        dict(name="store_step", op="store", dtype="bf16", codes="e4m3", heads=16, kv_heads=8,
             head_dim=128, block_size=16, tokens=256, packed=True, pad=9, spread=True, lens_seed=4),
        # an odd prompt of a model with small heads
        dict(name="store_odd", op="store", dtype="fp16", codes="e4m3", heads=20, kv_heads=5,
             head_dim=64, block_size=32, tokens=1999, packed=True, pad=0, spread=False,
             lens_seed=5),
        # the benchmark's chunked prefill
        dict(name="store_prefill", op="store", dtype="bf16", codes="int8", heads=16, kv_heads=8,
             head_dim=128, block_size=256, tokens=17556, packed=False, pad=0, spread=False,
             lens_seed=6),
        # one request's prefix, read back for its next chunk
        dict(name="load_prefix", op="load", dtype="fp16", codes="int8", kv_heads=4, head_dim=64,
             block_size=16, blocks=65, missing=5, lens_seed=7),
        # the prefixes of a batch of chunks
        dict(name="load_batch", op="load", dtype="bf16", codes="e4m3", kv_heads=8, head_dim=128,
             block_size=256, blocks=150, missing=0, lens_seed=8),
        # one request: latency
        dict(name="decode_one", op="decode", dtype="bf16", codes="e4m3", heads=16, kv_heads=8,
             head_dim=128, block_size=256, batch=1, ctx_lo=1000, ctx_hi=1000, lens_seed=9),
        # the benchmark's decode batch
        dict(name="decode_batch", op="decode", dtype="bf16", codes="e4m3", heads=16, kv_heads=8,
             head_dim=128, block_size=256, batch=256, ctx_lo=100, ctx_hi=2048, lens_seed=10),
        # small heads in wider groups, short blocks
        dict(name="decode_groups", op="decode", dtype="fp16", codes="int8", heads=32, kv_heads=8,
             head_dim=64, block_size=16, batch=200, ctx_lo=1, ctx_hi=4096, lens_seed=11),
        # a few long contexts, the largest
        dict(name="decode_long", op="decode", dtype="bf16", codes="int8", heads=32, kv_heads=8,
             head_dim=128, block_size=256, batch=8, ctx_lo=32768, ctx_hi=131072, lens_seed=12),
    ]


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rotary", "store", "load", "decode", "decode"])
    d = rng.choice([64, 128])
    c = dict(op=op, dtype=rng.choice(["bf16", "fp16"]), head_dim=d,
             kv_heads=rng.choice([1, 2, 3, 4, 8, 8, 8, 12, 16]),
             block_size=rng.choice([8, 16, 16, 32, 48, 128, 256]), lens_seed=rng.randrange(1 << 30))
    if op != "rotary":
        c["codes"] = rng.choice(["e4m3", "int8"])
    if op != "load":
        c["heads"] = c["kv_heads"] * rng.choice([1, 2, 3, 4, 6, 8])
    if op in ("rotary", "store"):
        row = (c["heads"] + 2 * c["kv_heads"]) * d
        c["tokens"] = min(_log_int(rng, 1, 32768), 80000000 // row)
        c["packed"] = rng.random() < 0.5
        c["pad"] = rng.choice([0, 0, 2, 7])
    if op == "rotary":
        c["rotary_dim"] = rot = rng.choice([d, d, d // 2, d // 4])
        parts, left = [], rot // 2
        for _ in range(rng.randint(0, 2)):
            parts.append(rng.randint(1, max(1, left // 2)))
            left -= parts[-1]
        c["axes"] = " ".join(map(str, parts + [left]))
        c["adjacent"] = rng.random() < 0.4
        c["base"] = rng.choice([10000.0, 500000.0, 1000000.0])
        c["text"] = rng.randint(0, c["tokens"])
        c["grid_h"], c["grid_w"] = _log_int(rng, 1, 64), _log_int(rng, 1, 64)
        c["pos0"] = _log_int(rng, 1, 1000000) - 1
    elif op == "store":
        c["spread"] = c["tokens"] <= 512 and rng.random() < 0.5
    elif op == "load":
        c["blocks"] = _log_int(rng, 1, max(1, 80000000 // (c["block_size"] * c["kv_heads"] * d)))
        c["missing"] = rng.choice([0, 0, 3, 10])
    else:
        c["batch"] = _log_int(rng, 1, 256)
        c["ctx_hi"] = min(_log_int(rng, 16, 65536),
                          400000000 // (c["batch"] * c["kv_heads"] * d))
        c["ctx_lo"] = rng.randint(1, c["ctx_hi"])
    return c


# ---------------------------------------------------------------------------- the layout
def _ints(text):
    return [int(w) for w in text.split()]


def _lengths(case):
    """Tokens in the cache of each sequence (decode)."""
    rng = random.Random(case["lens_seed"])
    return [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["batch"])]


def _slots(case):
    """(slot of each new token, number of blocks): a prompt's tokens fill shuffled blocks from
    the middle of the first on, a decode batch's sit in a block each; every pad-th is -1."""
    rng = random.Random(case["lens_seed"] + 1)
    n, bs = case["tokens"], case["block_size"]
    start = 0 if case.get("spread") else bs // 2
    need = n if case.get("spread") else -(-(n + start) // bs)
    order = list(range(need))
    rng.shuffle(order)
    if case.get("spread"):
        slots = [b * bs + rng.randrange(bs) for b in order]
    else:
        slots = [order[(start + i) // bs] * bs + (start + i) % bs for i in range(n)]
    pad = case["pad"]
    return [-1 if pad and i % pad == pad - 1 else s for i, s in enumerate(slots)], need


def _inv_freq(case):
    rot = case["rotary_dim"]
    return [case["base"] ** (-2.0 * i / rot) for i in range(rot // 2)]


def _axis_of(case):
    return [a for a, n in enumerate(_ints(case["axes"])) for _ in range(n)]


def _positions(case):
    """int32 [axes, tokens]: text counts all axes up together; after it come frames of
    grid_h x grid_w patches at (frame, row, column), the frames' rows and columns alike."""
    n, text = case["tokens"], case["text"]
    i = torch.arange(n, device="cuda")
    j = (i - text).clamp(min=0)
    gh, gw = max(case["grid_h"], 1), max(case["grid_w"], 1)
    where = [j // (gh * gw), j // gw % gh, j % gw]
    axes = len(_ints(case["axes"]))
    where = {1: [j], 2: where[1:], 3: where}[axes]
    rows = [case["pos0"] + torch.where(i < text, i, text + w) for w in where]
    return torch.stack(rows).to(torch.int32)


def work(case):
    hk, d = case["kv_heads"], case["head_dim"]
    if case["op"] == "decode":
        lens = _lengths(case)
        keys, h = sum(lens), case["heads"]
        blocks = sum(-(-n // case["block_size"]) for n in lens)
        return {"bytes": keys * hk * 2 * (d + 4) + 4 * len(lens) * (h * d + 1) + 4 * blocks,
                "flops": 4 * h * d * keys}
    if case["op"] == "load":
        n, bs = case["blocks"], case["block_size"]
        full = n - (n // case["missing"] if case["missing"] else 0)
        return {"bytes": full * bs * hk * 2 * (3 * d + 4) + 4 * n, "flops": full * bs * hk * 2 * d}
    slots, nb = _slots(case)
    n, kept = len(slots), sum(s >= 0 for s in slots)
    if case["op"] == "store":  # rows in, codes and scales out, then the blocks read back
        rows = nb * case["block_size"]
        return {"bytes": kept * hk * 2 * (3 * d + 4) + rows * hk * 2 * (3 * d + 4) + 4 * n + 4 * nb,
                "flops": kept * hk * 2 * 4 * d + rows * hk * 2 * d}
    h, rot = case["heads"], case["rotary_dim"]
    axes = len(_ints(case["axes"]))
    return {"bytes": 4 * n * h * d + 8 * kept * hk * d + 4 * n * (axes + 1),
            "flops": 3 * n * (h + hk) * rot}


# ---------------------------------------------------------------------------- the inputs
def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = _TYPES[case["dtype"]]
    hk, d, bs = case["kv_heads"], case["head_dim"], case["block_size"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev, dtype=dt)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    st = dict(case=case)
    op = case["op"]
    if op in ("rotary", "store"):
        slots, nb = _slots(case)
        n, h = case["tokens"], case["heads"]
        if case["packed"]:  # one projection's rows: queries, keys, values
            rows = normal(n, h + 2 * hk, d)
            st["q"], st["k"], st["v"] = rows[:, :h], rows[:, h:h + hk], rows[:, h + hk:]
        else:
            st["q"], st["k"], st["v"] = normal(n, h, d), normal(n, hk, d), normal(n, hk, d)
        st["slots"] = ints(slots)
        st["kept"] = torch.tensor([i for i, s in enumerate(slots) if s >= 0], device=dev)
    elif op == "load":
        nb = case["blocks"]
        order = list(range(nb))
        random.Random(case["lens_seed"]).shuffle(order)
        gap = case["missing"]
        listed_blocks = [-1 if gap and i % gap == gap - 1 else b for i, b in enumerate(order)]
        st["blocks"] = ints(listed_blocks)
        st["have"] = torch.tensor([i for i, b in enumerate(listed_blocks) if b >= 0], device=dev)
    else:
        lens = _lengths(case)
        need = [-(-n // bs) for n in lens]
        nb = sum(need) + 2
        order = list(range(nb))
        random.Random(case["lens_seed"] + 1).shuffle(order)
        rows, at = [], 0
        for k in need:
            rows.append(order[at:at + k])
            at += k
        width = max(need)
        st["lens"], st["rows"] = lens, rows
        st["tables"] = ints([r + [-1] * (width - len(r)) for r in rows])
        st["total"] = ints(lens)
        st["q"] = normal(len(lens), case["heads"], d)
        st["out"] = torch.empty_like(st["q"])
    if op == "rotary":
        st["pos"] = _positions(case)
        st["q_out"] = torch.empty(st["q"].shape, dtype=dt, device=dev)
        st["k_cache"] = torch.zeros(nb, bs, hk, d, dtype=dt, device=dev)
        st["v_cache"] = torch.zeros(nb, bs, hk, d, dtype=dt, device=dev)
        st["freq"] = torch.tensor(_inv_freq(case), dtype=torch.float64, device=dev)
        st["axis"] = torch.tensor(_axis_of(case), device=dev)
    if op == "store":
        st["blocks"] = torch.arange(nb, dtype=torch.int32, device=dev)
    if op in ("store", "load"):
        st["k_out"] = torch.zeros(nb, bs, hk, d, dtype=dt, device=dev)
        st["v_out"] = torch.zeros(nb, bs, hk, d, dtype=dt, device=dev)
    if op == "store":
        st["kc"] = torch.zeros(nb, bs, hk, d, dtype=_CODES[case["codes"]], device=dev)
        st["vc"] = torch.zeros_like(st["kc"])
        st["ks"] = torch.zeros(nb, hk, bs, device=dev)
        st["vs"] = torch.zeros(nb, hk, bs, device=dev)
    elif op in ("load", "decode"):
        # caches as a store leaves them: rows of normal values, quantised
        for c, s in (("kc", "ks"), ("vc", "vs")):
            codes = torch.empty(nb, bs, hk, d, dtype=_CODES[case["codes"]], device=dev)
            scales = torch.empty(nb, hk, bs, device=dev)
            step = max(1, (1 << 26) // (bs * hk * d))
            for i in range(0, nb, step):
                part = normal(min(step, nb - i), bs, hk, d)
                y, z = _quantise(case["codes"], part)
                codes[i:i + step] = y.to(codes.dtype)
                scales[i:i + step] = z.transpose(1, 2)
            st[c], st[s] = codes, scales
    if own:
        import paged_kv_cache_107_gb300 as pk
        if op == "rotary":
            st["rotary"] = pk.Rotary(d, inv_freq=_inv_freq(case), axes=_axis_of(case),
                                     adjacent=case["adjacent"])
        else:
            st["cache"] = pk.Q8Cache.of(st["kc"], st["vc"], st["ks"], st["vs"])
        if op == "decode":
            st["ws"] = pk.DecodeWorkspace(len(lens), case["heads"], hk, d)
    return st


# ---------------------------------------------------------------------------- the calls
def _own(st):
    import paged_kv_cache_107_gb300 as pk
    op = st["case"]["op"]
    if op == "rotary":
        pk.pa_rotary_store(st["q_out"], st["q"], st["k"], st["v"], st["pos"], st["rotary"],
                           st["k_cache"], st["v_cache"], st["slots"])
        return st["q_out"], st["k_cache"], st["v_cache"]
    if op == "decode":
        return pk.pa_decode_q8(st["out"], st["q"], st["cache"], st["tables"], st["total"],
                               workspace=st["ws"])
    if op == "store":
        pk.pa_store_kvcache_q8(st["k"], st["v"], st["cache"], st["slots"])
    pk.pa_load_kvcache_q8(st["k_out"], st["v_out"], st["cache"], st["blocks"])
    if op == "store":
        return st["k_out"], st["v_out"], st["ks"], st["vs"]
    return st["k_out"], st["v_out"]


def _quantise(kind, x):
    """(codes as fp32 values, scales) of rows of values, a scale for each row."""
    x = x.float()
    top = x.abs().amax(-1)
    if kind == "e4m3":  # top = m 2^e, m of [0.5, 1): 448 = 0.875 * 2^9
        m, e = torch.frexp(top)
        e = (e - 9 + (m > 0.875)).clamp(min=-126)
        scale = torch.where(top > 0, torch.ldexp(torch.ones_like(top), e), 0.0)
        y = torch.ldexp(x, -e[..., None]).to(torch.float8_e4m3fn).float()
    else:
        base = top.clamp(min=127.0 * 2.0 ** -126)
        scale = torch.where(top > 0, base / 127.0, 0.0)
        y = torch.round(x * 127.0 / base[..., None])
    return y, scale


def _rotate(x, cos, sin, rot, adjacent):
    """Pairs of the first rot dims turned by cos, sin [tokens, 1, rot / 2]."""
    x = x.float()
    head, rest = x[..., :rot], x[..., rot:]
    if adjacent:
        a, b = head[..., 0::2], head[..., 1::2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, rest), -1)


def run(state):
    if own:
        return _own(state)
    st, case = state, state["case"]
    op, hk, d = case["op"], case["kv_heads"], case["head_dim"]
    if op == "rotary":
        angle = st["pos"][st["axis"]].double() * st["freq"][:, None]
        cos, sin = torch.cos(angle).float().t()[:, None], torch.sin(angle).float().t()[:, None]
        rot, adjacent = case["rotary_dim"], case["adjacent"]
        st["q_out"].copy_(_rotate(st["q"], cos, sin, rot, adjacent))
        kept = st["kept"]
        rows = st["slots"][kept].long()
        k = _rotate(st["k"], cos, sin, rot, adjacent)
        st["k_cache"].view(-1, hk, d)[rows] = k[kept].to(st["k_cache"].dtype)
        st["v_cache"].view(-1, hk, d)[rows] = st["v"][kept]
        return st["q_out"], st["k_cache"], st["v_cache"]
    if op == "store":
        kept = st["kept"]
        slot = st["slots"][kept].long()
        blk, off = slot // case["block_size"], slot % case["block_size"]
        for x, out, scales in ((st["k"], st["k_out"], st["ks"]), (st["v"], st["v_out"], st["vs"])):
            y, scale = _quantise(case["codes"], x[kept])
            scales[blk, :, off] = scale
            out[blk, off] = (y * scale[..., None]).to(out.dtype)
        return st["k_out"], st["v_out"], st["ks"], st["vs"]
    if op == "load":
        have = st["have"]
        blocks = st["blocks"][have].long()
        for c, s, o in (("kc", "ks", "k_out"), ("vc", "vs", "v_out")):
            x = st[c][blocks].float() * st[s][blocks].transpose(1, 2)[..., None]
            st[o][have] = x.to(st[o].dtype)
        return st["k_out"], st["v_out"]
    h, bs = case["heads"], case["block_size"]
    g = h // hk
    out = torch.empty_like(st["q"])
    for b, n in enumerate(st["lens"]):
        blocks = st["tables"][b, :-(-n // bs)].long()
        # [kv_heads, n, head_dim]
        k, v = ((st[c][blocks].float() * st[s][blocks].transpose(1, 2)[..., None])
                .view(-1, hk, d)[:n].transpose(0, 1) for c, s in (("kc", "ks"), ("vc", "vs")))
        q = (st["q"][b].float() / math.sqrt(d)).view(hk, g, d)
        s = torch.matmul(q, k.transpose(1, 2))
        e = torch.exp(s - s.amax(-1, keepdim=True))
        out[b] = (torch.matmul(e, v) / e.sum(-1, keepdim=True)).view(h, d).to(out.dtype)
    return out


def exact(case, seed):
    """The same from the definitions in 64 bits: values on their 8-bit grids by arithmetic,
    pairs turned as complex numbers, attention one query head at a time."""
    st = prepare(case, seed)
    op, hk, d, bs = case["op"], case["kv_heads"], case["head_dim"], case["block_size"]
    f64, dev = torch.float64, "cuda"
    if op == "rotary":
        rot = case["rotary_dim"]
        turn = torch.zeros(case["tokens"], 1, rot // 2, dtype=torch.complex128, device=dev)
        for i, (a, f) in enumerate(zip(_axis_of(case), _inv_freq(case))):
            angle = st["pos"][a].to(f64) * f
            turn[:, 0, i] = torch.polar(torch.ones_like(angle), angle)

        def rotated(x):
            y = x.to(f64)
            re = y[..., 0:rot:2] if case["adjacent"] else y[..., :rot // 2]
            im = y[..., 1:rot:2] if case["adjacent"] else y[..., rot // 2:rot]
            z = torch.complex(re.contiguous(), im.contiguous()) * turn
            y = y.clone()
            if case["adjacent"]:
                y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
            else:
                y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
            return y

        caches = []
        for rows in (rotated(st["k"]), st["v"].to(f64)):
            pool = torch.zeros(st["k_cache"].shape[0] * bs, hk, d, dtype=f64, device=dev)
            pool[st["slots"][st["kept"]].long()] = rows[st["kept"]]
            caches.append(pool.view(st["k_cache"].shape))
        return rotated(st["q"]), caches[0], caches[1]
    if op == "store":
        values, scales = [], []
        slot = st["slots"][st["kept"]].long()
        for x in (st["k"], st["v"]):
            x = x[st["kept"]].to(f64)
            top = x.abs().max(dim=-1, keepdim=True).values
            if case["codes"] == "int8":
                z = top / 127
                y = torch.round(torch.where(top > 0, x * 127 / top, 0.0))
            else:
                z = torch.exp2(torch.ceil(torch.log2(top / 448)))
                z = torch.where(top > 224 * z, z, z / 2)  # log2 is off by a bit at powers of two
                z = torch.where(top > 448 * z, z * 2, z)
                y = x / z
                grid = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
                y = torch.round(y / grid) * grid
            z = torch.where(top > 0, z, 0.0)
            pool = torch.zeros(st["k_out"].shape, dtype=f64, device=dev)
            pool.view(-1, hk, d)[slot] = torch.where(top > 0, y * z, 0.0)
            held = torch.zeros(st["k_out"].shape[0] * bs, hk, dtype=f64, device=dev)
            held[slot] = z[..., 0]
            values.append(pool)
            scales.append(held.view(-1, bs, hk).transpose(1, 2))
        return values[0], values[1], scales[0], scales[1]
    if op == "load":
        outs = []
        for c, s in (("kc", "ks"), ("vc", "vs")):
            pool = torch.zeros(st["k_out"].shape, dtype=f64, device=dev)
            for i, b in enumerate(st["blocks"].tolist()):
                if b >= 0:
                    pool[i] = st[c][b].to(f64) * st[s][b].to(f64).t()[:, :, None]
            outs.append(pool)
        return outs[0], outs[1]
    out = torch.zeros(st["q"].shape, dtype=f64, device=dev)
    for b, n in enumerate(st["lens"]):
        blocks = torch.tensor(st["rows"][b], device=dev)
        for j in range(hk):
            k, v = ((st[c][blocks, :, j].to(f64) * st[s][blocks, j].to(f64)[..., None])
                    .reshape(-1, d)[:n] for c, s in (("kc", "ks"), ("vc", "vs")))
            for i in range(j * case["heads"] // hk, (j + 1) * case["heads"] // hk):
                p = torch.softmax(k @ st["q"][b, i].to(f64) * d ** -0.5, dim=0)
                out[b, i] = p @ v
    return out
