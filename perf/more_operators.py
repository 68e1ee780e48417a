"""The paged KV cache held in 8 bits, as cases to time.

K and V lie as e4m3 codes in caches [blocks, heads, 16, d] with one fp32 scale
for each block and head (K's and V's side by side, [blocks, heads, 2]): a value
is its code times the scale.  A serving step over such a cache runs

  append   this step's K and V rows quantised into the cache by slot; a block's
           scale starts with the block and grows with its largest value, a
           power of two, and rows already there are rounded to the new one
  gather   rows of sequences read back as 16- or 32-bit values
  decode   attention of one new token per sequence over its context (all of
           it, or a window and the first tokens)
  prefill  the same for chunks of query rows

`own` false: each in elementary torch operations.  `own` true: the calls of
this package.  Keys and queries are N(0, 1), values N(0, 1) times a magnitude
of their token, so that scales differ from block to block.
"""
import math

import torch

own = False

BS = 16   # tokens per block
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
CODE = torch.float8_e4m3fn
CODE_MAX = 448.0
NO_WINDOW = 2 ** 31 - 1


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the decode step of the 8B shape: one row a sequence, at any offset of its last block
        {"name": "append-decode-256", "op": "append", "decodes": 256, "chunks": 0, "chunk": 0, "hkv": 8, "d": 128, "dtype": "bf16",
         "pad": 0},
        # the mixed step: 8 chunks of 512 rows and 248 decodes, some padding rows behind them
        {"name": "append-mixed-4344", "op": "append", "decodes": 248, "chunks": 8, "chunk": 512, "hkv": 8, "d": 128,
         "dtype": "bf16", "pad": 17},
        # a long prompt in ragged chunks, 16 heads of 64
        {"name": "append-prompt-16383", "op": "append", "decodes": 0, "chunks": 3, "chunk": 5461, "hkv": 16, "d": 64, "dtype": "fp16",
         "pad": 0},
        # a short prefix of one sequence read back: latency
        {"name": "gather-1x777", "op": "gather", "seqs": 1, "lo": 777, "hi": 777, "first": 0, "hkv": 8, "d": 128, "dtype": "bf16"},
        # contexts of 64 sequences handed over as dense rows
        {"name": "gather-64x8000", "op": "gather", "seqs": 64, "lo": 100, "hi": 8000, "first": 40, "hkv": 8, "d": 128,
         "dtype": "bf16"},
        # a few interactive sequences with small heads: latency
        {"name": "decode-4x2048", "op": "decode", "seqs": 4, "hq": 8, "hkv": 2, "d": 64, "dtype": "fp16", "window": NO_WINDOW,
         "sinks": 0, "lo": 300, "hi": 2048},
        # the decode step of the 1B shape
        {"name": "decode-64x4096-d64", "op": "decode", "seqs": 64, "hq": 32, "hkv": 8, "d": 64, "dtype": "bf16",
         "window": NO_WINDOW, "sinks": 0, "lo": 64, "hi": 4096},
        # the decode batch of the 8B shape, whole contexts
        {"name": "decode-256x8192", "op": "decode", "seqs": 256, "hq": 32, "hkv": 8, "d": 128, "dtype": "bf16",
         "window": NO_WINDOW, "sinks": 0, "lo": 32, "hi": 8192},
        # a few very long sequences
        {"name": "decode-7x131072-long", "op": "decode", "seqs": 7, "hq": 32, "hkv": 8, "d": 128, "dtype": "bf16",
         "window": NO_WINDOW, "sinks": 0, "lo": 60000, "hi": 131072},
        # the prefill part of the mixed step: 8 chunks of 512 behind 0 to 4,096 tokens
        {"name": "prefill-8x512", "op": "prefill", "chunks": 8, "qlo": 512, "qhi": 512, "plo": 0, "phi": 4096, "hq": 32,
         "hkv": 8, "d": 128, "dtype": "bf16", "window": NO_WINDOW, "sinks": 0},
        # whole prompts of ragged lengths, heads of 64
        {"name": "prefill-5x2000-d64", "op": "prefill", "chunks": 5, "qlo": 1200, "qhi": 2900, "plo": 0, "phi": 0, "hq": 16,
         "hkv": 4, "d": 64, "dtype": "fp16", "window": NO_WINDOW, "sinks": 0},
        # long prompts, ragged chunks, a wide window and first tokens behind a long context
        {"name": "prefill-3x4000-long", "op": "prefill", "chunks": 3, "qlo": 3500, "qhi": 4100, "plo": 8000, "phi": 28000,
         "hq": 32, "hkv": 8, "d": 128, "dtype": "bf16", "window": 4096, "sinks": 64},
    ]


HEADS = [(32, 8), (8, 2), (16, 16), (8, 1), (32, 2), (4, 4), (20, 4), (6, 2)]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw(rng):
    op = rng.choice(["append", "gather", "decode", "decode", "prefill", "prefill"])
    hq, hkv = rng.choice(HEADS)
    d, dtype = rng.choice([64, 128]), rng.choice(["bf16", "fp16"])
    if op == "append":
        return {"op": op, "decodes": rng.choice([0, _log(rng, 1, 2000)]), "chunks": rng.choice([0, rng.randint(1, 16)]),
                "chunk": _log(rng, 2, 8192), "hkv": hkv, "d": d, "dtype": dtype, "pad": rng.choice([0, rng.randint(1, 100)])}
    if op == "gather":
        hi = _log(rng, 16, 32768)
        return {"op": op, "seqs": _log(rng, 1, 256), "lo": max(1, hi // rng.choice([1, 20])), "hi": hi,
                "first": rng.choice([0, rng.randint(1, 200)]), "hkv": hkv, "d": d, "dtype": rng.choice(["bf16", "fp16", "fp32"])}
    window, sinks = rng.choice([(NO_WINDOW, 0), (_log(rng, 16, 8192), rng.choice([0, 4, rng.randint(1, 130)]))])
    if op == "decode":
        hi = _log(rng, 64, 131072)
        return {"op": op, "seqs": _log(rng, 1, 256), "hq": hq, "hkv": hkv, "d": d, "dtype": dtype, "window": window,
                "sinks": sinks, "lo": max(1, hi // 40), "hi": hi}
    q, prior = _log(rng, 16, 4096), rng.choice([0, _log(rng, 16, 28000)])
    return {"op": op, "chunks": rng.randint(1, 8), "qlo": max(1, q // 2), "qhi": q, "plo": prior // 3, "phi": prior,
            "hq": hq, "hkv": hkv, "d": d, "dtype": dtype, "window": window, "sinks": sinks}


def _weight(c):
    """A bound on a case's work that needs no random lengths (draw keeps to the largest listed case's)."""
    if c["op"] == "append":
        return (c["decodes"] + c["chunks"] * c["chunk"] + c["pad"]) * c["hkv"] * c["d"]
    if c["op"] == "gather":
        return c["seqs"] * c["hi"] * c["hkv"] * c["d"]
    if c["op"] == "decode":
        return c["seqs"] * c["hi"] * c["hkv"] * c["d"]
    return c["chunks"] * c["qhi"] * min(c["phi"] + c["qhi"], c["window"] + c["sinks"]) * c["hq"] * c["d"]


def draw(rng):
    most = {}
    for c in listed():
        most[c["op"]] = max(most.get(c["op"], 0), _weight(c))
    while True:
        c = _draw(rng)
        if 0 < _weight(c) <= most[c["op"]] and (c["op"] != "append" or c["decodes"] + c["chunks"] > 0):
            return c


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _lengths(g, n, lo, hi):
    """n whole numbers in [lo, hi], spread over their logarithm; on the host."""
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64).cpu()
    x = torch.exp(math.log(max(lo, 1)) + u * (math.log(max(hi, 1)) - math.log(max(lo, 1))))
    return x.round().long().clamp(lo, hi)


def _blocks(n):
    return (n + BS - 1) // BS


def _tables(g, lens, gone=None):
    """(tables, ids used): a row of shuffled block ids for each length, -1 behind them.  With `gone` (a pair: blocks
    kept at the front, first block kept again), the blocks between were given back: -1."""
    nb = _blocks(lens)
    j = torch.arange(int(nb.max())).unsqueeze(0)
    held = j < nb.unsqueeze(1)
    if gone is not None:
        held &= (j < gone[0].unsqueeze(1)) | (j >= gone[1].unsqueeze(1))
    held = held.cuda()
    used = int(held.sum())
    tables = torch.full(held.shape, -1, dtype=torch.int32, device="cuda")
    tables[held] = torch.randperm(used, generator=g, device="cuda").int()
    return tables, used


def _pow2(e):
    """2^e for whole e, by its bits: fp32."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _power_scale(a):
    """The least power of two s, at least 2^-60, with a <= 448 s; a finite, fp32."""
    m, e = torch.frexp(a)                                   # a = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(-60, 120)
    return _pow2(torch.where(a > 0, e, torch.full_like(e, -60)))


def _codes(x):
    return x.clamp(-CODE_MAX, CODE_MAX).to(CODE)


def _filled(g, used, hkv, d, spread):
    """A cache whose blocks are all written, and the scales [blocks, heads] of it; values N(0, 1), of magnitudes that
    spread over tokens.  Made in slices."""
    cache = torch.empty((used, hkv, BS, d), dtype=torch.uint8, device="cuda")
    scales = torch.empty((used, hkv), dtype=torch.float32, device="cuda")
    step = max(1, (1 << 27) // (hkv * BS * d))
    for a in range(0, used, step):
        n = min(used, a + step) - a
        x = _randn(g, (n, hkv, BS, d))
        if spread:
            x *= torch.exp(spread * _randn(g, (n, hkv, BS, 1)))
        s = _power_scale(x.abs().amax((2, 3)))
        cache[a:a + n] = _codes(x / s[:, :, None, None]).view(torch.uint8)
        scales[a:a + n] = s
    return cache.view(CODE), scales


def _pool(g, used, hkv, d):
    k, ks = _filled(g, used, hkv, d, 0.0)
    v, vs = _filled(g, used, hkv, d, 0.5)
    return {"k_cache": k, "v_cache": v, "kv_scales": torch.stack([ks, vs], 2).contiguous()}


def prepare(case, seed):
    g = _gen(seed)
    c, op = case, case["op"]
    hkv, d, dt = c["hkv"], c["d"], DT[c["dtype"]]
    st = {"case": dict(case), "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    if op == "append":
        # chunks first, then decodes, as the scheduler lays a step out; padding rows last
        n = torch.ones(c["chunks"] + c["decodes"], dtype=torch.int64)
        start = torch.randint(0, BS, n.shape, generator=g, device="cuda").cpu()
        if c["chunks"]:
            n[:c["chunks"]] = c["chunk"] - (7 + 13 * torch.arange(c["chunks"])) % max(1, c["chunk"] // 8)
            i = torch.arange(c["chunks"])   # two in three start a block
            start[:c["chunks"]] = torch.where(i % 3 == 2, 1 + 5 * i % (BS - 1), torch.zeros_like(i))
        tables, used = _tables(g, start + n)
        row = torch.repeat_interleave(torch.arange(len(n)), n)
        p = torch.arange(int(n.sum())) - (torch.cumsum(n, 0) - n)[row] + start[row]
        slots = tables.cpu()[row, p // BS].long() * BS + p % BS
        slots = torch.cat([slots, torch.full((c["pad"],), -1)]).cuda()
        T = slots.numel()
        # k and v are slices of one fused projection's rows; a chunk's tokens differ in magnitude
        kv = _randn(g, (T, 2 * hkv * d)) * torch.exp(0.3 * _randn(g, (T, 1)))
        k, v = kv.to(dt).split([hkv * d, hkv * d], dim=1)
        st.update(_pool(g, used, hkv, d), k=k.view(T, hkv, d), v=v.view(T, hkv, d), slots=slots)
        return st
    if op == "gather":
        n = _lengths(_gen(1), c["seqs"], c["lo"], c["hi"])   # as many rows for every seed
        first = torch.full_like(n, c["first"])
        tables, used = _tables(g, first + n)
        cu = torch.zeros(len(n) + 1, dtype=torch.int64)
        cu[1:] = torch.cumsum(n, 0)
        T = int(n.sum())
        st.update(_pool(g, used, hkv, d), tables=tables, cu=cu.int().cuda(), first=first.int().cuda() if c["first"] else None,
                  k=torch.empty((T, hkv, d), dtype=dt, device="cuda"), v=torch.empty((T, hkv, d), dtype=dt, device="cuda"),
                  n_host=n.tolist())
        return st
    hq, W, sinks = c["hq"], c["window"], c["sinks"]
    if op == "decode":
        ctx = _lengths(g, c["seqs"], c["lo"], c["hi"])
        qn = torch.ones(c["seqs"], dtype=torch.int64)
    else:
        n = c["chunks"]
        qn = c["qlo"] + (13 + 7919 * torch.arange(n)) % (c["qhi"] - c["qlo"] + 1)
        ctx = qn + torch.randint(c["plo"], c["phi"] + 1, (n,), generator=g, device="cuda").cpu()
    # blocks that no row of this step can see were given back
    front = torch.full_like(ctx, -(-sinks // BS))
    tables, used = _tables(g, ctx, (front, torch.maximum(front, (ctx - qn - W + 1).clamp(min=0) // BS)))
    cu = torch.zeros(len(qn) + 1, dtype=torch.int64)
    cu[1:] = torch.cumsum(qn, 0)
    T = int(qn.sum())
    st.update(_pool(g, used, hkv, d), q=_randn(g, (T, hq, d), dt), tables=tables, ctx=ctx.int().cuda(), cu=cu.int().cuda(),
              out=torch.empty((T, hq, d), dtype=dt, device="cuda"), ctx_host=ctx.tolist(), qn_host=qn.tolist(),
              max_q=int(qn.max()))
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    c = st["case"]
    if own:
        return _run_own(st, c)
    return {"append": _plain_append, "gather": _plain_gather, "decode": _plain_decode, "prefill": _plain_prefill}[c["op"]](st, c)


def _run_own(st, c):
    import paged_kv_cache_tables_gb300 as pkv
    op = c["op"]
    if op == "append":
        pkv.kv_append_e4m3(st["k"], st["v"], st["slots"], st["k_cache"], st["v_cache"], st["kv_scales"], dev_status=st["status"])
        return {n: st[n] for n in ("k_cache", "v_cache", "kv_scales")}
    if op == "gather":
        pkv.kv_gather_e4m3(st["k"], st["v"], st["k_cache"], st["v_cache"], st["kv_scales"], st["tables"], st["cu"],
                           first=st["first"], dev_status=st["status"])
        return {n: st[n] for n in ("k", "v")}
    if op == "decode":
        pkv.paged_decode_attention_e4m3(st["out"], st["q"], st["k_cache"], st["v_cache"], st["kv_scales"], st["tables"],
                                        st["ctx"], window=c["window"], num_sinks=c["sinks"], dev_status=st["status"])
        return st["out"]
    pkv.paged_prefill_attention_e4m3(st["out"], st["q"], st["cu"], st["max_q"], st["k_cache"], st["v_cache"], st["kv_scales"],
                                     st["tables"], st["ctx"], window=c["window"], num_sinks=c["sinks"], dev_status=st["status"])
    return st["out"]


def _plain_append(st, c):
    keep = st["slots"] >= 0
    slot = st["slots"][keep]
    blocks, at = torch.unique(slot // BS, return_inverse=True)      # the blocks written, and each row's among them
    off = slot % BS
    begun = torch.zeros(len(blocks), dtype=torch.bool, device="cuda")
    begun[at[off == 0]] = True
    for i, (name, rows) in enumerate((("k_cache", st["k"]), ("v_cache", st["v"]))):
        x = rows[keep].float()
        a = torch.where(x.isfinite(), x.abs(), torch.zeros_like(x)).amax(-1)
        most = torch.zeros((len(blocks), x.shape[1]), device="cuda").index_reduce_(0, at, a, "amax")
        was = torch.where(begun[:, None], torch.zeros_like(most), st["kv_scales"][blocks, :, i])
        now = torch.maximum(was, _power_scale(most))
        tiles = st[name].view(torch.uint8)[blocks]
        other = _codes(tiles.view(CODE).float() * (was / now)[:, :, None, None]).view(torch.uint8)
        tiles = torch.where((~begun[:, None] & (now > was))[:, :, None, None], other, tiles)
        tiles[at, :, off] = _codes(x / now[at][..., None]).view(torch.uint8)
        st[name].view(torch.uint8)[blocks] = tiles
        st["kv_scales"][blocks, :, i] = now
    return {n: st[n] for n in ("k_cache", "v_cache", "kv_scales")}


def _plain_gather(st, c):
    cu = st["cu"].long()
    t = torch.arange(st["k"].shape[0], device="cuda")
    s = torch.searchsorted(cu[1:], t, right=True)
    p = t - cu[s] + (st["first"].long()[s] if st["first"] is not None else 0)
    b = st["tables"][s, p // BS].long()
    for i, (name, cache) in enumerate((("k", "k_cache"), ("v", "v_cache"))):
        x = st[cache].view(torch.uint8)[b, :, p % BS].view(CODE).float()
        st[name].copy_(x * st["kv_scales"][b, :, i, None])
    return {n: st[n] for n in ("k", "v")}


def _values(st, i, blocks, off):
    """K (i = 0) or V (i = 1) rows at these blocks and offsets, [..., heads, d] in 32 bits."""
    x = st[("k_cache", "v_cache")[i]].view(torch.uint8)[blocks, :, off].view(CODE).float()
    return x * st["kv_scales"][blocks, :, i, None]


def _plain_decode(st, c):
    hq, hkv, d, W, sinks = c["hq"], c["hkv"], c["d"], c["window"], c["sinks"]
    q, out = st["q"].float().view(-1, hkv, hq // hkv, d) / math.sqrt(d), st["out"]
    ctx = st["ctx"].long()
    order = sorted(range(len(st["ctx_host"])), key=lambda s: st["ctx_host"][s])   # equal lengths side by side
    a = 0
    while a < len(order):
        n = min(st["ctx_host"][order[a]], W + sinks)
        b = a
        while b < len(order) and (b - a + 1) * min(st["ctx_host"][order[b]], W + sinks) * hkv * d <= 1 << 28:
            n, b = min(st["ctx_host"][order[b]], W + sinks), b + 1
        b = max(b, a + 1)
        s = torch.tensor(order[a:b], device="cuda")
        a = b
        # the visible positions of each sequence, side by side: first tokens, then the window
        start = (ctx[s] - W).clamp(min=0)[:, None]
        i = torch.arange(n, device="cuda")
        pos = torch.where(start > sinks, torch.where(i < sinks, i, start + i - sinks), i)
        seen = pos < ctx[s][:, None]
        pos = torch.where(seen, pos, torch.zeros_like(pos))
        at, off = st["tables"][s].gather(1, pos // BS).long(), pos % BS
        x = torch.matmul(q[s], _values(st, 0, at, off).permute(0, 2, 3, 1))   # [sequences, heads, group, n]
        x = x.masked_fill(~seen[:, None, None], -math.inf)
        x = torch.exp(x - x.amax(-1, keepdim=True))
        o = torch.matmul(x, _values(st, 1, at, off).permute(0, 2, 1, 3)) / x.sum(-1, keepdim=True)
        out[s] = o.reshape(len(s), hq, d).to(out.dtype)
    return out


def _plain_prefill(st, c):
    hq, hkv, d, W, sinks = c["hq"], c["hkv"], c["d"], c["window"], c["sinks"]
    G, out, q0 = hq // hkv, st["out"], 0
    rows = 512
    for s, (ctx, qn) in enumerate(zip(st["ctx_host"], st["qn_host"])):
        for a in range(0, qn, rows):
            b = min(qn, a + rows)
            p = ctx - qn + torch.arange(a, b, device="cuda")
            first = max(ctx - qn + a - W + 1, 0)
            t = torch.cat([torch.arange(0, min(sinks, first), device="cuda"),
                           torch.arange(first, ctx - qn + b, device="cuda")])
            at, off = st["tables"][s][t // BS].long(), t % BS
            k, v = _values(st, 0, at, off).transpose(0, 1), _values(st, 1, at, off).transpose(0, 1)
            seen = (t <= p[:, None]) & ((t < sinks) | (t > p[:, None] - W))
            q = st["q"][q0 + a:q0 + b].float().view(b - a, hkv, G, d).permute(1, 2, 0, 3) / math.sqrt(d)
            x = torch.matmul(q, k.transpose(1, 2).unsqueeze(1))           # [heads, group, rows, keys]
            x = x.masked_fill(~seen, -math.inf)
            x = torch.exp(x - x.amax(-1, keepdim=True))
            o = torch.matmul(x, v.unsqueeze(1)) / x.sum(-1, keepdim=True)
            out[q0 + a:q0 + b] = o.permute(2, 0, 1, 3).reshape(b - a, hq, d).to(out.dtype)
        q0 += qn
    return out


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c, op = case, case["op"]
    hkv, d = c["hkv"], c["d"]
    size = 4 if c["dtype"] == "fp32" else 2
    if op == "append":
        T = c["decodes"] + c["chunks"] * c["chunk"]
        blocks = c["decodes"] + c["chunks"] * c["chunk"] / BS
        return {"bytes": T * (2 * hkv * d * (size + 1) + 8) + blocks * hkv * 8, "flops": 4.0 * T * hkv * d}
    g = _gen(1) if torch.cuda.is_available() else None
    lengths = lambda n, lo, hi: _lengths(g, n, lo, hi) if g else torch.full((n,), (lo + hi) // 2)   # noqa: E731
    token = hkv * (2 * d + 8 / BS) + 4 / BS       # codes, scales and table entries of a position
    if op == "gather":
        T = float(lengths(c["seqs"], c["lo"], c["hi"]).sum())
        return {"bytes": T * (token + 2 * hkv * d * size), "flops": 2.0 * T * hkv * d}
    # lengths of a typical seed
    hq, W, sinks = c["hq"], c["window"], c["sinks"]
    if op == "decode":
        ctx = lengths(c["seqs"], c["lo"], c["hi"])
        seen = float(torch.minimum(ctx, torch.full_like(ctx, W + sinks)).sum())
        return {"bytes": token * seen + 2 * size * c["seqs"] * hq * d, "flops": 4.0 * hq * d * seen}
    qn, prior = (c["qlo"] + c["qhi"]) // 2, (c["plo"] + c["phi"]) // 2
    p = torch.arange(prior, prior + qn, dtype=torch.float64)
    seen = float(torch.minimum(p + 1, torch.full_like(p, W + sinks)).sum()) * c["chunks"]
    keys = min(prior + qn, W + sinks + qn) * c["chunks"]
    return {"bytes": token * keys + 2 * size * c["chunks"] * qn * hq * d, "flops": 4.0 * hq * d * seen}


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    return {"append": _exact_append, "gather": _exact_gather}.get(case["op"], _exact_attention)(st, case)


def _two_to(e):
    """2^e for whole e in 64 bits, by its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _rounded(x):
    """The e4m3 value next to x (64 bits): three bits behind the leading one, steps of 2^-9 below 2^-6, ties to even
    (torch.round's), no further than 448."""
    _, e = torch.frexp(x)
    step = _two_to((e - 1).clamp(min=-6) - 3)
    return (torch.round(x / step) * step).clamp(-CODE_MAX, CODE_MAX)


def _decoded(codes):
    """Bytes as e4m3 values, in 64 bits, by their fields."""
    b = codes.view(torch.uint8).long()
    e, m = (b >> 3) & 15, (b & 7).double()
    x = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * _two_to(e - 7))
    return torch.where(b >= 128, -x, x)


def _exact_append(st, c):
    """Block by block of the definition."""
    out, scales = {}, st["kv_scales"].double()
    slots = st["slots"].tolist()
    by_block = {}
    for t, slot in enumerate(slots):
        if slot >= 0:
            by_block.setdefault(slot // BS, []).append(t)
    for i, name in enumerate(("k_cache", "v_cache")):
        cache, rows = _decoded(st[name]), st[name[0]].double()
        # blocks of equally many rows together, for speed
        sizes = {}
        for b, ts in by_block.items():
            sizes.setdefault(len(ts), []).append(b)
        for n, blocks in sizes.items():
            b = torch.tensor(blocks, device="cuda")
            ts = torch.tensor([by_block[x] for x in blocks], device="cuda")               # [blocks, n]
            off = torch.tensor([[slots[t] % BS for t in by_block[x]] for x in blocks], device="cuda")
            x = rows[ts].transpose(1, 2)                                                   # [blocks, heads, n, d]
            top = x.abs().flatten(2).max(-1).values
            need = _two_to(torch.ceil(torch.log2(top.clamp(min=1e-300) / CODE_MAX)).clamp(min=-60))
            need = torch.where(top > need * CODE_MAX, need * 2, need)                      # log2's own rounding, either way
            need = torch.where((top <= need / 2 * CODE_MAX) & (need > 2.0 ** -60), need / 2, need)
            anew = (off == 0).any(1)[:, None]
            new = torch.where(anew | (need > scales[b, :, i]), need, scales[b, :, i])
            grown = ~anew & (new > scales[b, :, i])
            kept = torch.where(grown[..., None, None], _rounded(cache[b] * (scales[b, :, i] / new)[..., None, None]), cache[b])
            where = off[:, None, :, None].expand(x.shape)
            cache[b] = kept.scatter(2, where, _rounded(x / new[..., None, None]))
            scales[b, :, i] = new
        out[name] = cache
    out["kv_scales"] = scales
    return out


def _exact_gather(st, c):
    where = []
    for s, n in enumerate(st["n_host"]):
        t = c["first"] + torch.arange(n, device="cuda")
        where.append(st["tables"][s][torch.div(t, BS, rounding_mode="floor")].long() * BS + t % BS)
    where = torch.cat(where)
    b, o = torch.div(where, BS, rounding_mode="floor"), where % BS
    scales = st["kv_scales"].double()
    return {n: _decoded(st[n + "_cache"].view(torch.uint8).transpose(1, 2)[b, o]) * scales[b, :, i].unsqueeze(-1)
            for i, n in enumerate(("k", "v"))}


def _exact_attention(st, c):
    """Row by row of the definition, in slices that bound the memory: for each slice, all positions that any of its
    rows sees, with the rule written as a weight of zero."""
    hq, hkv, d, W, sinks = c["hq"], c["hkv"], c["d"], c["window"], c["sinks"]
    G = hq // hkv
    pairs = sum(n * min(x, W + sinks) for x, n in zip(st["ctx_host"], st["qn_host"]))
    if 4.0 * pairs * hq * d > 8e12:
        return None   # more than a few seconds of 64-bit products
    out = torch.zeros((st["q"].shape[0], hq, d), dtype=torch.float64, device="cuda")
    scales = st["kv_scales"].double()
    q0 = 0
    for s, (ctx, qn) in enumerate(zip(st["ctx_host"], st["qn_host"])):
        for a in range(0, qn, 256):
            b = min(qn, a + 256)
            lowest, highest = ctx - qn + a, ctx - qn + b - 1
            from_ = max(sinks, lowest - W + 1)
            t = torch.cat([torch.arange(min(sinks, highest + 1)), torch.arange(from_, max(from_, highest + 1))]).cuda()
            blk, o = st["tables"][s].long()[torch.div(t, BS, rounding_mode="floor")], t % BS
            p = torch.arange(lowest, highest + 1, device="cuda").unsqueeze(1)
            hidden = ((t > p) | ((t >= sinks) & (p - t >= W))).unsqueeze(1)
            for h in range(hkv):
                k = _decoded(st["k_cache"].view(torch.uint8)[blk, h, o]) * scales[blk, h, 0].unsqueeze(1)
                v = _decoded(st["v_cache"].view(torch.uint8)[blk, h, o]) * scales[blk, h, 1].unsqueeze(1)
                q = st["q"][q0 + a:q0 + b, h * G:(h + 1) * G].double()
                x = torch.einsum("rgd,td->rgt", q, k) * d ** -0.5
                x = torch.softmax(x.masked_fill(hidden, float("-inf")), -1)
                out[q0 + a:q0 + b, h * G:(h + 1) * G] = torch.einsum("rgt,td->rgd", x, v)
        q0 += qn
    return out
