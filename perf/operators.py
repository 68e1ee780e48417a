"""The operators around one serving step over the paged KV cache, as cases to time.

One step of a serving loop with a sliding window runs, in this order:

  tables   block tables, slot map, positions and cumulative lengths of the step
           from the request lengths and a free list, all on the GPU
  rope     per-head RMS norm of q and k (optional), rotary positions, and (on
           the append path) k and v written into the paged cache by slot
  decode   attention of one new token per sequence over a window and the first
           tokens of its paged context
  prefill  the same for chunks of query rows
  release  blocks that fell out of the window, or whose request finished, go
           back to the free list

`own` false: each in elementary torch operations.  `own` true: the calls of
this package.  Attention inputs are N(0, 1) as in the step configurations;
contexts are log-uniform or uniform, and block ids come from a shuffled list.
"""
import math

import torch

own = False

BS = 16   # tokens per block
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token for each of the 256 running sequences: the step every decode iteration starts with
        {"name": "tables-decode-256", "op": "tables", "seqs": 256, "prefill": 0, "chunk": 0, "max_blocks": 512, "lo": 32,
         "hi": 8000, "pad": 0},
        # a very large mixed step: prefill chunks of 120 requests beside 3,900 decodes, in arrays of a fixed capacity
        {"name": "tables-mixed-4020", "op": "tables", "seqs": 4020, "prefill": 120, "chunk": 1024, "max_blocks": 512,
         "lo": 16, "hi": 7000, "pad": 1000},
        # a decode batch after a step: a few requests finished, the others slid by a token or a chunk
        {"name": "release-256", "op": "release", "seqs": 256, "max_blocks": 512, "lo": 32, "hi": 8192, "window": 1024,
         "sinks": 4, "finished": 0.05},
        # a large pool after a burst: thousands of long requests, a third of them finished
        {"name": "release-4000", "op": "release", "seqs": 4000, "max_blocks": 2048, "lo": 100, "hi": 32768, "window": 4096,
         "sinks": 64, "finished": 0.33},
        # decode step of the 1B shape (64 sequences, head_dim 64): q and k rotated, k and v appended
        {"name": "rope-append-decode-64", "op": "rope", "tokens": 64, "hq": 32, "hkv": 8, "d": 64, "rot": 64, "dtype": "bf16",
         "interleaved": False, "norm": False, "append": True, "scaling": "bands", "far": 2048},
        # mixed step of the 8B shape: 8 chunks of 512 and 248 decodes, heads normed, one padding row in 50
        {"name": "norm-rope-append-4344", "op": "rope", "tokens": 4344, "hq": 32, "hkv": 8, "d": 128, "rot": 128,
         "dtype": "bf16", "interleaved": False, "norm": True, "append": True, "scaling": "plain", "far": 8192},
        # a long prompt's rows at positions up to half a million, interleaved pairs over half of each head, not appended
        {"name": "rope-partial-16383", "op": "rope", "tokens": 16383, "hq": 16, "hkv": 16, "d": 128, "rot": 64,
         "dtype": "fp16", "interleaved": True, "norm": False, "append": False, "scaling": "yarn", "far": 524288},
        # a few interactive sequences, small window: latency
        {"name": "decode-4x512", "op": "decode", "seqs": 4, "hq": 8, "hkv": 2, "d": 64, "dtype": "fp16", "window": 512,
         "sinks": 4, "lo": 300, "hi": 2048},
        # the 8B-shaped decode batch with a window of 1,024
        {"name": "decode-256x1024", "op": "decode", "seqs": 256, "hq": 32, "hkv": 8, "d": 128, "dtype": "bf16",
         "window": 1024, "sinks": 4, "lo": 32, "hi": 8192},
        # a few very long sequences: almost all of the context lies outside the window and is released
        {"name": "decode-7x8000-long", "op": "decode", "seqs": 7, "hq": 32, "hkv": 8, "d": 128, "dtype": "bf16",
         "window": 8000, "sinks": 64, "lo": 60000, "hi": 131072},
        # the prefill part of the mixed step: 8 chunks of 512 behind 0 to 4,096 tokens
        {"name": "prefill-8x512", "op": "prefill", "chunks": 8, "qlo": 512, "qhi": 512, "plo": 0, "phi": 4096, "hq": 32,
         "hkv": 8, "d": 128, "dtype": "bf16", "window": 1024, "sinks": 4},
        # long prompts, ragged chunk lengths, a wide window behind a long context
        {"name": "prefill-3x4000-long", "op": "prefill", "chunks": 3, "qlo": 3500, "qhi": 4100, "plo": 8000, "phi": 28000,
         "hq": 32, "hkv": 8, "d": 128, "dtype": "bf16", "window": 4096, "sinks": 64},
    ]


HEADS = [(32, 8), (8, 2), (16, 16), (8, 1), (32, 2), (4, 4), (20, 4), (6, 2)]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw(rng):
    op = rng.choice(["tables", "release", "rope", "rope", "decode", "decode", "prefill"])
    if op == "tables":
        seqs = _log(rng, 1, 4096)
        prefill = rng.choice([0, rng.randint(0, min(seqs, 100))])
        return {"op": op, "seqs": seqs, "prefill": prefill, "chunk": _log(rng, 2, 1024), "max_blocks": 512, "lo": 1,
                "hi": 7000, "pad": rng.choice([0, rng.randint(1, 1000)])}
    if op == "release":
        mb = rng.choice([128, 333, 512, 2048])
        return {"op": op, "seqs": _log(rng, 1, 4000), "max_blocks": mb, "lo": 1, "hi": mb * BS,
                "window": rng.choice([0, _log(rng, 1, 8192)]), "sinks": rng.choice([0, 4, rng.randint(1, 100)]),
                "finished": round(rng.uniform(0, 0.6), 3)}
    hq, hkv = rng.choice(HEADS)
    d = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "rope":
        return {"op": op, "tokens": _log(rng, 1, 16384), "hq": hq, "hkv": hkv, "d": d,
                "rot": rng.choice([d, d, d // 2, d // 4]), "dtype": dtype, "interleaved": rng.random() < 0.5,
                "norm": rng.random() < 0.5, "append": rng.random() < 0.6,
                "scaling": rng.choice(["plain", "linear", "ntk", "bands", "yarn"]), "far": _log(rng, 2048, 1 << 20)}
    window, sinks = _log(rng, 16, 8192), rng.choice([0, 4, rng.randint(1, 130)])
    if op == "decode":
        hi = _log(rng, 64, 131072)
        return {"op": op, "seqs": _log(rng, 1, 256), "hq": hq, "hkv": hkv, "d": d, "dtype": dtype, "window": window,
                "sinks": sinks, "lo": max(1, hi // 40), "hi": hi}
    q, prior = _log(rng, 16, 4096), rng.choice([0, _log(rng, 16, 28000)])
    return {"op": op, "chunks": rng.randint(1, 8), "qlo": max(1, q // 2), "qhi": q, "plo": prior // 3, "phi": prior,
            "hq": hq, "hkv": hkv, "d": d, "dtype": dtype, "window": window, "sinks": sinks}


def _weight(c):
    """A bound on a case's work that needs no random lengths (draw keeps to the largest listed case's)."""
    if c["op"] == "decode":
        return c["seqs"] * min(c["hi"], c["window"] + c["sinks"]) * c["hkv"] * c["d"]
    if c["op"] == "prefill":
        return c["chunks"] * c["qhi"] * min(c["phi"] + c["qhi"], c["window"] + c["sinks"]) * c["hq"] * c["d"]
    if c["op"] == "rope":
        return c["tokens"] * (c["hq"] + 2 * c["hkv"]) * c["d"]
    if c["op"] == "release":
        return c["seqs"] * c["max_blocks"]
    return c["seqs"] + c["prefill"] * c["chunk"] + c["pad"]


def draw(rng):
    most = {}
    for c in listed():
        most[c["op"]] = max(most.get(c["op"], 0), _weight(c))
    while True:
        c = _draw(rng)
        if _weight(c) <= most[c["op"]]:
            return c


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _lengths(g, n, lo, hi):
    """n whole numbers in [lo, hi], spread over their logarithm; on the host."""
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64).cpu()
    x = torch.exp(math.log(max(lo, 1)) + u * (math.log(max(hi, 1)) - math.log(max(lo, 1))))
    return x.round().long().clamp(lo, hi)


def _blocks(n):
    return (n + BS - 1) // BS


def _tables(g, lens, max_blocks, first=None):
    """(tables, ids used): a row of shuffled block ids for each length, -1 behind them.  With `first` (a pair of
    whole-number tensors: blocks kept at the front, first block kept again), the blocks between are released: -1."""
    nb = _blocks(lens)
    j = torch.arange(max_blocks).unsqueeze(0)
    held = j < nb.unsqueeze(1)
    if first is not None:
        held &= (j < first[0].unsqueeze(1)) | (j >= first[1].unsqueeze(1))
    held = held.cuda()
    used = int(held.sum())
    tables = torch.full((len(lens), max_blocks), -1, dtype=torch.int32, device="cuda")
    tables[held] = torch.randperm(used, generator=g, device="cuda").int()
    return tables, used


def _capacity(c):
    """Rows that the step's per-token arrays have room for (a captured step's arrays have a fixed size)."""
    return c["seqs"] - c["prefill"] + c["prefill"] * max(2, c["chunk"]) + c["pad"]


def _randn(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _scaling(c):
    """(base, factor, original context, low, high) of the case's scaling."""
    return {"plain": (10000.0, 1.0, 0, 0.0, 0.0), "linear": (10000.0, 4.0, 0, 0.0, 0.0),
            "ntk": (10000.0, 8.0, 0, 0.0, 0.0), "bands": (500000.0, 8.0, 8192, 1.0, 4.0),
            "yarn": (10000.0, 16.0, 4096, 1.0, 32.0)}[c["scaling"]]


def prepare(case, seed):
    g = _gen(seed)
    st = {"case": dict(case)}
    op = case["op"]
    if op == "tables":
        S, P = case["seqs"], case["prefill"]
        lens = _lengths(g, S, case["lo"], case["hi"])
        new = torch.ones(S, dtype=torch.int64)
        if P:
            new[:P] = _lengths(g, P, 2, max(2, case["chunk"]))
            lens[:P] = torch.where(torch.rand(P, generator=g, device="cuda").cpu() < 0.5, torch.zeros(P, dtype=torch.int64),
                                   lens[:P] // 4)   # half of the chunks start a request
        tables, used = _tables(g, lens, case["max_blocks"])
        need = int((_blocks(lens + new) - _blocks(lens)).sum())
        spare = need + 1000
        free = (used + torch.randperm(spare, generator=g, device="cuda")).int()
        T = _capacity(case)
        i32 = lambda *shape: torch.empty(shape, dtype=torch.int32, device="cuda")   # noqa: E731
        st.update(seq_lens=lens.int().cuda(), new_lens=new.int().cuda(), tables=tables, free=free,
                  count=torch.full((1,), spare, dtype=torch.int32, device="cuda"), num_blocks=used + spare,
                  count_out=i32(1), ctx=i32(S), cu=i32(S + 1), pos=i32(T),
                  slots=torch.empty(T, dtype=torch.int64, device="cuda"),
                  status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    elif op == "release":
        S = case["seqs"]
        lens = _lengths(g, S, case["lo"], case["hi"])
        fin = (torch.rand(S, generator=g, device="cuda") < case["finished"]).int()
        sb, dead = torch.zeros(S, dtype=torch.int64), torch.zeros(S, dtype=torch.int64)
        if case["window"]:
            # what had left the window a chunk of tokens ago was released then
            sb += _blocks(torch.tensor(case["sinks"]))
            dead = ((lens - 512 - case["window"] + 1).clamp(min=0) // BS).clamp(min=0)
        tables, used = _tables(g, lens, case["max_blocks"], (sb, torch.maximum(sb, dead)))
        spare = 4096
        free0 = torch.full((S * case["max_blocks"] + spare,), -1, dtype=torch.int32, device="cuda")
        free0[:spare] = (used + torch.randperm(spare, generator=g, device="cuda")).int()
        st.update(seq_lens=lens.int().cuda(), finished=fin, tables0=tables, free0=free0, num_blocks=used + spare,
                  count0=torch.full((1,), spare, dtype=torch.int32, device="cuda"), tables=tables.clone(),
                  free=free0.clone(), count=torch.empty(1, dtype=torch.int32, device="cuda"),
                  status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    elif op == "rope":
        T, hq, hkv, d, dt = case["tokens"], case["hq"], case["hkv"], case["d"], DT[case["dtype"]]
        # q, k and v are slices of one fused projection's rows, which end in 128 columns of a gate
        qkv = _randn(g, (T, (hq + 2 * hkv) * d + 128), dt)
        q, k, v, _ = qkv.split([hq * d, hkv * d, hkv * d, 128], dim=1)
        st.update(q=q.view(T, hq, d), k=k.view(T, hkv, d), v=v.view(T, hkv, d),
                  pos=torch.randint(0, case["far"], (T,), generator=g, device="cuda", dtype=torch.int32),
                  q_out=torch.empty((T, hq, d), dtype=dt, device="cuda"), wq=None, wk=None,
                  status=torch.zeros(1, dtype=torch.int32, device="cuda"))
        if case["norm"]:
            st.update(wq=(1 + 0.1 * _randn(g, (d,), torch.float32)).to(dt),
                      wk=(1 + 0.1 * _randn(g, (d,), torch.float32)).to(dt))
        if case["append"]:
            nb = _blocks(T) + 3
            st["slots"] = torch.randperm(nb * BS, generator=g, device="cuda")[:T].contiguous()
            st["slots"][torch.rand(T, generator=g, device="cuda") < 0.02] = -1   # padding rows
            st["k_cache"] = torch.zeros((nb, hkv, BS, d), dtype=dt, device="cuda")
            st["v_cache"] = torch.zeros((nb, hkv, BS, d), dtype=dt, device="cuda")
        else:
            st["k_out"] = torch.empty((T, hkv, d), dtype=dt, device="cuda")
        base, factor, original, low, high = _scaling(case)
        if own:
            import paged_kv_cache_tables_gb300 as pkv
            kind = {"plain": pkv.ROPE_PLAIN, "linear": pkv.ROPE_LINEAR, "ntk": pkv.ROPE_NTK, "bands": pkv.ROPE_BANDS,
                    "yarn": pkv.ROPE_YARN}[case["scaling"]]
            st["freqs"], st["mscale"] = pkv.rope_frequencies(case["rot"], base=base, scaling=kind, factor=factor,
                                                             original_context=original, low=low, high=high)
        else:
            # angles are taken in 64 bits: a far position times a frequency loses whole turns in 32
            st["inv"], st["mscale"] = _inverse_frequencies(case["rot"], case["scaling"], base, factor, original, low, high)
    else:
        hq, hkv, d, dt = case["hq"], case["hkv"], case["d"], DT[case["dtype"]]
        W, sinks = case["window"], case["sinks"]
        if op == "decode":
            ctx = _lengths(g, case["seqs"], case["lo"], case["hi"])
            qn = torch.ones(case["seqs"], dtype=torch.int64)
        else:
            n = case["chunks"]
            qn = case["qlo"] + (13 + 7919 * torch.arange(n)) % (case["qhi"] - case["qlo"] + 1)
            ctx = qn + torch.randint(case["plo"], case["phi"] + 1, (n,), generator=g, device="cuda").cpu()
        # blocks that no row of this step can see have been released
        sb = torch.full_like(ctx, -(-sinks // BS))
        dead = (ctx - qn - W + 1).clamp(min=0) // BS
        tables, used = _tables(g, ctx, int(_blocks(ctx).max()), (sb, torch.maximum(sb, dead)))
        T = int(qn.sum())
        cu = torch.zeros(len(qn) + 1, dtype=torch.int64)
        cu[1:] = torch.cumsum(qn, 0)
        st.update(q=_randn(g, (T, hq, d), dt), k_cache=_randn(g, (used, hkv, BS, d), dt),
                  v_cache=_randn(g, (used, hkv, BS, d), dt), tables=tables, ctx=ctx.int().cuda(), cu=cu.int().cuda(),
                  out=torch.empty((T, hq, d), dtype=dt, device="cuda"), ctx_host=ctx.tolist(), qn_host=qn.tolist(),
                  max_q=int(qn.max()), status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    c = st["case"]
    if own:
        return _run_own(st, c)
    return {"tables": _plain_tables, "release": _plain_release, "rope": _plain_rope, "decode": _plain_decode,
            "prefill": _plain_prefill}[c["op"]](st, c)


def _run_own(st, c):
    import paged_kv_cache_tables_gb300 as pkv
    op = c["op"]
    if op == "tables":
        pkv.step_tables(st["seq_lens"], st["new_lens"], st["tables"], st["free"], st["count"], st["num_blocks"], st["ctx"],
                        st["cu"], st["slots"], st["pos"], free_count_out=st["count_out"], dev_status=st["status"])
        return {k: st[k] for k in ("tables", "count_out", "ctx", "cu", "slots", "pos")}
    if op == "release":
        # the pool as it was before the call (a pass can be made again)
        st["tables"].copy_(st["tables0"])
        st["count"].copy_(st["count0"])
        pkv.release_blocks(st["tables"], st["seq_lens"], st["free"], st["count"], st["num_blocks"], finished=st["finished"],
                           window=c["window"], num_sinks=c["sinks"], dev_status=st["status"])
        return {k: st[k] for k in ("tables", "free", "count")}
    if op == "rope" and c["append"]:
        pkv.qk_rope_append(st["q_out"], st["q"], st["k"], st["v"], st["pos"], st["slots"], st["freqs"], st["k_cache"],
                           st["v_cache"], interleaved=c["interleaved"], mscale=st["mscale"], q_weight=st["wq"],
                           k_weight=st["wk"], eps=1e-6, dev_status=st["status"])
        return {k: st[k] for k in ("q_out", "k_cache", "v_cache")}
    if op == "rope":
        pkv.qk_rope(st["q_out"], st["k_out"], st["q"], st["k"], st["pos"], st["freqs"], interleaved=c["interleaved"],
                    mscale=st["mscale"], q_weight=st["wq"], k_weight=st["wk"], eps=1e-6)
        return {k: st[k] for k in ("q_out", "k_out")}
    if op == "decode":
        pkv.paged_window_decode_attention(st["out"], st["q"], st["k_cache"], st["v_cache"], st["tables"], st["ctx"],
                                          c["window"], num_sinks=c["sinks"], dev_status=st["status"])
        return st["out"]
    pkv.paged_window_prefill_attention(st["out"], st["q"], st["cu"], st["max_q"], st["k_cache"], st["v_cache"],
                                       st["tables"], st["ctx"], c["window"], num_sinks=c["sinks"], dev_status=st["status"])
    return st["out"]


def _plain_tables(st, c):
    lens, new, tables = st["seq_lens"].long(), st["new_lens"].long(), st["tables"]
    S, T = lens.numel(), st["slots"].numel()
    ctx = lens + new
    old = (lens + BS - 1) // BS
    need = (ctx + BS - 1) // BS - old
    ends = torch.cumsum(need, 0)
    count = st["count"].long()
    # the k-th block taken is the k-th from the end of the free list
    k = torch.arange(int(ends[-1]), device="cuda")
    row = torch.searchsorted(ends, k, right=True)
    col = old[row] + k - (ends - need)[row]
    tables[row, col] = st["free"][count - 1 - k]
    st["count_out"].copy_(count - ends[-1:])
    st["ctx"].copy_(ctx)
    cu = torch.cumsum(new, 0)
    st["cu"][0] = 0
    st["cu"][1:] = cu
    t = torch.arange(T, device="cuda")
    s = torch.searchsorted(cu, t, right=True)
    real = s < S
    s = s.clamp(max=S - 1)
    p = torch.where(real, lens[s] + t - (cu - new)[s], torch.zeros_like(t))
    st["slots"].copy_(torch.where(real, tables[s, p // BS].long() * BS + p % BS, torch.full_like(t, -1)))
    st["pos"].copy_(p)
    return {k: st[k] for k in ("tables", "count_out", "ctx", "cu", "slots", "pos")}


def _plain_release(st, c):
    tables = st["tables"].copy_(st["tables0"])
    st["count"].copy_(st["count0"])
    lens = st["seq_lens"].long()
    j = torch.arange(tables.shape[1], device="cuda")
    nb = (lens + BS - 1) // BS
    lo, hi = torch.zeros_like(lens), torch.zeros_like(lens)
    if c["window"]:
        # the next token sees positions from len - window + 1 on
        lo = torch.full_like(lens, -(-c["sinks"] // BS))
        hi = (lens - c["window"] + 1).clamp(min=0) // BS
    fin = st["finished"] != 0
    lo, hi = torch.where(fin, torch.zeros_like(lo), lo), torch.where(fin, nb, torch.minimum(hi, nb))
    out = (j >= lo[:, None]) & (j < hi[:, None]) & (tables >= 0)
    ids = tables[out]
    n = st["count"].long()
    st["free"][n + torch.arange(ids.numel(), device="cuda")] = ids
    st["count"].add_(ids.numel())
    tables.masked_fill_(out, -1)
    return {k: st[k] for k in ("tables", "free", "count")}


def _inverse_frequencies(r, kind, base, factor, original, low, high):
    """Radians per position of each rotated pair, in 64 bits, and what cos and sin are multiplied by."""
    if kind == "ntk":
        base = base * factor ** (r / (r - 2))
    i = torch.arange(r // 2, dtype=torch.float64, device="cuda")
    f = torch.exp(-math.log(base) * 2 * i / r)
    if kind == "linear":
        return f / factor, 1.0
    if kind == "bands":
        s = ((original * f / (2 * math.pi) - low) / (high - low)).clamp(0, 1)   # rotations over the original context
        return s * f + (1 - s) * f / factor, 1.0
    if kind == "yarn":
        at = lambda turns: r * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))   # noqa: E731
        first, last = max(math.floor(at(high)), 0), min(math.ceil(at(low)), r - 1)
        ramp = ((i - first) / max(last - first, 1e-3)).clamp(0, 1)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _plain_rope(st, c):
    r, m = c["rot"], st["mscale"]
    a = st["pos"].double()[:, None] * st["inv"]
    cos, sin = (m * torch.cos(a)).float()[:, None], (m * torch.sin(a)).float()[:, None]

    def turned(x, w):
        y = x.float()
        if w is not None:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w.float()
        z = y.clone()
        i, j = (slice(0, r, 2), slice(1, r, 2)) if c["interleaved"] else (slice(0, r // 2), slice(r // 2, r))
        z[..., i] = y[..., i] * cos - y[..., j] * sin
        z[..., j] = y[..., i] * sin + y[..., j] * cos
        return z.to(x.dtype)

    st["q_out"].copy_(turned(st["q"], st["wq"]))
    k = turned(st["k"], st["wk"])
    if not c["append"]:
        st["k_out"].copy_(k)
        return {n: st[n] for n in ("q_out", "k_out")}
    keep = st["slots"] >= 0
    slot = st["slots"][keep]
    st["k_cache"][slot // BS, :, slot % BS] = k[keep]
    st["v_cache"][slot // BS, :, slot % BS] = st["v"][keep]
    return {n: st[n] for n in ("q_out", "k_cache", "v_cache")}


def _gathered(cache, table, pos):
    """Rows of the positions through one sequence's table, [heads, positions, d], in 32 bits."""
    return cache[table[pos // BS].long(), :, pos % BS].float().transpose(0, 1)


def _plain_decode(st, c):
    hq, hkv, d, W, sinks = c["hq"], c["hkv"], c["d"], c["window"], c["sinks"]
    q, out = st["q"].float().view(-1, hkv, hq // hkv, d) / math.sqrt(d), st["out"]
    S = q.shape[0]
    ctx = st["ctx"].long()
    # the visible positions of each sequence, side by side: first tokens, then the window
    front = torch.minimum(torch.full_like(ctx, sinks), (ctx - W).clamp(min=0))
    n = min(max(st["ctx_host"]), W + sinks)
    i = torch.arange(n, device="cuda")
    start = (ctx - W).clamp(min=0)
    pos = torch.where(i < front[:, None], i, start[:, None] + i - front[:, None])
    pos = torch.where((start > sinks)[:, None], pos, i.expand(S, n))   # window and first tokens overlap: all of them
    seen = pos < ctx[:, None]
    pos = torch.where(seen, pos, torch.zeros_like(pos))
    step = max(1, (1 << 28) // (n * hkv * d))
    for s in range(0, S, step):
        e = min(S, s + step)
        at = st["tables"][s:e].gather(1, pos[s:e] // BS).long().clamp(min=0)
        off = pos[s:e] % BS
        k = st["k_cache"][at, :, off].float()                             # [s, n, heads, d]
        x = torch.matmul(q[s:e], k.permute(0, 2, 3, 1))                   # [s, heads, group, n]
        x = x.masked_fill(~seen[s:e, None, None], -math.inf)
        x = torch.exp(x - x.amax(-1, keepdim=True))
        v = st["v_cache"][at, :, off].float().permute(0, 2, 1, 3)
        o = torch.matmul(x, v) / x.sum(-1, keepdim=True)
        out[s:e] = o.reshape(e - s, hq, d).to(out.dtype)
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
            k = _gathered(st["k_cache"], st["tables"][s], t)
            v = _gathered(st["v_cache"], st["tables"][s], t)
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
    g = _gen(1) if torch.cuda.is_available() else None
    if op == "tables":
        S, T = c["seqs"], _capacity(c)
        taken = (c["seqs"] - c["prefill"] + c["prefill"] * c["chunk"] / 3) / BS
        return {"bytes": 4.0 * (2 * S + S + 2 * S + 1) + 8 * taken + 12 * T, "flops": 0.0}
    if op == "release":
        S, mean = c["seqs"], (c["hi"] - c["lo"]) / max(math.log(c["hi"] / max(c["lo"], 1)), 1e-9) / BS if c["hi"] > c["lo"] else c["hi"] / BS
        held = min(mean, (c["window"] + 512) / BS) if c["window"] else mean
        out = c["finished"] * held + (1 - c["finished"]) * (32 if c["window"] else 0)
        return {"bytes": S * (8 + 4 * held + 8 * out), "flops": 0.0}
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    if op == "rope":
        T, heads = c["tokens"], hq + (2 if c["append"] else 1) * hkv
        norm = 4 * (hq + hkv) * d if c["norm"] else 0
        return {"bytes": T * (2 * 2 * heads * d + 4 + (8 if c["append"] else 0)), "flops": T * (3.0 * (hq + hkv) * c["rot"] + norm)}
    # lengths of a typical seed
    W, sinks = c["window"], c["sinks"]
    if op == "decode":
        n = c["seqs"]
        ctx = _lengths(g, n, c["lo"], c["hi"]) if g else torch.full((n,), (c["lo"] + c["hi"]) // 2)
        seen = float(torch.minimum(ctx, torch.full_like(ctx, W + sinks)).sum())
        return {"bytes": 2 * 2 * hkv * d * seen + 2 * 2 * n * hq * d + 4 * seen / BS, "flops": 4.0 * hq * d * seen}
    qn, prior = (c["qlo"] + c["qhi"]) // 2, (c["plo"] + c["phi"]) // 2
    p = torch.arange(prior, prior + qn, dtype=torch.float64)
    seen = float(torch.minimum(p + 1, torch.full_like(p, W + sinks)).sum()) * c["chunks"]
    keys = min(prior + qn, W + sinks + qn) * c["chunks"]
    return {"bytes": 2 * 2 * hkv * d * keys + 2 * 2 * c["chunks"] * qn * hq * d, "flops": 4.0 * hq * d * seen}


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    op = case["op"]
    if op in ("tables", "release"):
        return None   # whole numbers
    st = prepare(case, seed)
    if op == "rope":
        return _exact_rope(st, case)
    return _exact_attention(st, case)


def _exact_rope(st, c):
    r, d = c["rot"], c["d"]
    base, factor, original, low, high = _scaling(c)
    inv, m = [], 1.0
    for i in range(r // 2):
        w = base ** (-2.0 * i / r)
        if c["scaling"] == "linear":
            w /= factor
        elif c["scaling"] == "ntk":
            w = (base * factor ** (r / (r - 2.0))) ** (-2.0 * i / r)
        elif c["scaling"] == "bands":
            length = 2 * math.pi / w
            if length > original / low:
                w /= factor
            elif length >= original / high:
                s = (original / length - low) / (high - low)
                w = (1 - s) * w / factor + s * w
        elif c["scaling"] == "yarn":
            lo = max(math.floor(r * math.log(original / (high * 2 * math.pi)) / (2 * math.log(base))), 0)
            hi = min(math.ceil(r * math.log(original / (low * 2 * math.pi)) / (2 * math.log(base))), r - 1)
            t = min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
            w = w * (1 - t) + w / factor * t
            m = 0.1 * math.log(factor) + 1.0
        inv.append(w)
    a = st["pos"].double().unsqueeze(1) * torch.tensor(inv, dtype=torch.float64, device="cuda").unsqueeze(0)
    turn = m * torch.polar(torch.ones_like(a), a).unsqueeze(1)

    def turned(x, w):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / d + 1e-6) * w.double()
        if c["interleaved"]:
            z = torch.complex(x[..., 0:r:2].contiguous(), x[..., 1:r:2].contiguous()) * turn
            front = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(x[..., :r // 2].contiguous(), x[..., r // 2:r].contiguous()) * turn
            front = torch.cat([z.real, z.imag], -1)
        return torch.cat([front, x[..., r:]], -1)

    q, k = turned(st["q"], st["wq"]), turned(st["k"], st["wk"])
    if not c["append"]:
        return {"q_out": q, "k_out": k}
    kc = torch.zeros(st["k_cache"].shape, dtype=torch.float64, device="cuda")
    vc = torch.zeros_like(kc)
    rows = torch.nonzero(st["slots"] >= 0).flatten()
    b, o = torch.div(st["slots"][rows], BS, rounding_mode="floor"), st["slots"][rows] % BS
    kc[b, :, o] = k[rows]
    vc[b, :, o] = st["v"][rows].double()
    return {"q_out": q, "k_cache": kc, "v_cache": vc}


def _exact_attention(st, c):
    """Row by row of the definition, in slices that bound the memory: for each slice, all positions that any of its
    rows sees, with the rule written as a weight of zero."""
    hq, hkv, d, W, sinks = c["hq"], c["hkv"], c["d"], c["window"], c["sinks"]
    G = hq // hkv
    out = torch.zeros((st["q"].shape[0], hq, d), dtype=torch.float64, device="cuda")
    q0 = 0
    for s in range(len(st["ctx_host"])):
        ctx, qn = st["ctx_host"][s], st["qn_host"][s]
        for a in range(0, qn, 256):
            b = min(qn, a + 256)
            lowest, highest = ctx - qn + a, ctx - qn + b - 1
            pos = [t for t in range(min(sinks, highest + 1))] + list(range(max(sinks, lowest - W + 1), highest + 1))
            t = torch.tensor(pos, device="cuda")
            row = st["tables"][s].long()[t // BS] * BS + t % BS
            p = torch.arange(lowest, highest + 1, device="cuda").unsqueeze(1)
            hidden = ((t > p) | ((t >= sinks) & (p - t >= W))).unsqueeze(1)
            for h in range(hkv):
                k = st["k_cache"][torch.div(row, BS, rounding_mode="floor"), h, row % BS].double()
                v = st["v_cache"][torch.div(row, BS, rounding_mode="floor"), h, row % BS].double()
                q = st["q"][q0 + a:q0 + b, h * G:(h + 1) * G].double()
                x = torch.einsum("rgd,td->rgt", q, k) * d ** -0.5
                x = torch.softmax(x.masked_fill(hidden, float("-inf")), -1)
                out[q0 + a:q0 + b, h * G:(h + 1) * G] = torch.einsum("rgt,td->rgd", x, v)
        q0 += qn
    return out
