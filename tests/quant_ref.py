"""Plain 64-bit references for the cache held in 8 bits, written from the
definitions, and the error bounds that its attention kernels are held to.

e4m3 codes are handled as a table of their 256 values: the code next to x is
found among the table's midpoints, so no conversion of torch's is relied on.

Bounds.  A row is read back as code times scale, rounded once to the output's
type: half a step.  Attention: as in window_ref for scores, exp2 and the fp32
sums; the softmax weights, times the block's scale and at least 2^6 where the
largest of a row stands, meet the codes as fp16 values: with a bf16 output
rounded once, half a step of fp16 (2^-11 relative), or of its subnormals (2^-25,
against weights of which one is at least 2^6: 2^-31 times the largest |v| the
scales can hold, for each position); else value and residual, which is inside
window_ref's 2^-16 and the subnormals' half step again.  log2 of a V scale off by
half a step of fp32 at up to 2^7 (2^-18, in the exponent, so 2^-18 of the weight
in the products but not in the sum), the scale's reciprocal by 2^-23.
"""
import math

import torch

import window_ref as ref

BF16, F16, F32, CODE = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn
CODE_MAX = 448.0


def _value(b):
    e, m = (b >> 3) & 15, b & 7
    x = math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
    return -x if b & 128 else x


# values of codes 0..126 rise; 127 is NaN, 128..255 the negatives
VALUES = torch.tensor([float("nan") if b & 127 == 127 else _value(b) for b in range(256)], dtype=torch.float64)
_MID = (VALUES[:126] + VALUES[1:127]) / 2


def decode(codes):
    """Values of uint8 codes."""
    return VALUES[codes.long()]


def encode(x):
    """Codes next to x (64 bits), ties to the even code; infinities the code of 448."""
    a = x.abs()
    up = torch.searchsorted(_MID, a.nan_to_num(0.0), right=True)      # midpoints at or below a
    tie = (up > 0) & (_MID[(up - 1).clamp(min=0)] == a)
    code = torch.where(tie & (up % 2 == 1), up - 1, up)
    code = torch.where(x.isnan(), torch.full_like(code, 127), code)
    return torch.where(torch.signbit(x), code + 128, code).to(torch.uint8)


def scale_of(a):
    """The least power of two s >= 2^-60 with a <= 448 s."""
    e = -60
    while a > math.ldexp(CODE_MAX, e):
        e += 1
    return math.ldexp(1.0, e)


def append(rows, slots, cache, scales, kv):
    """pkv_kv_append_e4m3 of one of K (kv 0) and V: rows [T, Hkv, d] in 64 bits,
    cache uint8 [NB, Hkv, 16, d] and scales float64 [NB, Hkv, 2], on the CPU, in place."""
    todo = {}
    for t, slot in enumerate(slots):
        if 0 <= slot < cache.shape[0] * 16:
            todo.setdefault(slot // 16, []).append(t)
    for b, ts in todo.items():
        offs = [slots[t] % 16 for t in ts]
        for h in range(cache.shape[1]):
            x = rows[ts, h]
            need = scale_of(x[x.isfinite()].abs().max().item() if x.isfinite().any() else 0.0)
            old = 0.0 if 0 in offs else scales[b, h, kv].item()
            old = old if old > 0 else 0.0
            new = max(old, need)
            if 0 not in offs and new > old:
                keep = [o for o in range(16) if o not in offs]
                cache[b, h, keep] = encode(decode(cache[b, h, keep]) * (old / new))
            for o, row in zip(offs, x):
                cache[b, h, o] = encode(row / new)
            scales[b, h, kv] = new


def pool(g, NB, Hkv, d, spread=0.5, odd_scales=False):
    """(codes uint8 [NB, Hkv, 16, d], scales float32 [NB, Hkv]) of N(0, 1) values whose magnitude varies by token; odd
    scales are no powers of two."""
    x = torch.randn(NB, Hkv, 16, d, generator=g, dtype=torch.float64)
    x *= torch.exp(spread * torch.randn(NB, Hkv, 16, 1, generator=g, dtype=torch.float64))
    top = x.abs().amax((2, 3)).clamp(min=1e-30)
    s = torch.exp2(torch.ceil(torch.log2(top / CODE_MAX)))
    if odd_scales:
        s = (s * (0.7 + torch.rand(s.shape, generator=g, dtype=torch.float64))).float().double()
    return encode(x / s[..., None, None]), s.float()


def gathered(codes, scales, table, n):
    """The first n positions of a sequence, [n, Hkv, d] in 64 bits."""
    t = torch.arange(n)
    blk = table.long()[t // 16]
    ok = (blk >= 0) & (blk < codes.shape[0])
    b = blk.clamp(0, codes.shape[0] - 1)
    rows = decode(codes[b, :, t % 16]) * scales.double()[b].unsqueeze(-1)
    return torch.where(ok.view(n, 1, 1), rows, torch.zeros((), dtype=torch.float64))


def attention_bound(out, spread, mass, d, scale, out_dtype, largest_v, n):
    """largest_v: the largest |v| that the scales of the visible blocks can hold (448 s); n: positions."""
    ds = d * 2.0 ** -23 * mass * scale
    err = (2 * ds + 2.0 ** -16 + 2.0 ** -18 + 2.0 ** -22 + 2.0 ** -14) * spread + 2.0 ** -31 * largest_v * n
    if out_dtype == BF16:
        err = err + 2.0 ** -11 * spread
    return err + ref.rounding(out, err, out_dtype)


def assert_stored(got, want, bound, what=""):
    """assert_within for outputs that may pass fp16's range: what is at or past 65,520 is stored as infinity.  With got's
    infinities as +-65,520 and want cut off there, the bound holds as before: cutting off two numbers at one place brings
    them no further apart."""
    if got.dtype == F16:
        got = got.double().clamp(-65520.0, 65520.0)
        want = want.clamp(-65520.0, 65520.0)
    ref.assert_within(got, want, bound, what)


class Step:
    """Sequences of the given contexts and new rows over a cache in 8 bits, in shuffled blocks.  What no row may see
    holds NaN codes; blocks out of sight are not in the table (-1, or an id past the pool), and blocks in no table have
    NaN scales."""

    def __init__(self, ctx, qn, Hq, Hkv, d, dtype, window, sinks, seed=0, poison=True, heavy=False, spread=0.5,
                 odd_scales=False, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.ctx, self.qn, self.window, self.sinks, self.d = ctx, qn, window, sinks, d
        self.scale = 1 / math.sqrt(d)
        nb = [-(-c // 16) for c in ctx]
        self.max_blocks = max(nb + [1]) + 1
        ids = torch.randperm(sum(nb) + 2, generator=g)
        NB = len(ids)
        self.q = torch.randn(sum(qn), Hq, d, generator=g).to(dtype)
        if heavy:
            self.q *= 4
        self.kc, ks = pool(g, NB, Hkv, d, 0.0, odd_scales)
        self.vc, vs = pool(g, NB, Hkv, d, spread, odd_scales)
        self.scales = torch.stack([ks, vs], 2).contiguous()
        self.table = torch.full((len(ctx), self.max_blocks), -1, dtype=torch.int32)
        used, at = torch.zeros(NB, dtype=torch.bool), 0
        for s, (c, n) in enumerate(zip(ctx, qn)):
            self.table[s, :nb[s]] = ids[at:at + nb[s]].int()
            at += nb[s]
            t = torch.arange(nb[s] * 16)
            p = torch.arange(c - n, c).view(n, 1)
            vis = (ref.seen(p, t, window, sinks) & (t < c)).any(0) if n else torch.zeros(nb[s] * 16, dtype=torch.bool)
            blk = self.table[s].long()[t // 16]
            if poison:
                self.kc[blk[~vis], :, (t % 16)[~vis]] = 127
                self.vc[blk[~vis], :, (t % 16)[~vis]] = 255
            gone = ~vis.view(-1, 16).any(1)
            used[blk.view(-1, 16)[:, 0][~gone]] = True
            if poison:
                self.table[s, :nb[s]][gone] = NB + 7 if s % 2 else -1
        if poison:
            self.scales[~used] = float("nan")
        self.dev = {}
        if device == "cuda":
            self.k, self.v = self.kc.cuda().view(CODE), self.vc.cuda().view(CODE)
            self.dev = dict(q=self.q.cuda(), scales=self.scales.cuda(), table=self.table.cuda(),
                            ctx=torch.tensor(ctx, dtype=torch.int32).cuda(),
                            cu=torch.tensor([0] + torch.tensor(qn).cumsum(0).tolist(), dtype=torch.int32).cuda())
            self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def reference(self, out_dtype):
        out, bound, at = [], [], 0
        for s, (c, n) in enumerate(zip(self.ctx, self.qn)):
            q = self.q[at:at + n].double()
            at += n
            if c == 0 or n == 0:
                out.append(torch.zeros_like(q))
                bound.append(torch.zeros_like(q))
                continue
            k = gathered(self.kc, self.scales[..., 0], self.table[s], c)
            v = gathered(self.vc, self.scales[..., 1], self.table[s], c)
            o, sp, mass = ref.attend(q, c - n, k, v, self.window, self.sinks, self.scale)
            blk = self.table[s].long()[:-(-c // 16)]
            blk = blk[(blk >= 0) & (blk < len(self.scales))]
            largest = CODE_MAX * self.scales[blk, :, 1].double().nan_to_num(0.0).max().item() if len(blk) else 0.0
            out.append(o)
            bound.append(attention_bound(o, sp, mass, self.d, self.scale, out_dtype, largest, c))
        return torch.cat(out), torch.cat(bound)

    def decode(self, out_dtype, **kw):
        from paged_kv_cache_tables_gb300 import paged_decode_attention_e4m3
        out = torch.full(self.q.shape, float("nan"), dtype=out_dtype, device="cuda")
        paged_decode_attention_e4m3(out, self.dev["q"], self.k, self.v, self.dev["scales"], self.dev["table"],
                                    self.dev["ctx"], window=self.window, num_sinks=self.sinks, dev_status=self.status, **kw)
        return out

    def prefill(self, out_dtype, max_q=None, **kw):
        from paged_kv_cache_tables_gb300 import paged_prefill_attention_e4m3
        out = torch.full(self.q.shape, float("nan"), dtype=out_dtype, device="cuda")
        paged_prefill_attention_e4m3(out, self.dev["q"], self.dev["cu"], max_q or max(self.qn), self.k, self.v,
                                     self.dev["scales"], self.dev["table"], self.dev["ctx"], window=self.window,
                                     num_sinks=self.sinks, dev_status=self.status, **kw)
        return out
