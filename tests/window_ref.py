"""Plain 64-bit references for the sliding-window operators, written from their
definitions, and the error bounds that the kernels are held to.

Bounds.  A score q . k of head_dim d is accumulated in fp32: at most d
roundings of at most 2^-23 of sum |q_i k_i| each (the tensor cores truncate, a
full step).  With the scale that moves a score by ds, every softmax weight by a
factor within exp(+-2 ds) (numerator and denominator), so an output by at most
2 ds * sum p |v| (ds << 1).  On top, relative to sum p |v|: the weights' 16-bit
value plus residual (2 half steps of 2^-8: 2^-16 for bf16, less for fp16), exp2
(2^-22), and the fp32 sums over up to 2^14 keys in parts of 16 (2^10 roundings
of 2^-24 at most: 2^-14; an fp32 sum of n terms in a chain).  The output's own
rounding to 16 bits is half a step, eps / 2 relative, or half the smallest
subnormal.

Prefill with a 16-bit output rounds the weights to that type once (no residual):
2^x of scores relative to a maximum that the row's own has reached or passed, so
the largest weight, and with it the sum, is at least 1.  A weight w then moves by
at most eps / 2 w, or half the smallest subnormal, and the output by at most
eps / 2 sum p |v| + TINY / 2 sum |v| (the sum is taken of the unrounded weights).
"""
import numpy as np
import torch

EPS = {torch.float32: 2.0 ** -23, torch.float16: 2.0 ** -10, torch.bfloat16: 2.0 ** -7}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133}


def rounding(ref, err, dtype):
    """What storing a value within `err` of `ref` in dtype can add: half a step."""
    return EPS[dtype] / 2 * (ref.abs() + err) + TINY[dtype] / 2


def seen(p, t, window, sinks):
    """Whether position p sees position t (broadcast)."""
    return (t <= p) & ((t > p - window) | (t < sinks))


def attend(q, first, keys, values, window, sinks, scale):
    """q [R, Hq, d] at positions first..first+R-1; keys, values [n, Hkv, d],
    entry t at position t (entries no row sees may hold anything).  All in
    64 bits on the CPU.  Returns (out, sum p |v|, largest sum |q_i k_i| seen)."""
    R, Hq, d = q.shape
    n, Hkv = keys.shape[:2]
    G = Hq // Hkv
    p = torch.arange(first, first + R).view(R, 1)
    vis = seen(p, torch.arange(n).view(1, n), window, sinks)
    used = vis.any(0)
    k = torch.where(used.view(n, 1, 1), keys, torch.zeros((), dtype=torch.float64))
    v = torch.where(used.view(n, 1, 1), values, torch.zeros((), dtype=torch.float64))
    qg = q.view(R, Hkv, G, d)
    x = torch.einsum("rhgd,thd->rhgt", qg, k) * scale
    x = x.masked_fill(~vis.view(R, 1, 1, n), float("-inf"))
    mass = torch.einsum("rhgd,thd->rhgt", qg.abs(), k.abs())
    mass = torch.where(vis.view(R, 1, 1, n), mass, torch.zeros((), dtype=torch.float64)).amax(-1)
    w = torch.exp(x - x.amax(-1, keepdim=True))
    w = w / w.sum(-1, keepdim=True)
    out = torch.einsum("rhgt,thd->rhgd", w, v)
    spread = torch.einsum("rhgt,thd->rhgd", w, v.abs())
    return out.reshape(R, Hq, d), spread.reshape(R, Hq, d), mass.reshape(R, Hq, 1)


def attention_bound(out, spread, mass, d, scale, out_dtype, weights=None):
    """weights: (type the weights are rounded to, a bound on sum |v|), or None for value and residual."""
    ds = d * 2.0 ** -23 * mass * scale
    err = (2 * ds + 2.0 ** -16 + 2.0 ** -22 + 2.0 ** -14) * spread
    if weights is not None:
        err = err + EPS[weights[0]] / 2 * spread + TINY[weights[0]] / 2 * weights[1]
    return err + rounding(out, err, out_dtype)


def gathered(cache, table, n):
    """The first n positions of a sequence, [n, Hkv, d] in 64 bits on the CPU."""
    t = torch.arange(n)
    blk = table.cpu().long()[t // 16]
    ok = (blk >= 0) & (blk < cache.shape[0])
    rows = cache.cpu()[blk.clamp(0, cache.shape[0] - 1), :, t % 16].double()
    return torch.where(ok.view(n, 1, 1), rows, torch.zeros((), dtype=torch.float64))


def assert_within(got, ref, bound, what=""):
    got = got.double().cpu()
    assert got.shape == ref.shape, (got.shape, ref.shape)
    bad = ~((got - ref).abs() <= bound)   # NaN counts as bad
    if bad.any():
        i = tuple(int(x) for x in np.unravel_index(int(((got - ref).abs() - bound).nan_to_num(1e30).argmax()), got.shape))
        raise AssertionError("%s: %d of %d outside the bound; worst at %s: got %.8g, expected %.8g, bound %.3g"
                             % (what, int(bad.sum()), bad.numel(), i, got[i], ref[i], bound[i]))


def release(table, seq_lens, finished, window, sinks, free, count, num_blocks):
    """pkv_release_blocks on Python lists; returns (table, free, count)."""
    table, free = [list(r) for r in table], list(free)
    for s, n in enumerate(seq_lens):
        for j in range(-(-n // 16)):
            out = bool(finished[s]) if finished is not None else False
            if not out and window > 0:
                # no position of the block is seen by any position from n on
                out = 16 * (j + 1) <= n - window + 1 and 16 * j >= sinks
            if out and 0 <= table[s][j] < num_blocks:
                free[count] = table[s][j]
                count += 1
                table[s][j] = -1
    return table, free, count


def step_tables(lens, new, table, free, count, max_tokens):
    """pkv_step_tables on Python lists (a step that fits)."""
    table = [list(r) for r in table]
    ctx, cu, slots, pos = [], [0], [], []
    for s, (n, m) in enumerate(zip(lens, new)):
        for j in range(-(-n // 16), -(-(n + m) // 16)):
            count -= 1
            table[s][j] = free[count]
        for p in range(n, n + m):
            slots.append(table[s][p // 16] * 16 + p % 16)
            pos.append(p)
        ctx.append(n + m)
        cu.append(cu[-1] + m)
    pad = max_tokens - len(slots)
    return table, count, ctx, cu, slots + [-1] * pad, pos + [0] * pad
