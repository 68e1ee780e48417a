"""Sliding-window attention over the paged cache (decode and prefill) against
the definition in 64 bits, with the bounds derived in window_ref."""
import math

import pytest
import torch

import window_ref as ref
from paged_kv_cache_tables_gb300 import (PkvError, paged_decode_attention, paged_prefill_attention,
                                         paged_window_decode_attention, paged_window_prefill_attention)

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


class Step:
    """Sequences of the given contexts and new rows in shuffled blocks.  What no row may see holds NaN: the tail of
    the last block, hidden positions, and blocks out of sight are not even in the table (their entries are -1 or an
    id past the pool)."""

    def __init__(self, ctx, qn, Hq, Hkv, d, dtype, window, sinks, seed=0, poison=True, heavy=False):
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
        k = torch.randn(NB, Hkv, 16, d, generator=g).to(dtype)
        v = torch.randn(NB, Hkv, 16, d, generator=g).to(dtype)
        self.table = torch.full((len(ctx), self.max_blocks), -1, dtype=torch.int32)
        at = 0
        for s, (c, n) in enumerate(zip(ctx, qn)):
            self.table[s, :nb[s]] = ids[at:at + nb[s]].int()
            at += nb[s]
            t = torch.arange(nb[s] * 16)
            p = torch.arange(c - n, c).view(n, 1)
            vis = (ref.seen(p, t, window, sinks) & (t < c)).any(0) if n else torch.zeros(nb[s] * 16, dtype=torch.bool)
            if not poison:
                continue
            blk = self.table[s].long()[t // 16]
            k[blk[~vis], :, (t % 16)[~vis]] = float("nan")
            v[blk[~vis], :, (t % 16)[~vis]] = float("inf")
            gone = ~vis.view(-1, 16).any(1)
            self.table[s, :nb[s]][gone] = NB + 7 if s % 2 else -1
        self.k, self.v = k.cuda(), v.cuda()
        self.dev = dict(q=self.q.cuda(), table=self.table.cuda(), ctx=torch.tensor(ctx, dtype=torch.int32).cuda(),
                        cu=torch.tensor([0] + torch.tensor(qn).cumsum(0).tolist(), dtype=torch.int32).cuda())
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def reference(self, out_dtype, prefill=False):
        out, bound, at = [], [], 0
        for s, (c, n) in enumerate(zip(self.ctx, self.qn)):
            q = self.q[at:at + n].double()
            at += n
            if c == 0 or n == 0:
                out.append(torch.zeros_like(q))
                bound.append(torch.zeros_like(q))
                continue
            v = ref.gathered(self.v, self.table[s], c)
            o, sp, mass = ref.attend(q, c - n, ref.gathered(self.k, self.table[s], c), v, self.window, self.sinks,
                                     self.scale)
            out.append(o)
            # a 16-bit output of prefill: weights of that type, over at most c values of |v| up to the largest
            w = (out_dtype, c * v.abs().nan_to_num(0, 0, 0).max()) if prefill and out_dtype != F32 else None
            bound.append(ref.attention_bound(o, sp, mass, self.d, self.scale, out_dtype, w))
        return torch.cat(out), torch.cat(bound)

    def decode(self, out_dtype, **kw):
        out = torch.full(self.q.shape, float("nan"), dtype=out_dtype, device="cuda")
        paged_window_decode_attention(out, self.dev["q"], self.k, self.v, self.dev["table"], self.dev["ctx"], self.window,
                                      num_sinks=self.sinks, dev_status=self.status, **kw)
        return out

    def prefill(self, out_dtype, max_q=None, **kw):
        out = torch.full(self.q.shape, float("nan"), dtype=out_dtype, device="cuda")
        paged_window_prefill_attention(out, self.dev["q"], self.dev["cu"], max_q or max(self.qn), self.k, self.v,
                                       self.dev["table"], self.dev["ctx"], self.window, num_sinks=self.sinks,
                                       dev_status=self.status, **kw)
        return out


WINDOWS = [(1, 0), (1, 1), (2, 0), (16, 0), (17, 4), (31, 16), (33, 17), (128, 0), (129, 4), (200, 100), (1000, 128),
           (700, 1), (100000, 0), (2 ** 31 - 1, 2 ** 31 - 1), (3, 2 ** 31 - 1)]
CONTEXTS = [0, 1, 2, 15, 16, 17, 33, 127, 128, 129, 256, 300, 511, 777, 1100, 1999]


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("Hq,Hkv,d,dtype,out_dtype", [(8, 2, 64, F16, F32), (4, 1, 128, BF16, F32), (8, 2, 128, BF16, BF16)])
def test_decode(cuda_lib, window, sinks, Hq, Hkv, d, dtype, out_dtype):
    st = Step(CONTEXTS, [1] * len(CONTEXTS), Hq, Hkv, d, dtype, window, sinks, seed=window % 97)
    got = st.decode(out_dtype)
    want, bound = st.reference(out_dtype)
    ref.assert_within(got, want, bound, "window %d, sinks %d" % (window, sinks))
    assert (got[0] == 0).all() and st.status.item() == 0


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (6, 2), (20, 4), (16, 2), (9, 1), (16, 1), (32, 2), (16, 16), (15, 5)])
@pytest.mark.parametrize("d,dtype", [(64, BF16), (128, F16), (64, F16), (128, BF16)])
def test_decode_head_layouts(cuda_lib, Hq, Hkv, d, dtype):
    ctx = [700, 5, 0, 64]
    st = Step(ctx, [1] * 4, Hq, Hkv, d, dtype, 300, 20, seed=Hq, heavy=True)
    want, bound = st.reference(dtype)
    ref.assert_within(st.decode(dtype), want, bound)
    assert st.status.item() == 0


@pytest.mark.parametrize("S,hi,window", [(1, 40000, 30000), (1, 9000, 100), (2, 3000, 2900), (5, 9000, 9000), (64, 300, 128),
                                         (160, 200, 64), (700, 90, 40)])
def test_decode_every_split(cuda_lib, S, hi, window):
    """From one sequence (a range over a whole cluster) to many (a CTA a range); the same bits at every call."""
    ctx = [max(1, hi - 37 * i % hi) for i in range(S)]
    st = Step(ctx, [1] * S, 4, 2, 128, BF16, window, 4, seed=S)
    got = st.decode(F32)
    want, bound = st.reference(F32)
    ref.assert_within(got, want, bound)
    for _ in range(3):
        assert torch.equal(st.decode(F32), got)


@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 0), (33, 17), (200, 100), (700, 1), (100000, 0)])
@pytest.mark.parametrize("Hq,Hkv,d,dtype,out_dtype", [(4, 4, 64, F16, F32), (32, 4, 128, BF16, F32), (12, 4, 128, F16, F16),
                                                      (20, 4, 64, BF16, BF16)])
def test_decode_many_ranges(cuda_lib, window, sinks, Hq, Hkv, d, dtype, out_dtype):
    """More ranges than SMs: contexts from none to a few hundred tokens beside long ones, in one batch."""
    ctx = [CONTEXTS[i % len(CONTEXTS)] if i % 3 else (i * 37) % 400 for i in range(100)]
    st = Step(ctx, [1] * len(ctx), Hq, Hkv, d, dtype, window, sinks, seed=window % 83)
    got = st.decode(out_dtype)
    want, bound = st.reference(out_dtype)
    ref.assert_within(got, want, bound, "window %d, sinks %d" % (window, sinks))
    assert st.status.item() == 0
    for _ in range(2):
        assert torch.equal(st.decode(out_dtype), got)


def test_decode_many_ranges_reports_bad_entries(cuda_lib):
    ctx = [40 + i for i in range(200)]
    st = Step(ctx, [1] * 200, 8, 2, 64, F16, 64, 4, poison=False)
    st.table[60, 4] = 10 ** 6     # context 100, positions 64 to 79: visible, reads zeros
    st.dev["table"] = st.table.cuda()
    want, bound = st.reference(F32)
    ref.assert_within(st.decode(F32), want, bound)
    assert st.status.item() == 1
    st.status.zero_()
    st.dev["ctx"][3], st.dev["ctx"][5] = -7, 10 ** 8
    got = st.decode(F32)
    assert st.status.item() == 3 and (got[3] == 0).all() and torch.isfinite(got).all()
    keep = [i for i in range(200) if i not in (3, 5)]
    ref.assert_within(got[keep], want[keep], bound[keep])


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("Hq,Hkv,d,dtype,out_dtype", [(8, 2, 64, F16, F32), (4, 1, 128, BF16, F32), (8, 2, 128, BF16, BF16)])
def test_prefill(cuda_lib, window, sinks, Hq, Hkv, d, dtype, out_dtype):
    # prior context and rows: none, one, around a block, around a key tile, around a pair of query tiles
    ctx, qn = [1, 1, 16, 129, 300, 63, 400, 1200, 700, 0, 64], [1, 1, 16, 129, 1, 62, 65, 130, 257, 0, 64]
    # poisoned positions only where no row of the whole chunk sees them
    st = Step(ctx, qn, Hq, Hkv, d, dtype, window, sinks, seed=window % 89)
    got = st.prefill(out_dtype)
    want, bound = st.reference(out_dtype, True)
    ref.assert_within(got, want, bound, "window %d, sinks %d" % (window, sinks))
    assert st.status.item() == 0


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (6, 2), (20, 4), (9, 1), (16, 1), (32, 2), (16, 16), (15, 5)])
@pytest.mark.parametrize("d,dtype", [(64, BF16), (128, F16), (64, F16), (128, BF16)])
def test_prefill_head_layouts(cuda_lib, Hq, Hkv, d, dtype):
    st = Step([500, 90, 260], [170, 90, 3], Hq, Hkv, d, dtype, 150, 20, seed=Hq, heavy=True)
    want, bound = st.reference(dtype, True)
    ref.assert_within(st.prefill(dtype), want, bound)
    assert st.status.item() == 0


@pytest.mark.parametrize("Hq,Hkv,d,dtype,out_dtype", [(32, 2, 64, BF16, BF16), (32, 2, 128, F16, F16), (32, 2, 128, BF16, F32),
                                                      (20, 4, 128, BF16, BF16), (20, 4, 64, F16, F32)])
@pytest.mark.parametrize("window,sinks", [(300, 20), (40, 0), (5000, 0)])
def test_prefill_of_many_units(cuda_lib, Hq, Hkv, d, dtype, out_dtype, window, sinks):
    """More units than SMs: a CTA takes several, of one key tile up to many, and some chunks have none."""
    st = Step([700, 1400, 333, 900, 640, 0], [700, 650, 1, 512, 333, 0], Hq, Hkv, d, dtype, window, sinks)
    want, bound = st.reference(out_dtype, True)
    got = st.prefill(out_dtype)
    ref.assert_within(got, want, bound)
    assert torch.equal(got, st.prefill(out_dtype)) and st.status.item() == 0


def test_prefill_without_sinks_far_behind(cuda_lib):
    """Rows whose first walked key tile holds none of their keys, long contexts."""
    st = Step([6000, 5000], [300, 1], 4, 1, 128, BF16, 20, 0, seed=3)
    want, bound = st.reference(F32)
    ref.assert_within(st.prefill(F32), want, bound)
    st = Step([6000, 5000], [300, 700], 4, 1, 64, F16, 1500, 300, seed=4)
    want, bound = st.reference(F32)
    ref.assert_within(st.prefill(F32), want, bound)


@pytest.mark.parametrize("d", [64, 128])
def test_a_window_of_the_whole_context_is_causal_attention(cuda_lib, d):
    st = Step([300, 64, 1, 900], [100, 64, 1, 7], 8, 2, d, BF16, 10 ** 6, 0, poison=False)
    plain = torch.full(st.q.shape, float("nan"), dtype=F32, device="cuda")
    paged_prefill_attention(plain, st.dev["q"], st.dev["cu"], 100, st.k, st.v, st.dev["table"], st.dev["ctx"])
    want, bound = st.reference(F32)
    ref.assert_within(st.prefill(F32), plain.double().cpu(), 2 * bound)
    st = Step([300, 64, 1, 900], [1] * 4, 8, 2, d, BF16, 10 ** 6, 0, poison=False)
    plain = torch.full(st.q.shape, float("nan"), dtype=F32, device="cuda")
    paged_decode_attention(plain, st.dev["q"], st.k, st.v, st.dev["table"], st.dev["ctx"])
    want, bound = st.reference(F32)
    ref.assert_within(st.decode(F32), plain.double().cpu(), 2 * bound)


def test_one_row_chunks_equal_decode(cuda_lib):
    ctx = [700, 33, 1, 250]
    st = Step(ctx, [1] * 4, 8, 2, 128, BF16, 100, 10)
    want, bound = st.reference(F32)
    ref.assert_within(st.prefill(F32), want, bound)
    ref.assert_within(st.decode(F32), want, bound)


def test_bad_blocks_and_contexts_are_reported(cuda_lib):
    # a visible entry outside the pool reads zeros: the value of a zero key and a zero row
    st = Step([40, 200], [1, 1], 4, 1, 64, F16, 64, 4, poison=False)
    st.table[1, 12] = 9999
    st.dev["table"] = st.table.cuda()
    want, bound = st.reference(F32)
    ref.assert_within(st.decode(F32), want, bound)
    assert st.status.item() == 1
    st.status.zero_()
    ref.assert_within(st.prefill(F32), want, bound)
    assert st.status.item() == 1
    # a context past the table is clamped by decode (and skipped by prefill), a negative one is empty
    st = Step([96, 200], [1, 1], 4, 1, 64, F16, 64, 4, poison=False)
    st.dev["table"] = torch.cat([st.table[:, :12], st.table[:, :1]], 1).contiguous().cuda()
    st.dev["ctx"][:] = torch.tensor([-5, 10 ** 6], dtype=torch.int32)
    got = st.decode(F32)
    assert st.status.item() == 2 and (got[0] == 0).all() and torch.isfinite(got).all()
    st.status.zero_()
    got = st.prefill(F32)
    assert st.status.item() == 2 | 16 and torch.isnan(got).all()


def test_chunks_outside_the_rows_are_skipped(cuda_lib):
    st = Step([40, 200, 30], [5, 6, 7], 4, 1, 64, F16, 64, 4)
    want, _ = st.reference(F32)
    st.dev["cu"][:] = torch.tensor([0, 5, 30, 18], dtype=torch.int32)   # the second ends past the rows, the third is negative
    got = st.prefill(F32, max_q=32)
    assert st.status.item() == 16
    assert torch.isfinite(got[:5]).all() and torch.isnan(got[5:]).all()
    st.status.zero_()
    st.dev["cu"][:] = torch.tensor([-3, 2, 5, 18], dtype=torch.int32)
    got = st.prefill(F32, max_q=32)
    assert st.status.item() == 16 and torch.isnan(got[:2]).all()


def test_rows_behind_the_last_chunk_are_left_as_they_were(cuda_lib):
    st = Step([40, 200], [5, 70], 4, 1, 64, F16, 64, 4)
    out = torch.full((100, 4, 64), 7.0, dtype=F16, device="cuda")
    q = torch.zeros(100, 4, 64, dtype=F16, device="cuda")
    q[:75] = st.dev["q"]
    paged_window_prefill_attention(out, q, st.dev["cu"], 70, st.k, st.v, st.dev["table"], st.dev["ctx"], 64, num_sinks=4)
    want, bound = st.reference(F16, True)
    ref.assert_within(out[:75], want, bound)
    assert (out[75:] == 7).all()


def test_captured_and_on_side_streams(cuda_lib):
    """Two graphs and two streams share the inputs; replayed on contexts that change between replays."""
    st = Step([300, 700, 64, 900], [1] * 4, 8, 2, 128, BF16, 128, 4, poison=False)
    pf = Step([300, 700, 64, 900], [40, 1, 64, 130], 8, 2, 128, BF16, 128, 4, poison=False)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    gd, gp = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(gd, stream=side):
        od = st.decode(F32)
    with torch.cuda.graph(gp, stream=side):
        op = pf.prefill(F32)
    for shift in (0, 17):
        st.ctx = [c - shift for c in st.ctx]
        st.dev["ctx"].copy_(torch.tensor(st.ctx))
        gd.replay()
        gp.replay()
        ref.assert_within(od, *st.reference(F32))
        ref.assert_within(op, *pf.reference(F32))
    many = Step([50 + i for i in range(200)], [1] * 200, 8, 2, 64, F16, 40, 4, poison=False)
    gm = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(gm, stream=side):
        om = many.decode(F32)
    gm.replay()
    ref.assert_within(om, *many.reference(F32))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for s in streams:
        with torch.cuda.stream(s):
            outs.append((st.decode(F32), pf.prefill(F32)))
    torch.cuda.synchronize()
    for a, b in outs:
        assert torch.equal(a, od) and torch.equal(b, op)


def test_offsets_past_32_bits(cuda_lib):
    """A cache of more than 2^32 elements, its last blocks in use."""
    NB, Hkv, d = 264000, 8, 128
    k = torch.zeros(NB, Hkv, 16, d, dtype=BF16, device="cuda")
    v = torch.zeros(NB, Hkv, 16, d, dtype=BF16, device="cuda")
    assert (NB - 20) * Hkv * 16 * d > 2 ** 32
    g = torch.Generator(device="cuda").manual_seed(1)
    k[-20:] = torch.randn(20, Hkv, 16, d, generator=g, device="cuda", dtype=BF16)
    v[-20:] = torch.randn(20, Hkv, 16, d, generator=g, device="cuda", dtype=BF16)
    small = Step([300], [1], 16, 8, d, BF16, 100, 20, poison=False)
    small.k, small.v = k[-20:].clone(), v[-20:].clone()
    small.table = torch.arange(20, dtype=torch.int32).view(1, 20)
    want, bound = small.reference(F32)
    small.k, small.v = k, v
    small.dev["table"] = (small.table + NB - 20).cuda()
    ref.assert_within(small.decode(F32), want, bound)
    ref.assert_within(small.prefill(F32), want, bound)


def test_refusals(cuda_lib):
    st = Step([40, 200], [1, 1], 4, 1, 64, F16, 64, 4)
    for window, sinks in ((0, 4), (-1, 0), (64, -1)):
        st.window, st.sinks = window, sinks
        with pytest.raises(PkvError):
            st.decode(F32)
        with pytest.raises(PkvError):
            st.prefill(F32)
    st.window, st.sinks = 64, 4
    for scale in (0.0, -1.0, float("nan")):
        with pytest.raises(PkvError):
            st.decode(F32, scale=scale)
        with pytest.raises(PkvError):
            st.prefill(F32, scale=scale)
    with pytest.raises(PkvError):
        st.decode(BF16)          # an output of the other 16-bit type
    st.dev["q"] = st.dev["q"].float()
    with pytest.raises((PkvError, TypeError)):
        st.decode(F32)
    st.dev["q"] = st.q.cuda().transpose(1, 2)
    with pytest.raises((ValueError, PkvError)):
        st.decode(F32)
    assert st.status.item() == 0


def test_equal_results_at_any_pool_size_and_block_order(cuda_lib):
    a = Step([500, 90], [1, 1], 8, 2, 64, F16, 128, 4, poison=False)
    want = a.decode(F32)
    perm = torch.randperm(a.k.shape[0] + 50, generator=torch.Generator().manual_seed(9))[:a.k.shape[0]]
    k = torch.zeros(a.k.shape[0] + 50, *a.k.shape[1:], dtype=F16, device="cuda")
    v = torch.zeros_like(k)
    k[perm.cuda()], v[perm.cuda()] = a.k, a.v
    table = torch.where(a.table >= 0, perm[a.table.clamp(min=0).long()].int(), a.table)
    a.k, a.v, a.dev["table"] = k, v, table.cuda()
    assert torch.equal(a.decode(F32), want)
