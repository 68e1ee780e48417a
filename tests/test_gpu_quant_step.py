"""The step of a serving loop over a cache held in 8 bits, as its operators are
used together: tables from the request lengths, queries and keys normed and
rotated, keys and values appended as codes, attention over a window and the first
tokens, rows read back, blocks given back and, in the end, swapped out to host
memory and in again.  And the calls that a loop makes around that: two at once on
two streams, caches past 4 GB, batches padded to a capacity.  Codes and scales are
held to the definition exactly, outputs to it within the derived bounds."""
import math
import os
import shutil
import subprocess
import sys

import pytest
import torch

import quant_ref as qr
import window_ref as ref
from paged_kv_cache_tables_gb300 import _binding as B
from paged_kv_cache_tables_gb300 import (copy_blocks, kv_append_e4m3, kv_gather_e4m3, paged_decode_attention_e4m3,
                                         paged_prefill_attention_e4m3, qk_rope, release_blocks, rope_frequencies,
                                         step_tables)
from quant_ref import BF16, F16, F32, Step
from test_gpu_rope import check as check_rotated

pytestmark = pytest.mark.gpu

WINDOW, SINKS, EPS = 40, 5, 1e-6
WHOLE = 2 ** 31 - 1


class Loop:
    """Arrays of one capacity: a step of fewer tokens leaves padding rows behind its last."""

    def __init__(self, S, Hq, Hkv, d, dtype, max_blocks, pool, capacity, chunk):
        self.S, self.Hq, self.Hkv, self.d, self.dtype, self.NB = S, Hq, Hkv, d, dtype, pool
        self.capacity, self.chunk, self.scale = capacity, chunk, 1 / math.sqrt(d)
        i32 = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")   # noqa: E731
        g = self.g = torch.Generator().manual_seed(S)
        free = torch.randperm(pool, generator=g).int()
        self.lens, self.new, self.table = i32(S), i32(S), i32(S, max_blocks).fill_(-1)
        self.free, self.count, self.cu = free.cuda(), i32(1).fill_(pool), i32(S + 1)
        self.finished, self.status, self.first = i32(S), i32(1), i32(S)
        self.slots = torch.zeros(capacity, dtype=torch.int64, device="cuda")
        self.pos = i32(capacity)
        self.qkv = torch.zeros(capacity, (Hq + 2 * Hkv) * d, dtype=dtype, device="cuda")
        self.q_out = torch.zeros(capacity, Hq, d, dtype=dtype, device="cuda")
        self.k_out = torch.zeros(capacity, Hkv, d, dtype=dtype, device="cuda")
        self.out = torch.zeros(capacity, Hq, d, dtype=F32, device="cuda")
        self.k_back = torch.zeros(capacity, Hkv, d, dtype=F32, device="cuda")
        self.v_back = torch.zeros_like(self.k_back)
        # what no call has written yet: NaN codes, NaN scales
        self.kc = torch.full((pool, Hkv, 16, d), 127, dtype=torch.uint8)
        self.vc = self.kc.clone()
        self.scales = torch.full((pool, Hkv, 2), float("nan"), dtype=torch.float64)
        self.dkc, self.dvc = self.kc.cuda().view(qr.CODE), self.vc.cuda().view(qr.CODE)
        self.dscales = self.scales.float().cuda()
        self.freqs, self.m = rope_frequencies(d // 2)
        self.p_lens, self.p_table = [0] * S, self.table.tolist()
        self.p_free, self.p_count = free.tolist(), pool

    def parts(self):
        a, b, T = self.Hq * self.d, self.Hkv * self.d, self.capacity
        return (self.qkv[:, :a].view(T, self.Hq, self.d), self.qkv[:, a:a + b].view(T, self.Hkv, self.d),
                self.qkv[:, a + b:].view(T, self.Hkv, self.d))

    def step(self, decode):
        q, k, v = self.parts()
        cache = (self.dkc, self.dvc, self.dscales)
        self.first.copy_(self.lens)
        step_tables(self.lens, self.new, self.table, self.free, self.count, self.NB, self.lens, self.cu, self.slots,
                    self.pos, dev_status=self.status)
        qk_rope(self.q_out, self.k_out, q, k, self.pos, self.freqs, mscale=self.m, eps=EPS)
        kv_append_e4m3(self.k_out, v, self.slots, *cache, dev_status=self.status)
        if decode:
            paged_decode_attention_e4m3(self.out[:self.S], self.q_out[:self.S], *cache, self.table, self.lens,
                                        window=WINDOW, num_sinks=SINKS, dev_status=self.status)
        else:
            paged_prefill_attention_e4m3(self.out, self.q_out, self.cu, self.chunk, *cache, self.table, self.lens,
                                         window=WINDOW, num_sinks=SINKS, dev_status=self.status)
        kv_gather_e4m3(self.k_back, self.v_back, *cache, self.table, self.cu, first=self.first, dev_status=self.status)
        release_blocks(self.table, self.lens, self.free, self.count, self.NB, finished=self.finished, window=WINDOW,
                       num_sinks=SINKS, dev_status=self.status)

    def fill(self, new, finished):
        self.new.copy_(torch.tensor(new, dtype=torch.int32))
        self.finished.copy_(torch.tensor(finished, dtype=torch.int32))
        self.qkv.copy_(torch.randn(self.qkv.shape, generator=self.g).to(self.dtype))
        for t in (self.out, self.k_back, self.v_back):
            t.fill_(-7.0)

    def verify(self, new, finished):
        before = list(self.p_lens)
        t, n, ctx, cu, slots, pos = ref.step_tables(before, new, self.p_table, self.p_free, self.p_count, self.capacity)
        assert self.status.item() == 0 and self.slots.tolist() == slots and self.lens.tolist() == ctx
        q, k, v = (x.cpu() for x in self.parts())
        T = cu[-1]
        where = torch.tensor(pos[:T])
        k_out, q_out = self.k_out.cpu(), self.q_out.cpu()
        check_rotated(k_out[:T], k[:T], where, self.freqs, self.m, self.d // 2, False, None, EPS, "k")
        qr.append(k_out.double(), slots, self.kc, self.scales, 0)
        qr.append(v.double(), slots, self.vc, self.scales, 1)
        assert torch.equal(self.dkc.view(torch.uint8).cpu(), self.kc)
        assert torch.equal(self.dvc.view(torch.uint8).cpu(), self.vc)
        assert torch.equal(self.dscales.cpu().double().nan_to_num(-1.0), self.scales.nan_to_num(-1.0))
        for got in (self.out, self.k_back, self.v_back):
            assert (got[T:] == -7.0).all()
        out, k_back, v_back = (x.double().cpu() for x in (self.out, self.k_back, self.v_back))
        for s in range(self.S):
            a, b = cu[s], cu[s + 1]
            if a == b:
                continue
            table = torch.tensor(t[s])
            keys = qr.gathered(self.kc, self.scales[..., 0], table, ctx[s])
            values = qr.gathered(self.vc, self.scales[..., 1], table, ctx[s])
            assert torch.equal(k_back[a:b], keys[before[s]:]) and torch.equal(v_back[a:b], values[before[s]:])
            want, spread, mass = ref.attend(q_out[a:b].double(), before[s], keys, values, WINDOW, SINKS, self.scale)
            held = table.long()[table >= 0]
            largest = qr.CODE_MAX * self.scales[held, :, 1].max().item()
            ref.assert_within(out[a:b], want, qr.attention_bound(want, spread, mass, self.d, self.scale, F32, largest,
                                                                 ctx[s]), "sequence %d" % s)
        self.p_lens = ctx
        self.p_table, self.p_free, self.p_count = ref.release(t, ctx, finished, WINDOW, SINKS, self.p_free, n, self.NB)
        assert self.table.tolist() == self.p_table and self.count.item() == self.p_count
        for s in range(self.S):
            if finished[s]:
                self.p_lens[s] = 0
        self.lens.masked_fill_(self.finished != 0, 0)

    def swap(self):
        """Every block in use out to host memory, other codes in its place, and in again elsewhere."""
        used = sorted({b for row in self.p_table for b in row if b >= 0})
        pairs = torch.tensor([[b, i] for i, b in enumerate(used)], dtype=torch.int32).cuda()
        arrays = [self.dkc, self.dvc, self.dscales]
        hosts = [torch.empty((len(used),) + a.shape[1:], dtype=a.dtype).pin_memory() for a in arrays]
        to = [b for b in range(self.NB) if b not in used][:len(used)]
        assert len(to) == len(used)
        back = torch.tensor([[i, b] for i, b in enumerate(to)], dtype=torch.int32).cuda()
        for a, h in zip(arrays, hosts):
            copy_blocks(h, a, pairs, dev_status=self.status)
        for a, h in zip(arrays, hosts):
            a.view(torch.uint8).fill_(127)
            copy_blocks(a, h, back, dev_status=self.status)
        for a in (self.kc, self.vc):
            rows = a[used].clone()
            a.fill_(127)
            a[to] = rows
        rows = self.scales[used].clone()
        nan = self.dscales.clone()
        nan.view(torch.uint8).fill_(127)
        self.scales.copy_(nan.cpu().double())
        self.scales[to] = rows
        move = dict(zip(used, to))
        self.p_table = [[move.get(b, -1) for b in row] for row in self.p_table]
        swapped = {b: a for a, b in move.items()}            # (entries past the count say nothing)
        self.p_free = [swapped.get(b, b) for b in self.p_free]
        self.table.copy_(torch.tensor(self.p_table, dtype=torch.int32))
        self.free.copy_(torch.tensor(self.p_free, dtype=torch.int32))


@pytest.mark.parametrize("S,Hq,Hkv,d,dtype", [(6, 8, 2, 64, BF16), (5, 4, 4, 128, F16), (3, 12, 2, 128, BF16)])
def test_prompts_then_decode_steps_from_a_graph(cuda_lib, S, Hq, Hkv, d, dtype):
    loop = Loop(S, Hq, Hkv, d, dtype, max_blocks=16, pool=S * 12, capacity=200, chunk=60)
    idle, one = [0] * S, [1] * S
    for new in ([60, 1, 33, 17, 16, 48][:S], [20, 40, 0, 31, 60, 2][:S]):
        loop.fill(new, idle)
        loop.step(decode=False)
        loop.verify(new, idle)
    loop.fill(one, idle)
    loop.step(decode=True)
    loop.verify(one, idle)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        loop.step(decode=True)
    torch.cuda.current_stream().wait_stream(side)
    for step in range(40):
        finished = [int(step in (9, 30) and s == step % S) for s in range(S)]
        if step == 20:
            loop.swap()
        loop.fill(one, finished)
        graph.replay()
        loop.verify(one, finished)


def test_prompt_steps_from_one_graph(cuda_lib):
    """A graph of the prompts' step, replayed on other lengths: none, one, a whole chunk."""
    S = 4
    loop = Loop(S, 8, 2, 128, BF16, max_blocks=16, pool=60, capacity=150, chunk=64)
    idle = [0] * S
    loop.fill([3, 0, 1, 20], idle)
    loop.step(decode=False)
    loop.verify([3, 0, 1, 20], idle)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        loop.step(decode=False)
    torch.cuda.current_stream().wait_stream(side)
    for new in ([64, 1, 0, 16], [0, 0, 0, 0], [1, 64, 64, 1], [1, 1, 1, 1], [0, 13, 2, 64]):
        loop.fill(new, idle)
        graph.replay()
        loop.verify(new, idle)


# ---- decode in order of the contexts' lengths, whole and in ranges --------------------------------------------------
@pytest.mark.parametrize("S,hi,Hq,Hkv,window,sinks", [(64, 900, 16, 8, WHOLE, 0), (32, 4000, 32, 8, WHOLE, 0),
                                                      (200, 500, 8, 8, 300, 4), (48, 2500, 40, 8, 2000, 0),
                                                      (1024, 60, 8, 8, WHOLE, 0), (1025, 60, 8, 8, WHOLE, 0)])
def test_decode_of_uneven_contexts(cuda_lib, S, hi, Hq, Hkv, window, sinks):
    """Contexts from 0 up, in no order; equal ones among them; the same bits at every call."""
    g = torch.Generator().manual_seed(S)
    ctx = torch.randint(0, hi + 1, (S,), generator=g)
    ctx[::7], ctx[1::5] = 0, hi // 2
    ctx[S // 2] = hi
    st = Step(ctx.tolist(), [1] * S, Hq, Hkv, 64, F16, window, sinks, seed=S, poison=False)
    got = st.decode(F32)
    want, bound = st.reference(F32)
    ref.assert_within(got, want, bound)
    assert st.status.item() == 0 and torch.equal(st.decode(F32), got)


# ---- two calls at once ----------------------------------------------------------------------------------------------
def test_calls_on_two_streams(cuda_lib):
    """Two steps over two caches, interleaved on two streams, give the bits that they give alone."""
    a = Step([4000, 17, 2500], [700, 17, 300], 8, 2, 128, BF16, WHOLE, 0, seed=1, poison=False)
    b = Step([1800] * 9, [40] * 9, 16, 4, 64, F16, 500, 3, seed=2, poison=False)
    c = Step([3000, 100, 0, 900], [1] * 4, 8, 2, 128, BF16, WHOLE, 0, seed=3, poison=False)
    e = Step([600] * 90, [1] * 90, 16, 4, 64, F16, 500, 3, seed=4, poison=False)
    alone = [a.prefill(F32), b.prefill(F32), c.decode(F32), e.decode(F32)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[torch.full_like(x, float("nan")) for x in alone] for _ in range(6)]
    torch.cuda.synchronize()

    def prefill(st, out, stream):
        paged_prefill_attention_e4m3(out, st.dev["q"], st.dev["cu"], max(st.qn), st.k, st.v, st.dev["scales"],
                                     st.dev["table"], st.dev["ctx"], window=st.window, num_sinks=st.sinks,
                                     dev_status=st.status, stream=stream)

    def decode(st, out, stream):
        paged_decode_attention_e4m3(out, st.dev["q"], st.k, st.v, st.dev["scales"], st.dev["table"], st.dev["ctx"],
                                    window=st.window, num_sinks=st.sinks, dev_status=st.status, stream=stream)

    for turn, o in enumerate(outs):
        one, two = streams if turn % 2 else streams[::-1]
        prefill(a, o[0], one)
        prefill(b, o[1], two)
        decode(c, o[2], two)
        decode(e, o[3], one)
    torch.cuda.synchronize()
    for o in outs:
        for got, want in zip(o, alone):
            assert torch.equal(got, want)


def test_appends_and_reads_on_another_stream(cuda_lib):
    g = torch.Generator().manual_seed(8)
    S, Hkv, d, n = 3, 2, 128, 50
    k, v = (torch.randn(S * n, Hkv, d, generator=g).to(BF16).cuda() for _ in range(2))
    kc = torch.zeros(20, Hkv, 16, d, dtype=torch.uint8, device="cuda").view(qr.CODE)
    vc, sc = kc.clone(), torch.zeros(20, Hkv, 2, device="cuda")
    table = torch.arange(S * 4, dtype=torch.int32, device="cuda").view(S, 4)
    slots = torch.cat([s * 64 + torch.arange(n) for s in range(S)]).cuda()
    cu = torch.arange(0, S * n + 1, n, dtype=torch.int32, device="cuda")
    want_k, want_v = torch.empty(S * n, Hkv, d, device="cuda"), torch.empty(S * n, Hkv, d, device="cuda")
    kv_append_e4m3(k, v, slots, kc, vc, sc)
    kv_gather_e4m3(want_k, want_v, kc, vc, sc, table, cu)
    torch.cuda.synchronize()
    kc2, vc2, sc2 = (torch.zeros_like(x.view(torch.uint8)).view(x.dtype) for x in (kc, vc, sc))
    got_k, got_v = torch.zeros_like(want_k), torch.zeros_like(want_v)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    kv_append_e4m3(k, v, slots, kc2, vc2, sc2, stream=stream)
    kv_gather_e4m3(got_k, got_v, kc2, vc2, sc2, table, cu, stream=stream)
    stream.synchronize()
    assert torch.equal(got_k, want_k) and torch.equal(got_v, want_v) and torch.equal(sc, sc2)


# ---- caches whose offsets pass 32 bits ------------------------------------------------------------------------------
def test_caches_past_4_gb(cuda_lib):
    """The last blocks of a pool whose codes take 4.9 GB for K and for V hold the same rows as a small pool's: the same
    bits come out of every operator."""
    Hq, Hkv, d, big = 16, 8, 128, 300_000
    st = Step([900, 33, 16], [130, 33, 1], Hq, Hkv, d, BF16, WHOLE, 0, seed=5, poison=False)
    NB = st.kc.shape[0]
    assert (big - NB) * Hkv * 16 * d > 2 ** 32 and (big - NB) * Hkv * 16 * d - 2 ** 32 < 2 ** 31
    kc = torch.zeros(big, Hkv, 16, d, dtype=torch.uint8, device="cuda")
    vc = torch.zeros_like(kc)
    sc = torch.ones(big, Hkv, 2, device="cuda")
    kc[-NB:], vc[-NB:], sc[-NB:] = st.k.view(torch.uint8), st.v.view(torch.uint8), st.dev["scales"]
    kc, vc = kc.view(qr.CODE), vc.view(qr.CODE)
    table = torch.where(st.dev["table"] >= 0, st.dev["table"] + (big - NB), st.dev["table"])
    args = (kc, vc, sc, table)
    out = torch.empty(st.q.shape, device="cuda")
    paged_prefill_attention_e4m3(out, st.dev["q"], st.dev["cu"], 130, *args, st.dev["ctx"], dev_status=st.status)
    assert torch.equal(out, st.prefill(F32))
    dec = Step([900, 33, 16], [1, 1, 1], Hq, Hkv, d, BF16, WHOLE, 0, seed=5, poison=False)
    assert torch.equal(dec.table, st.table)
    for a, b in ((dec.k, st.k), (dec.v, st.v)):          # the same cache under other queries
        a.view(torch.uint8).copy_(b.view(torch.uint8))
    dec.dev["scales"].copy_(st.dev["scales"])
    out = torch.empty(dec.q.shape, device="cuda")
    paged_decode_attention_e4m3(out, dec.dev["q"], *args, dec.dev["ctx"], dev_status=st.status)
    assert torch.equal(out, dec.decode(F32))
    cu = torch.tensor([0, 900, 933, 949], dtype=torch.int32, device="cuda")
    got = [torch.empty(949, Hkv, d, dtype=BF16, device="cuda") for _ in range(4)]
    kv_gather_e4m3(*got[:2], *args, cu, dev_status=st.status)
    kv_gather_e4m3(*got[2:], st.k, st.v, st.dev["scales"], st.dev["table"], cu, dev_status=st.status)
    assert torch.equal(got[0], got[2]) and torch.equal(got[1], got[3])
    # 40 rows into the pool's last three blocks
    slots = torch.arange(40, device="cuda") + (NB - 3) * 16 + 3
    kv_append_e4m3(got[0][:40], got[1][:40], slots, st.k, st.v, st.dev["scales"], dev_status=st.status)
    kv_append_e4m3(got[0][:40], got[1][:40], slots + (big - NB) * 16, kc, vc, sc, dev_status=st.status)
    for a, b in ((kc, st.k), (vc, st.v)):
        assert torch.equal(a[-NB:].view(torch.uint8), b.view(torch.uint8))
    assert torch.equal(sc[-NB:], st.dev["scales"]) and (sc[:-NB] == 1).all()
    assert not kc.view(torch.uint8)[:-NB].any() and not vc.view(torch.uint8)[:-NB].any() and st.status.item() == 0


# ---- padded batches and queries that are not finite -----------------------------------------------------------------
@pytest.mark.parametrize("d,dtype,out_dtype", [(64, F16, F32), (128, BF16, BF16)])
def test_rows_behind_the_last_query(cuda_lib, d, dtype, out_dtype):
    """Rows of q and out from cu_seqlens[num_seqs] on: read by no one, left as they were."""
    st = Step([300, 0, 40], [150, 0, 7], 8, 2, d, dtype, WHOLE, 0, seed=6)
    want, bound = st.reference(out_dtype)
    n = len(st.q)
    q = torch.full((n + 200, 8, d), float("nan"), dtype=dtype, device="cuda")
    q[:n] = st.dev["q"]
    out = torch.full((n + 200, 8, d), -7.0, dtype=out_dtype, device="cuda")
    paged_prefill_attention_e4m3(out, q, st.dev["cu"], 150, st.k, st.v, st.dev["scales"], st.dev["table"], st.dev["ctx"],
                                 dev_status=st.status)
    ref.assert_within(out[:n], want, bound)
    assert (out[n:] == -7.0).all() and st.status.item() == 0


@pytest.mark.parametrize("d,dtype,out_dtype", [(64, F16, F32), (128, BF16, BF16), (128, BF16, F32)])
def test_queries_that_are_not_finite_stay_apart(cuda_lib, d, dtype, out_dtype):
    """A head of a token whose query holds NaN or infinities gives no number; every other row keeps its own."""
    for qn in ([1, 1, 1], [140, 9, 1]):
        st = Step([700, 33, 16], qn, 8, 2, d, dtype, WHOLE, 0, seed=7)
        want, bound = st.reference(out_dtype)
        bad = torch.zeros(st.q.shape[:2], dtype=torch.bool)
        bad[0, 1] = bad[0, 7] = bad[-1, 4] = True
        st.dev["q"][0, 1, 3] = float("nan")
        st.dev["q"][0, 7, 9] = float("inf")
        st.dev["q"][-1, 4, 0] = float("-inf")
        got = (st.decode if len(st.q) == 3 else st.prefill)(out_dtype)
        assert got.cpu()[bad].isnan().any(-1).all()
        ref.assert_within(got.cpu()[~bad], want[~bad], bound[~bad])
        assert st.status.item() == 0


# ---- the calls from Python ------------------------------------------------------------------------------------------
OLDER = """
#include <stddef.h>
int PyGILState_Check(void);
#define HELD(name) int name(void) { return PyGILState_Check(); }
HELD(pkv_paged_window_decode_attention)
HELD(pkv_paged_window_prefill_attention)
HELD(pkv_qk_rope)
HELD(pkv_qk_rope_append)
HELD(pkv_step_tables)
HELD(pkv_release_blocks)
size_t pkv_release_workspace_size(int n) { return 4 * (size_t)n; }
"""

WHOLE_LIBRARY = OLDER + """
HELD(pkv_kv_append_e4m3)
HELD(pkv_kv_gather_e4m3)
HELD(pkv_paged_decode_attention_e4m3)
HELD(pkv_paged_prefill_attention_e4m3)
"""

CALLS = """
import importlib.util, sys, torch
spec = importlib.util.spec_from_file_location("_torch_calls", sys.argv[1])
m = importlib.util.module_from_spec(spec)
spec.loader.exec_module(m)
x = torch.zeros(2, 2, 64, dtype=torch.float16, device="cuda")
c = torch.zeros(4, 2, 16, 64, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
k = torch.zeros(4, 2, 2, device="cuda")
i = torch.zeros(2, dtype=torch.int32, device="cuda")
t = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
cu = torch.zeros(3, dtype=torch.int32, device="cuda")
calls = [lambda: m.append_e4m3(x, x, i.long(), c, c, k, None, None),
         lambda: m.gather_e4m3(x, x, c, c, k, t, cu, None, None, None),
         lambda: m.decode_e4m3(x, x, c, c, k, t, i, 16, 0, None, None, None),
         lambda: m.prefill_e4m3(x, x, cu, 1, c, c, k, t, i, 16, 0, None, None, None)]
def outcome(f):
    try:
        return f()
    except RuntimeError as e:
        assert "rebuild" in str(e), e
        return "missing"
print([outcome(f) for f in calls])
"""


@pytest.mark.parametrize("library,want", [(WHOLE_LIBRARY, [0] * 4), (OLDER, ["missing"] * 4)], ids=["whole", "older"])
def test_python_calls_against_other_libraries(cuda_lib, tmp_path, library, want):
    """The interpreter is free while an entry point runs (it returns whether it is held); a library that has none of the
    four is named, and serves the module's other calls."""
    (tmp_path / "fake.c").write_text(library)
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(tmp_path / "libpkv.so"), str(tmp_path / "fake.c")], check=True)
    shutil.copy(B.CALLS_PATH, tmp_path / "_torch_calls.so")
    (tmp_path / "calls.py").write_text(CALLS)
    res = subprocess.run([sys.executable, "calls.py", str(tmp_path / "_torch_calls.so")], cwd=tmp_path, capture_output=True,
                         text=True, timeout=300, env=dict(os.environ, PYTHONPATH=""))
    assert res.returncode == 0, res.stderr
    assert res.stdout.strip() == str(want)
