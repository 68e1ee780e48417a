"""The step of a serving loop as its operators are used together: tables from
the request lengths, queries and keys normed and rotated and appended, attention
over a window and the first tokens, blocks given back.  A prompt chunk for every
sequence, then decode steps replayed from one captured graph, with sequences
that finish and start again, in a pool that only holds the window: the tables are
checked exactly, every cached row against the rotation's formula, every output
against the definition on the cached rows."""
import math

import pytest
import torch

import window_ref as ref
from paged_kv_cache_tables_gb300 import (ROPE_YARN, paged_window_decode_attention, paged_window_prefill_attention,
                                         qk_rope_append, release_blocks, rope_frequencies, step_tables)
from test_gpu_rope import check as check_rotated

pytestmark = pytest.mark.gpu

WINDOW, SINKS, EPS = 40, 5, 1e-6
ROT = dict(scaling=ROPE_YARN, factor=16.0, original_context=4096, low=1.0, high=32.0)


class Loop:
    def __init__(self, S, Hq, Hkv, d, dtype, max_blocks, pool, capacity, chunk):
        self.S, self.Hq, self.Hkv, self.d, self.dtype = S, Hq, Hkv, d, dtype
        i32 = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")   # noqa: E731
        g = torch.Generator().manual_seed(S)
        free = torch.randperm(pool, generator=g).int()
        self.NB, self.capacity = pool, capacity
        self.lens, self.new, self.table = i32(S), i32(S), i32(S, max_blocks).fill_(-1)
        self.free, self.count, self.cu = free.cuda(), i32(1).fill_(pool), i32(S + 1)
        self.finished, self.status = i32(S), i32(1)
        self.slots = torch.zeros(capacity, dtype=torch.int64, device="cuda")
        self.pos = i32(capacity)
        self.qkv = torch.zeros(capacity, (Hq + 2 * Hkv) * d, dtype=dtype, device="cuda")
        self.q_out = torch.zeros(capacity, Hq, d, dtype=dtype, device="cuda")
        self.kc = torch.full((pool, Hkv, 16, d), float("nan"), dtype=dtype, device="cuda")
        self.vc = torch.full_like(self.kc, float("nan"))
        self.out = torch.zeros(capacity, Hq, d, dtype=torch.float32, device="cuda")
        self.wq = (1 + 0.1 * torch.randn(d, generator=g)).to(dtype).cuda()
        self.wk = (1 + 0.1 * torch.randn(d, generator=g)).to(dtype).cuda()
        self.freqs, self.m = rope_frequencies(d // 2, **ROT)
        # the same in plain Python
        self.g, self.chunk = g, chunk
        self.p_lens, self.p_table = [0] * S, self.table.tolist()
        self.p_free, self.p_count = free.tolist(), pool
        self.raw = [[] for _ in range(S)]     # each sequence's (k, v) rows as they came

    def parts(self):
        a, b = self.Hq * self.d, self.Hkv * self.d
        T = self.capacity
        return (self.qkv[:, :a].view(T, self.Hq, self.d), self.qkv[:, a:a + b].view(T, self.Hkv, self.d),
                self.qkv[:, a + b:].view(T, self.Hkv, self.d))

    def front(self):
        """Everything up to the attention."""
        q, k, v = self.parts()
        step_tables(self.lens, self.new, self.table, self.free, self.count, self.NB, self.lens, self.cu, self.slots,
                    self.pos, dev_status=self.status)
        qk_rope_append(self.q_out, q, k, v, self.pos, self.slots, self.freqs, self.kc, self.vc, interleaved=True,
                       mscale=self.m, q_weight=self.wq, k_weight=self.wk, eps=EPS, dev_status=self.status)

    def back(self):
        release_blocks(self.table, self.lens, self.free, self.count, self.NB, finished=self.finished, window=WINDOW,
                       num_sinks=SINKS, dev_status=self.status)

    def prefill(self):
        self.front()
        paged_window_prefill_attention(self.out, self.q_out, self.cu, self.chunk, self.kc, self.vc, self.table, self.lens,
                                       WINDOW, num_sinks=SINKS, dev_status=self.status)
        self.back()

    def decode(self):
        self.front()
        paged_window_decode_attention(self.out[:self.S], self.q_out[:self.S], self.kc, self.vc, self.table, self.lens, WINDOW,
                                      num_sinks=SINKS, dev_status=self.status)
        self.back()

    def fill(self, new, finished):
        """The step's inputs; returns what the caller has to hold against the outputs."""
        self.new.copy_(torch.tensor(new, dtype=torch.int32))
        self.finished.copy_(torch.tensor(finished, dtype=torch.int32))
        self.qkv.copy_(torch.randn(self.qkv.shape, generator=self.g).to(self.dtype))

    def verify(self, new, finished, expect_tokens):
        S = self.S
        before = list(self.p_lens)
        t, n, ctx, cu, slots, pos = ref.step_tables(before, new, self.p_table, self.p_free, self.p_count, self.capacity)
        assert self.status.item() == 0
        assert self.cu.tolist() == cu and self.slots.tolist() == slots and self.pos.tolist() == pos
        assert self.lens.tolist() == ctx and cu[-1] == expect_tokens
        q, k, v = (x.cpu() for x in self.parts())
        out = self.out.double().cpu()
        q_out = self.q_out.double().cpu()
        for s in range(S):
            a, b = cu[s], cu[s + 1]
            self.raw[s] += [(k[i], v[i]) for i in range(a, b)]
            if a == b:
                continue
            rows = torch.tensor(range(ctx[s]))
            table = torch.tensor(t[s])
            keys, values = ref.gathered(self.kc, table, ctx[s]), ref.gathered(self.vc, table, ctx[s])
            # the rows still held are the formula's, and the values' bits
            held = torch.tensor([p for p in rows.tolist() if t[s][p // 16] >= 0 and (p < SINKS or p > before[s] - WINDOW)])
            raw_k = torch.stack([self.raw[s][p][0] for p in held.tolist()])
            raw_v = torch.stack([self.raw[s][p][1] for p in held.tolist()])
            check_rotated(keys[held].to(self.dtype), raw_k, held, self.freqs, self.m, self.d // 2, True, self.wk, EPS, "k")
            assert torch.equal(values[held], raw_v.double())
            check_rotated(self.q_out[a:b].cpu(), q[a:b], torch.tensor(pos[a:b]), self.freqs, self.m, self.d // 2, True,
                          self.wq, EPS, "q")
            want, spread, mass = ref.attend(q_out[a:b], ctx[s] - new[s], keys, values, WINDOW, SINKS, 1 / math.sqrt(self.d))
            ref.assert_within(out[a:b], want, ref.attention_bound(want, spread, mass, self.d, 1 / math.sqrt(self.d),
                                                                  torch.float32), "sequence %d" % s)
        self.p_lens = ctx
        t, self.p_free, self.p_count = ref.release(t, ctx, finished, WINDOW, SINKS, self.p_free, n, self.NB)
        self.p_table = t
        assert self.table.tolist() == t and self.count.item() == self.p_count
        assert self.free.tolist()[:self.p_count] == self.p_free[:self.p_count]
        # a finished sequence's place starts again empty
        for s in range(S):
            if finished[s]:
                self.p_lens[s], self.raw[s] = 0, []
        self.lens.masked_fill_(self.finished != 0, 0)


@pytest.mark.parametrize("S,Hq,Hkv,d,dtype", [(6, 8, 2, 64, torch.bfloat16), (5, 4, 4, 128, torch.float16)])
def test_prefill_then_decode_steps_from_a_graph(cuda_lib, S, Hq, Hkv, d, dtype):
    loop = Loop(S, Hq, Hkv, d, dtype, max_blocks=16, pool=S * 10, capacity=200, chunk=60)
    idle = [0] * S
    # prompts in two chunks, of uneven lengths, one of them a single token
    for new in ([60, 1, 33, 17, 16, 48][:S], [20, 40, 0, 31, 60, 2][:S]):
        loop.fill(new, idle)
        loop.prefill()
        loop.verify(new, idle, sum(new))
    # decode: captured once, replayed; a graph of a fixed capacity
    one = [1] * S
    loop.fill(one, idle)
    loop.decode()
    loop.verify(one, idle, S)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        loop.decode()
    torch.cuda.current_stream().wait_stream(side)
    for step in range(45):
        finished = [int(step in (9, 30) and s == step % S) for s in range(S)]
        loop.fill(one, finished)
        graph.replay()
        loop.verify(one, finished, S)
    assert max(loop.p_lens) > WINDOW + SINKS + 32 and loop.p_count >= S * 10 - S * 6


def test_a_pool_that_runs_out_takes_nothing(cuda_lib):
    """The step that does not fit leaves tables, list and cache alone, and the next one that fits goes on."""
    loop = Loop(3, 4, 1, 64, torch.bfloat16, max_blocks=16, pool=6, capacity=100, chunk=60)
    loop.fill([40, 30, 10], [0, 0, 0])       # 3 + 2 + 1 blocks
    loop.prefill()
    loop.verify([40, 30, 10], [0, 0, 0], 80)
    cache = loop.kc.clone()
    loop.fill([1, 20, 10], [0, 0, 0])
    loop.front()
    assert loop.status.item() == 64 and loop.lens.tolist() == [40, 30, 10] and loop.cu.tolist() == [0] * 4
    assert (loop.slots == -1).all() and loop.table.tolist() == loop.p_table and loop.count.item() == 0
    assert torch.equal(loop.kc.nan_to_num(7), cache.nan_to_num(7))
    loop.status.zero_()
    loop.fill([8, 2, 6], [0, 1, 0])          # fits the open blocks; the second finishes
    loop.prefill()
    loop.verify([8, 2, 6], [0, 1, 0], 16)
    assert loop.count.item() == 2
    loop.fill([1, 16, 0], [0, 0, 0])         # its place takes a new prompt
    loop.prefill()
    loop.verify([1, 16, 0], [0, 0, 0], 17)
    assert loop.count.item() == 0
