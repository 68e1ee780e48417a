"""Calls that the step's operators allow and their own tests do not make."""
import os
import shutil
import subprocess
import sys

import pytest
import torch

import window_ref as ref
from paged_kv_cache_tables_gb300 import _binding as B
from paged_kv_cache_tables_gb300 import (paged_decode_attention, paged_window_decode_attention,
                                         paged_window_prefill_attention, step_tables)
from test_gpu_window import BF16, F16, F32, Step
from test_gpu_window_step import SINKS, WINDOW, Loop

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("out_dtype", [F16, F32])
@pytest.mark.parametrize("rows,max_q", [(129, 128), (130, 129), (65, 1)])
def test_a_chunk_longer_than_max_q_len_is_skipped_and_reported(cuda_lib, rows, max_q, out_dtype):
    """Lengths built on the device can outgrow the host's max_q_len: no row of such a chunk is written."""
    st = Step([300, 200, 90], [rows, 1, min(60, max_q)], 4, 1, 64, F16, 64, 4)
    want, bound = st.reference(out_dtype, True)
    got = st.prefill(out_dtype, max_q=max_q)
    assert torch.isnan(got[:rows]).all() and st.status.item() == B.DEV_BAD_CHUNK
    ref.assert_within(got[rows:], want[rows:], bound[rows:])


@pytest.mark.parametrize("S", [3, 200, 300])
def test_step_tables_straight_before_decode_attention(cuda_lib, S):
    """Plain decode reads context_lens to plan before it waits for the work ahead of it: here the launch that writes them,
    in place, every step another length, captured and replayed."""
    MB, NB = 12, S * 12
    g = torch.Generator().manual_seed(S)
    k = torch.randn(NB, 2, 16, 64, generator=g).to(BF16).cuda()
    v = torch.randn(NB, 2, 16, 64, generator=g).to(BF16).cuda()
    q = torch.randn(S, 4, 64, generator=g).to(BF16)
    lens = [(7 * s) % 60 for s in range(S)]
    table = [list(range(s * 12, s * 12 + -(-n // 16))) + [-1] * (MB - -(-n // 16)) for s, n in enumerate(lens)]
    held = {b for r in table for b in r}
    free = [b for b in torch.randperm(NB, generator=g).tolist() if b not in held]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")   # noqa: E731
    d_lens, d_table, d_free, d_count = i32(lens), i32(table), i32(free), i32([len(free)])
    new = i32([1 + s % 2 for s in range(S)])
    T = int(new.sum())
    cu, pos, status = i32([0] * (S + 1)), i32([0] * T), i32([0])
    slots = torch.zeros(T, dtype=torch.int64, device="cuda")
    steps = 40
    out = torch.full((steps, S, 4, 64), float("nan"), device="cuda")
    now = torch.zeros(S, 4, 64, device="cuda")
    dq = q.cuda()
    work = torch.empty(B.decode_workspace_size(S, 4, 2, 64), dtype=torch.uint8, device="cuda")

    def step():
        step_tables(d_lens, new, d_table, d_free, d_count, NB, d_lens, cu, slots, pos, dev_status=status)
        paged_decode_attention(now, dq, k, v, d_table, d_lens, workspace=work, dev_status=status)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    for i in range(steps):
        graph.replay() if i % 2 else step()
        out[i] = now
    count, fresh = len(free), new.tolist()
    for i in range(steps):
        table, count, lens, _, _, _ = ref.step_tables(lens, fresh, table, free, count, T)
        if i % 13 and i != steps - 1:
            continue
        for s in range(0, S, 1 + S // 60):
            keys, values = ref.gathered(k, torch.tensor(table[s]), lens[s]), ref.gathered(v, torch.tensor(table[s]), lens[s])
            want, spread, mass = ref.attend(q[s:s + 1].double(), lens[s] - 1, keys, values, 10 ** 6, 0, 0.125)
            ref.assert_within(out[i, s:s + 1], want, ref.attention_bound(want, spread, mass, 64, 0.125, F32), (i, s))
    assert status.item() == 0 and d_lens.tolist() == lens and d_table.tolist() == table


@pytest.mark.parametrize("d,dtype", [(64, BF16), (128, F16)])
def test_a_step_of_chunks_and_decodes(cuda_lib, d, dtype):
    """One batch, its tables built once: the first P sequences are chunks, the others decode a token each, on slices of the
    step's arrays."""
    loop = Loop(6, 8, 2, d, dtype, max_blocks=16, pool=60, capacity=200, chunk=60)
    idle = [0] * 6
    loop.fill([1, 30, 0, 17, 16, 48], idle)
    loop.prefill()
    loop.verify([1, 30, 0, 17, 16, 48], idle, 112)
    for P, chunks in ((3, [60, 5, 33]), (1, [59]), (5, [1, 2, 17, 1, 40])):
        new, Tp = chunks + [1] * (6 - P), sum(chunks)
        T = Tp + 6 - P
        loop.fill(new, idle)
        loop.front()
        paged_window_prefill_attention(loop.out[:Tp], loop.q_out[:Tp], loop.cu[:P + 1], 60, loop.kc, loop.vc, loop.table[:P],
                                       loop.lens[:P], WINDOW, num_sinks=SINKS, dev_status=loop.status)
        paged_window_decode_attention(loop.out[Tp:T], loop.q_out[Tp:T], loop.kc, loop.vc, loop.table[P:], loop.lens[P:], WINDOW,
                                      num_sinks=SINKS, dev_status=loop.status)
        loop.back()
        loop.verify(new, idle, T)


FAKE = """
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

CALLS = """
import importlib.util, sys, torch
spec = importlib.util.spec_from_file_location("_torch_calls", sys.argv[1])
m = importlib.util.module_from_spec(spec)
spec.loader.exec_module(m)
x = torch.zeros(2, 2, 64, dtype=torch.float16, device="cuda")
c = torch.zeros(4, 2, 16, 64, dtype=torch.float16, device="cuda")
i = torch.zeros(2, dtype=torch.int32, device="cuda")
t = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
cu, f = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(32, dtype=torch.int64, device="cuda")
held = [m.window_decode(x, x, c, c, t, i, 16, 0, None, None, None),
        m.window_prefill(x, x, cu, 1, c, c, t, i, 16, 0, None, None, None),
        m.qk_rope(x, x, x, x, i, f, False, 1.0, None, None, 0.0, None),
        m.qk_rope_append(x, x, x, x, i, i.long(), f, c, c, False, 1.0, None, None, 0.0, None, None),
        m.step_tables(i, i, t, i, i[:1], 4, i, cu, i.long(), i, None, None, None),
        m.release_blocks(t, i, i, i[:1], 4, None, 0, 0, None, None, None)]
assert held == [0] * 6, held
"""


def test_other_threads_run_while_a_call_is_made(cuda_lib, tmp_path):
    """A launch can wait for room in the stream's queue: as with the entry points that ctypes calls, the interpreter is
    free meanwhile.  The module runs against a library whose entry points return whether it is held."""
    (tmp_path / "fake.c").write_text(FAKE)
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(tmp_path / "libpkv.so"), str(tmp_path / "fake.c")], check=True)
    shutil.copy(B.CALLS_PATH, tmp_path / "_torch_calls.so")
    (tmp_path / "calls.py").write_text(CALLS)
    res = subprocess.run([sys.executable, "calls.py", str(tmp_path / "_torch_calls.so")], cwd=tmp_path, capture_output=True,
                         text=True, timeout=300, env=dict(os.environ, PYTHONPATH=""))
    assert res.returncode == 0, res.stderr
