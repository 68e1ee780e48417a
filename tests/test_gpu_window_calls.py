"""Calls that the step's operators allow and their own tests do not make."""
import os
import shutil
import subprocess
import sys

import pytest
import torch

import window_ref as ref
from paged_kv_cache_tables_gb300 import _binding as B
from test_gpu_window import F16, F32, Step

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
