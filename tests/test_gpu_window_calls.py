"""Calls that the step's operators allow and their own tests do not make."""
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
