"""Attention over 8 bits where the factor between a product of codes and its
score is too small for fp32: queries of zeros or next to it, tiles of zeros (which
append gives the scale 2^-60), small scales.  The scores are then 0, or so near
it that the weights are equal, and hidden positions stay hidden."""
import pytest
import torch

import window_ref as ref
from quant_ref import BF16, F16, F32, Step, assert_stored
from paged_kv_cache_tables_gb300 import kv_append_e4m3

pytestmark = pytest.mark.gpu
WHOLE = 2 ** 31 - 1
TYPES = [(BF16, BF16), (F16, F16), (BF16, F32), (F16, F32)]
# one query tile a unit (keys in one CTA, or over several), two tiles, decode
CALLS = [([90], [40]), ([4090], [3]), ([700, 333, 900, 640, 0], [700, 1, 512, 333, 0]), ([90, 0, 333, 7], [1, 1, 1, 1])]


def step(ctx, qn, d, dtype, window, sinks, k_scale, zero_keys, zero_rows, magnitude=1.0):
    st = Step(ctx, qn, 16, 4, d, dtype, window, sinks, seed=len(ctx))
    if zero_keys:
        st.kc[st.kc != 127] = 0
        st.k = st.kc.cuda().view(st.k.dtype)
    st.scales[..., 0] = torch.where(st.scales[..., 0].isnan(), st.scales[..., 0], torch.tensor(k_scale))
    st.dev["scales"] = st.scales.cuda()
    st.q = (st.q.float() * magnitude).to(dtype)
    if zero_rows:
        st.q[::zero_rows, 1::2] = 0
    st.dev["q"] = st.q.cuda()
    return st


def check(st, out_dtype, **kw):
    want, bound = st.reference(out_dtype)
    got = (st.decode if all(n == 1 for n in st.qn) else st.prefill)(out_dtype, **kw)
    ref.assert_within(got, want, bound)
    assert st.status.item() == 0


@pytest.mark.parametrize("ctx,qn", CALLS)
@pytest.mark.parametrize("window,sinks", [(WHOLE, 0), (33, 5)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype,out_dtype", TYPES)
def test_zero_queries_and_zero_keys(cuda_lib, ctx, qn, window, sinks, d, dtype, out_dtype):
    """Rows of zeros among others, and all rows, over keys of zeros and others."""
    for zero_keys, zero_rows in ((True, 1), (True, 2), (False, 2)):
        check(step(ctx, qn, d, dtype, window, sinks, 2.0 ** (-60 if zero_keys else -24), zero_keys, zero_rows), out_dtype)


@pytest.mark.parametrize("ctx,qn", CALLS)
@pytest.mark.parametrize("magnitude,k_scale", [(2.0 ** -118, 2.0 ** -20), (2.0 ** -124, 2.0 ** -60), (2.0 ** -124, 1.0), (2.0 ** -124, 2.0 ** 110),
                                               (1.0, 2.0 ** -100)])
def test_queries_next_to_zero(cuda_lib, ctx, qn, magnitude, k_scale):
    for out_dtype in (BF16, F32):
        check(step(ctx, qn, 128, BF16, 33, 5, k_scale, False, 3, magnitude), out_dtype)


@pytest.mark.parametrize("ctx,qn", CALLS)
def test_a_tiny_scale(cuda_lib, ctx, qn):
    for dtype in (BF16, F16):
        st = step(ctx, qn, 64, dtype, 33, 5, 2.0 ** -30, False, 0)
        st.scale = 1e-35
        check(st, F32, scale=st.scale)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [64, 128])
def test_a_step_on_zeros(cuda_lib, d, dtype):
    """A warm-up step: keys, values and queries of zeros appended and attended to give zeros; values that are not zeros
    their mean."""
    for ctx, qn in CALLS:
        st = Step(ctx, qn, 16, 4, d, dtype, WHOLE, 0, poison=False)
        st.dev["q"].zero_()
        for values in (0.0, 1.0):
            T = sum(ctx)
            slots = torch.cat([st.table[s].long()[torch.arange(c) // 16] * 16 + torch.arange(c) % 16 for s, c in enumerate(ctx)])
            rows = torch.zeros(T, 4, d, dtype=dtype, device="cuda")
            kv_append_e4m3(rows, rows + values, slots.cuda(), st.k, st.v, st.dev["scales"], dev_status=st.status)
            got = (st.decode if all(n == 1 for n in qn) else st.prefill)(dtype)
            seen = torch.cat([torch.full((n,), c > 0) for c, n in zip(ctx, qn)]).cuda()
            assert (got[seen] == values).all() and (got[~seen] == 0).all() and st.status.item() == 0
