"""Window prefill with a 16-bit output keeps the softmax weights as a 16-bit
value and its 16-bit residual, as with a 32-bit output: held to window_ref's
bound for value and residual (not to its wider one for weights rounded once),
and to fixed limits where a row sees few keys."""
import pytest
import torch

import window_ref as ref
from paged_kv_cache_tables_gb300 import paged_window_prefill_attention
from test_gpu_window import BF16, F16, F32, WINDOWS, Step

pytestmark = pytest.mark.gpu


def bound16(st, dtype):
    """(value, bound) of a 16-bit output.  The bound of a 32-bit output counts value and residual; a residual below the
    smallest subnormal adds half of that for each weight (the largest is at least 1), times sum |v| of at most c values
    of the largest |v|; the store adds half a step."""
    want, b32 = st.reference(F32)
    err = b32 + ref.TINY[dtype] / 2 * max(st.ctx) * st.v.double().abs().nan_to_num(0, 0, 0).max().cpu()
    return want, err + ref.rounding(want, err, dtype)


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("Hq,Hkv,d,dtype", [(8, 2, 128, BF16), (6, 2, 64, BF16), (4, 1, 128, F16), (16, 1, 64, F16)])
def test_value_and_residual(cuda_lib, window, sinks, Hq, Hkv, d, dtype):
    ctx, qn = [1, 1, 16, 129, 300, 63, 400, 1200, 700, 0, 64], [1, 1, 16, 129, 1, 62, 65, 130, 257, 0, 64]
    st = Step(ctx, qn, Hq, Hkv, d, dtype, window, sinks, seed=window % 89)
    got = st.prefill(dtype)
    ref.assert_within(got, *bound16(st, dtype), "window %d, sinks %d" % (window, sinks))
    assert st.status.item() == 0


@pytest.mark.parametrize("Hq,Hkv,d,dtype", [(32, 2, 64, BF16), (32, 2, 128, F16), (20, 4, 128, BF16)])
@pytest.mark.parametrize("window,sinks", [(300, 20), (40, 0)])
def test_value_and_residual_of_many_units(cuda_lib, Hq, Hkv, d, dtype, window, sinks):
    """More units than SMs, so that a CTA takes several, two query tiles each."""
    st = Step([700, 1400, 333, 900, 640, 0], [700, 650, 1, 512, 333, 0], Hq, Hkv, d, dtype, window, sinks)
    got = st.prefill(dtype)
    ref.assert_within(got, *bound16(st, dtype))
    assert torch.equal(got, st.prefill(dtype)) and st.status.item() == 0


@pytest.mark.parametrize("n", [2, 3, 5, 8, 16, 32])
@pytest.mark.parametrize("d,dtype", [(64, BF16), (128, BF16), (64, F16)])
def test_rows_that_see_few_keys(cuda_lib, n, d, dtype):
    """Windows and prompts of n keys, values N(0, 1): 2e-3, the limit of the causal kernels' outputs, and half an output
    step."""
    limit = lambda want: 2e-3 + torch.finfo(dtype).eps / 2 * (want.abs() + 2e-3)   # noqa: E731
    for st in (Step([700] * 4, [500] * 4, 8, 2, d, dtype, n, 0, seed=n), Step([n] * 64, [n] * 64, 8, 2, d, dtype, 64, 0, seed=n)):
        want, _ = st.reference(F32)
        ref.assert_within(st.prefill(dtype), want, limit(want), "%d keys" % n)


@pytest.mark.parametrize("chunks", [1, 40])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_equal_values_reproduce_themselves(cuda_lib, dtype, chunks):
    """Every value the same: the weighted mean is that value, off by less than the weights' 2^-14 before it is stored, so
    the store (half a step is 2^-9 or 2^-12 of it) gives its bits.  One query tile a unit, and two."""
    st = Step([300] * chunks, [200] * chunks, 8, 2, 128, dtype, 30, 2, poison=False)
    value = torch.tensor(1.1015625, dtype=dtype).item()
    st.v.fill_(value)
    assert (st.prefill(dtype) == value).all()
