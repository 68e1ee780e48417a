"""Prefill over 8 bits keeps the softmax weights as an fp16 value and its fp16
residual whatever the output's type is: a 16-bit output is the 32-bit one rounded,
and lies within the bound of value and residual (quant_ref's for a bf16 output
leaves room for weights rounded once)."""
import pytest
import torch

import window_ref as ref
from quant_ref import BF16, F16, F32, Step

pytestmark = pytest.mark.gpu
WHOLE = 2 ** 31 - 1


def bound16(st, dtype):
    """(value, bound): a 32-bit output's bound, and half a step of dtype for the store."""
    want, err = st.reference(F32)
    return want, err + ref.rounding(want, err, dtype)


# one query tile a unit, its keys in one CTA or over several; two query tiles, one unit a CTA or more
SHAPES = [([129], [129]), ([9000], [3]), ([300, 2600, 0, 128], [32, 64, 0, 128]), ([500, 40, 129, 1000], [1, 7, 128, 130]),
          ([700, 1400, 333, 900, 640, 0], [700, 650, 1, 512, 333, 0])]


@pytest.mark.parametrize("ctx,qn", SHAPES)
@pytest.mark.parametrize("window,sinks", [(WHOLE, 0), (40, 3)])
@pytest.mark.parametrize("Hq,Hkv,d,dtype", [(8, 2, 128, BF16), (16, 4, 64, BF16), (32, 2, 128, BF16), (5, 1, 64, F16), (8, 2, 128, F16)])
def test_a_16_bit_output_is_the_32_bit_one_rounded(cuda_lib, ctx, qn, window, sinks, Hq, Hkv, d, dtype):
    st = Step(ctx, qn, Hq, Hkv, d, dtype, window, sinks, seed=sum(qn) % 97)
    got = st.prefill(dtype)
    ref.assert_within(got, *bound16(st, dtype))
    assert torch.equal(got, st.prefill(F32).to(dtype)) and st.status.item() == 0


@pytest.mark.parametrize("n", [2, 3, 5, 16])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_that_see_few_keys(cuda_lib, n, d):
    """Where a weight's rounding shows most: a few keys, values of very different magnitude."""
    for st in (Step([700] * 4, [500] * 4, 8, 2, d, BF16, n, 0, seed=n, spread=3.0),
               Step([n] * 64, [n] * 64, 8, 2, d, BF16, 64, 0, seed=n, spread=3.0)):
        got = st.prefill(BF16)
        ref.assert_within(got, *bound16(st, BF16), "%d keys" % n)
        assert torch.equal(got, st.prefill(F32).to(BF16))


@pytest.mark.parametrize("ctx,qn", SHAPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_scores_that_rise_all_along(cuda_lib, ctx, qn, d, dtype):
    """Each page's scores 2^8 or more above the page's before, so that every part of the keys moves the maximum on and its
    weights are made, and stored, twice; the same bits at every call."""
    st = Step(ctx, qn, 8, 2, d, dtype, WHOLE, 0, seed=9, poison=False)
    st.kc.zero_()
    st.kc[..., 3] = 0x38                     # 1 in one dimension
    st.q[..., 3] = 1
    for s, c in enumerate(ctx):
        nb = -(-c // 16)
        st.scales[st.table[s].long()[:nb], :, 0] = (5.6 * d ** 0.5 * (torch.arange(nb) + 1.0)).view(nb, 1)   # 8.08 in log2
    st.k, st.dev["scales"], st.dev["q"] = st.kc.cuda().view(st.k.dtype), st.scales.cuda(), st.q.cuda()
    got = st.prefill(dtype)
    ref.assert_within(got, *bound16(st, dtype))
    for _ in range(3):
        assert torch.equal(st.prefill(dtype), got)
    assert st.status.item() == 0
