"""Attention over 8 bits multiplies K's codes by a query's 8-bit terms: queries
with one element far above the others, which meets keys of zero, so that the
scores come from the others.  Prefill takes elements down to 2^-13.8 of a row's
largest exactly and others to within 2^-21.8 of it (fp16: 2^-24.8); decode down to
2^-13 and within 2^-21 of a head's (fp16: 2^-14 and 2^-25)."""
import pytest
import torch

import quant_ref as qr
import window_ref as ref
from quant_ref import BF16, F16, F32, Step

pytestmark = pytest.mark.gpu
WHOLE = 2 ** 31 - 1
# one query tile a unit (keys in one CTA, or over several), two tiles, decode
CALLS = [([90], [40]), ([4090], [3]), ([700, 333, 900, 640, 0], [700, 1, 512, 333, 0]), ([90, 0, 333, 1700], [1, 1, 1, 1])]


def outlier(ctx, qn, d, dtype, largest, least):
    """Elements of N(0, 1), at least `least` in magnitude, and one of `largest` where K is zero."""
    st = Step(ctx, qn, 8, 2, d, dtype, WHOLE, 0, seed=d + len(ctx))
    st.q = torch.where(st.q.abs() < least, torch.copysign(st.q.abs().float() + least, st.q.float()).to(dtype), st.q)
    st.q[..., 5] = largest
    st.dev["q"] = st.q.cuda()
    st.kc[..., 5][st.kc[..., 5] != 127] = 0
    st.k = st.kc.cuda().view(st.k.dtype)
    return st


def run(st, out_dtype):
    got = (st.decode if all(n == 1 for n in st.qn) else st.prefill)(out_dtype)
    assert st.status.item() == 0
    return got


@pytest.mark.parametrize("ctx,qn", CALLS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype,out_dtype", [(BF16, BF16), (F16, F16), (BF16, F32), (F16, F32)])
def test_elements_down_to_2_13_are_exact(cuda_lib, ctx, qn, d, dtype, out_dtype):
    """2,000 beside magnitudes from 0.25 (2^-12.97 of it): no more than the bound of any other query."""
    st = outlier(ctx, qn, d, dtype, 2000.0, 0.25)
    ref.assert_within(run(st, out_dtype), *st.reference(out_dtype))


@pytest.mark.parametrize("ctx,qn", CALLS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype,part", [(BF16, 2.0 ** -21), (F16, 2.0 ** -24.8)])
@pytest.mark.parametrize("largest", [2000.0, 60000.0])
def test_smaller_elements(cuda_lib, ctx, qn, d, dtype, part, largest):
    """Elements of any magnitude: a score is off by `part` of the largest times scale sum |k| at most, besides."""
    st = outlier(ctx, qn, d, dtype, largest, 0.0)
    got, at = run(st, F32), 0
    for s, (c, n) in enumerate(zip(ctx, qn)):
        if c == 0 or n == 0:
            at += n
            continue
        k, v = (qr.gathered(x, st.scales[..., i], st.table[s], c) for i, x in enumerate((st.kc, st.vc)))
        o, spread, mass = ref.attend(st.q[at:at + n].double(), c - n, k, v, WHOLE, 0, st.scale)
        most = k.nan_to_num(0.0).abs().sum(-1).amax(0).repeat_interleave(4).view(1, 8, 1)   # of each query head's KV head
        largest_v = qr.CODE_MAX * st.scales[st.table[s].long()[:-(-c // 16)], :, 1].max().item()
        # in units of the accumulation's roundings, d 2^-23 of sum |q_i k_i|
        off = largest * part * most / (d * 2.0 ** -23)
        ref.assert_within(got[at:at + n], o, qr.attention_bound(o, spread, mass + off, d, st.scale, F32, largest_v, c))
        at += n
