"""Attention over 8 bits at the ends of the range of V's scales (2^-80 to 2^120,
those that a query sees within 2^100 of one another), and V's scales in the
softmax: tiles that hold the same values as other codes with other scales."""
import pytest
import torch

import quant_ref as qr
import window_ref as ref
from quant_ref import BF16, F16, F32, Step

pytestmark = pytest.mark.gpu
WHOLE = 2 ** 31 - 1
# one query tile a unit (keys in one CTA, or over several), two tiles, decode
CALLS = [([90], [40]), ([4090], [3]), ([700, 333, 900, 640, 0], [700, 1, 512, 333, 0]), ([90, 0, 333, 1700], [1, 1, 1, 1])]


def run(st, out_dtype):
    got = (st.decode if all(n == 1 for n in st.qn) else st.prefill)(out_dtype)
    assert st.status.item() == 0
    return got


def scaled(ctx, qn, d, low, high, odd):
    """Values of N(0, 1) times 2^3 as codes, V's scales 2^low to 2^high by block (or up to a fifth below those)."""
    st = Step(ctx, qn, 8, 2, d, BF16, WHOLE, 0, seed=d + len(ctx), poison=False)
    g = torch.Generator().manual_seed(d)
    st.vc = qr.encode(8 * torch.randn(st.vc.shape, generator=g, dtype=torch.float64))
    e = torch.where(torch.rand(st.scales.shape[:2], generator=g) < 0.5, low, high).float()
    b = torch.exp2(e) * (1 - 0.2 * odd * torch.rand(e.shape, generator=g))
    st.scales[..., 1] = b.clamp(min=2.0 ** low)
    st.v, st.dev["scales"] = st.vc.cuda().view(st.v.dtype), st.scales.cuda()
    return st


@pytest.mark.parametrize("ctx,qn", CALLS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("low,high", [(-80, -80), (-80, 20), (-60, 40), (20, 120), (120, 120)])
@pytest.mark.parametrize("odd", [0, 1])
def test_the_ends_of_the_range(cuda_lib, ctx, qn, d, low, high, odd):
    st = scaled(ctx, qn, d, low, high, odd)
    for out_dtype in (BF16, F32):
        ref.assert_within(run(st, out_dtype), *st.reference(out_dtype))


@pytest.mark.parametrize("ctx,qn", CALLS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_equal_values_under_different_scales(cuda_lib, ctx, qn, d, dtype):
    """1.125 in every tile, as 1.125 x 1, 2.25 x 0.5, 0.5625 x 2 or 1.5 x 0.75: the weighted mean is that value, off by less
    than 2^-13 of it before it is stored (value and residual 2^-16, the sums 2^-14, the scales' log2 and reciprocal 2^-18,
    exp2 2^-22), so the store, whose half a step is 2^-9 or 2^-12 of it, gives its bits."""
    st = Step(ctx, qn, 8, 2, d, dtype, WHOLE, 0, seed=d, poison=False)
    code = torch.tensor([0x39, 0x41, 0x31, 0x3C], dtype=torch.uint8)
    scale = torch.tensor([1.0, 0.5, 2.0, 0.75])
    assert (qr.decode(code) * scale == 1.125).all()
    kind = torch.randint(0, 4, st.scales.shape[:2], generator=torch.Generator().manual_seed(1))
    st.v = code[kind][..., None, None].expand(st.vc.shape).contiguous().cuda().view(st.v.dtype)
    st.dev["scales"][..., 1] = scale[kind].cuda()
    seen = torch.cat([torch.full((n,), c > 0) for c, n in zip(ctx, qn)]).cuda()
    got = run(st, dtype)
    assert (got[seen] == 1.125).all() and (got[~seen] == 0).all()
    got = run(st, F32)
    assert ((got[seen] - 1.125).abs() <= 1.125 * 2.0 ** -13).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("qn", [[1], [60]])
def test_a_large_scale_costs_no_bits_where_it_has_no_weight(cuda_lib, d, dtype, qn):
    """A block of V scales 2^40 times the others', at keys whose weight is below 2^-100.  A weight is off by half of fp16's
    smallest subnormal at most, 2^-25, where that of the largest y = score + log2 b is at least 2^7 and so the sum at least
    2^7 / b, b that position's scale: n 2^-32 times 448 b for n positions.  b is one of the others, so the bound is that
    without the block's factor."""
    st = Step([200], qn, 4, 1, d, dtype, WHOLE, 0, seed=5, poison=False, spread=0.0)
    blk = st.table[0, 3].item()
    st.q = (st.q.abs() * 8).to(dtype)      # away from that block's keys
    st.kc[blk] = 0x80 | 0x78               # -256
    st.dev["q"], st.k = st.q.cuda(), st.kc.cuda().view(st.k.dtype)
    bounds = [st.reference(t)[1] for t in (dtype, F32)]
    st.scales[blk, :, 1] *= 2.0 ** 40
    st.dev["scales"] = st.scales.cuda()
    for out_dtype, bound in zip((dtype, F32), bounds):
        ref.assert_within(run(st, out_dtype), st.reference(out_dtype)[0], bound)
