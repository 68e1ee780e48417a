"""Attention over the cache held in 8 bits (decode and prefill) against the
definition in 64 bits, with the bounds derived in quant_ref and window_ref."""
import pytest
import torch

import window_ref as ref
from quant_ref import BF16, F16, F32, Step, assert_stored
from paged_kv_cache_tables_gb300 import PkvError

pytestmark = pytest.mark.gpu
BAD_BLOCK, BAD_CONTEXT, BAD_CHUNK = 1, 2, 16

WHOLE = 2 ** 31 - 1
WINDOWS = [(1, 0), (1, 1), (2, 0), (16, 0), (17, 4), (31, 16), (33, 17), (128, 0), (129, 4), (200, 100), (1000, 128),
           (700, 1), (100000, 0), (WHOLE, WHOLE), (3, WHOLE), (WHOLE, 0)]
CONTEXTS = [0, 1, 2, 15, 16, 17, 33, 127, 128, 129, 256, 300, 511, 777, 1100, 1999]
TYPES = [(BF16, BF16), (F16, F16), (BF16, F32), (F16, F32)]


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("Hq,Hkv,d,dtype,out_dtype", [(8, 2, 64, F16, F32), (4, 1, 128, BF16, F32), (8, 2, 128, BF16, BF16)])
def test_decode(cuda_lib, window, sinks, Hq, Hkv, d, dtype, out_dtype):
    st = Step(CONTEXTS, [1] * len(CONTEXTS), Hq, Hkv, d, dtype, window, sinks, seed=window % 97)
    got = st.decode(out_dtype)
    want, bound = st.reference(out_dtype)
    ref.assert_within(got, want, bound, "window %d, sinks %d" % (window, sinks))
    assert (got[0] == 0).all() and st.status.item() == 0


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (6, 2), (20, 4), (16, 2), (9, 1), (16, 1), (32, 2), (16, 16), (15, 5)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype,out_dtype", TYPES)
def test_decode_head_layouts(cuda_lib, Hq, Hkv, d, dtype, out_dtype):
    st = Step([700, 5, 0, 64], [1] * 4, Hq, Hkv, d, dtype, 300, 20, seed=Hq, heavy=True, odd_scales=Hq % 2 == 0)
    want, bound = st.reference(out_dtype)
    ref.assert_within(st.decode(out_dtype), want, bound)
    assert st.status.item() == 0


@pytest.mark.parametrize("S,hi,window", [(1, 40000, WHOLE), (1, 9000, 100), (2, 2900, WHOLE), (5, 9000, 9000), (64, 300, 128),
                                         (160, 200, 64), (700, 90, 40)])
def test_decode_every_split(cuda_lib, S, hi, window):
    """From one sequence (a range over a whole cluster) to many (a CTA a range); the same bits at every call."""
    ctx = [max(1, hi - 37 * i % hi) for i in range(S)]
    st = Step(ctx, [1] * S, 4, 2, 128, BF16, window, 4, seed=S)
    got = st.decode(F32)
    want, bound = st.reference(F32)
    ref.assert_within(got, want, bound)
    for _ in range(3):
        assert torch.equal(st.decode(F32), got)


@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 0), (33, 17), (200, 100), (700, 1), (WHOLE, 0)])
@pytest.mark.parametrize("Hq,Hkv,d,dtype,out_dtype", [(4, 4, 64, F16, F32), (32, 4, 128, BF16, F32), (12, 4, 128, F16, F16),
                                                      (20, 4, 64, BF16, BF16), (64, 4, 128, BF16, BF16)])
def test_decode_many_ranges(cuda_lib, window, sinks, Hq, Hkv, d, dtype, out_dtype):
    """More ranges than SMs: contexts from none to a few hundred tokens beside long ones, in one batch."""
    ctx = [CONTEXTS[i % len(CONTEXTS)] if i % 3 else (i * 37) % 400 for i in range(100)]
    st = Step(ctx, [1] * len(ctx), Hq, Hkv, d, dtype, window, sinks, seed=window % 83)
    got = st.decode(out_dtype)
    want, bound = st.reference(out_dtype)
    ref.assert_within(got, want, bound, "window %d, sinks %d" % (window, sinks))
    assert st.status.item() == 0
    for _ in range(2):
        assert torch.equal(st.decode(out_dtype), got)


PREFILLS = [([1, 16, 17, 300], [1, 16, 17, 300]), ([500, 40, 129, 1000], [1, 7, 128, 130]), ([1500], [257]),
            ([64, 0, 333, 90, 16], [0, 0, 333, 45, 1])]


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("ctx,qn", PREFILLS)
@pytest.mark.parametrize("Hq,Hkv,d,dtype,out_dtype", [(8, 2, 64, F16, F16), (4, 1, 128, BF16, BF16), (6, 2, 128, F16, F32)])
def test_prefill(cuda_lib, window, sinks, ctx, qn, Hq, Hkv, d, dtype, out_dtype):
    st = Step(ctx, qn, Hq, Hkv, d, dtype, window, sinks, seed=window % 89)
    want, bound = st.reference(out_dtype)
    ref.assert_within(st.prefill(out_dtype), want, bound, "window %d, sinks %d" % (window, sinks))
    assert st.status.item() == 0


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (20, 4), (16, 2), (9, 1), (16, 1), (32, 2), (5, 5), (15, 5), (7, 1)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype,out_dtype", TYPES)
def test_prefill_head_layouts(cuda_lib, Hq, Hkv, d, dtype, out_dtype):
    st = Step([400, 77, 129], [139, 77, 2], Hq, Hkv, d, dtype, 150, 20, seed=Hq, heavy=True, odd_scales=Hq % 2 == 0)
    want, bound = st.reference(out_dtype)
    ref.assert_within(st.prefill(out_dtype), want, bound)
    assert st.status.item() == 0


@pytest.mark.parametrize("dtype,out_dtype", TYPES)
@pytest.mark.parametrize("d,window,sinks", [(64, WHOLE, 0), (128, WHOLE, 0), (128, 300, 20), (64, 40, 0)])
def test_prefill_of_many_units(cuda_lib, dtype, out_dtype, d, window, sinks):
    """More units of work than SMs; the same bits at every call."""
    st = Step([700, 1400, 333, 900, 640, 0], [700, 650, 1, 512, 333, 0], 32, 2, d, dtype, window, sinks)
    got = st.prefill(out_dtype)
    ref.assert_within(got, *st.reference(out_dtype))
    assert torch.equal(got, st.prefill(out_dtype)) and st.status.item() == 0


@pytest.mark.parametrize("ctx,qn", [([9000], [3]), ([5000], [200]), ([4097, 1, 40], [1, 1, 33]), ([300, 2600, 0, 128], [32, 64, 0, 128]),
                                    ([129], [129]), ([1300, 700], [64, 64])])
@pytest.mark.parametrize("window,sinks", [(WHOLE, 0), (700, 33), (20, 0)])
@pytest.mark.parametrize("Hq,Hkv,d,dtype,out_dtype", [(4, 1, 128, BF16, BF16), (10, 2, 64, F16, F32), (8, 1, 128, F16, F16),
                                                      (3, 1, 64, BF16, F32)])
def test_prefill_of_few_rows(cuda_lib, ctx, qn, window, sinks, Hq, Hkv, d, dtype, out_dtype):
    """A unit's keys over several CTAs, some without a key; the same bits at every call."""
    st = Step(ctx, qn, Hq, Hkv, d, dtype, window, sinks, seed=ctx[0] % 89, heavy=d == 64)
    want, bound = st.reference(out_dtype)
    got = st.prefill(out_dtype)
    ref.assert_within(got, want, bound)
    assert st.status.item() == 0 and torch.equal(got, st.prefill(out_dtype))


@pytest.mark.parametrize("chunks,extra", [(3, 0), (32, 300), (33, 0), (60, 77), (5, 2 ** 31 - 1 - 194)])
@pytest.mark.parametrize("Hq,Hkv,d,out_dtype", [(16, 16, 64, BF16), (30, 10, 128, F32)])
def test_prefill_takes_every_unit_once(cuda_lib, chunks, extra, Hq, Hkv, d, out_dtype):
    """Chunks of no row, of one and of many, behind contexts of their own, with a max_q_len that none reaches; some that
    are refused among them: the rows of those stay as they were, every other has its output."""
    qn = [[170, 0, 1, 64, 65, 130][i % 6] + (i if i % 6 == 0 else 0) for i in range(chunks)]
    ctx = [n + [900, 3, 400, 0, 64, 31][(i // 2) % 6] for i, n in enumerate(qn)]
    st = Step(ctx, qn, Hq, Hkv, d, BF16, 500, 3, seed=chunks, poison=False)
    want, bound = st.reference(out_dtype)
    got = st.prefill(out_dtype, max_q=max(qn) + extra)
    ref.assert_within(got, want, bound)
    assert st.status.item() == 0 and torch.equal(got, st.prefill(out_dtype))
    st.dev["ctx"][0] = qn[0] - 1              # fewer positions than rows
    st.dev["ctx"][2] = st.dev["table"].shape[1] * 16 + 1
    got = st.prefill(out_dtype, max_q=max(qn) + extra).cpu()
    rows = torch.arange(sum(qn))
    bad = (rows < qn[0]) | (rows == qn[0])    # chunk 2 is the row behind chunk 0's
    assert got[bad].isnan().all() and st.status.item() == BAD_CHUNK | BAD_CONTEXT
    ref.assert_within(got[~bad], want[~bad], bound[~bad])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("spread", [3.0, 10.0])
def test_scales_far_apart(cuda_lib, d, spread):
    """Values whose magnitude differs by many binades from token to token: the softmax decides which of them show."""
    for dtype, out_dtype in TYPES:
        st = Step([300, 700, 40], [1] * 3, 8, 2, d, dtype, WHOLE, 0, seed=3, spread=spread)
        assert_stored(st.decode(out_dtype), *st.reference(out_dtype))
        st = Step([300, 700, 40], [100, 3, 40], 8, 2, d, dtype, WHOLE, 0, seed=4, spread=spread)
        assert_stored(st.prefill(out_dtype), *st.reference(out_dtype))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_large_scale_at_a_hidden_weight(cuda_lib, d, dtype):
    """A block whose values are 2^40 times the others', at keys that the softmax gives a weight below 2^-100: its scale
    must not cost the others their precision."""
    for qn in ([1], [60]):
        st = Step([200], qn, 4, 1, d, dtype, WHOLE, 0, seed=5, poison=False, spread=0.0)
        blk = st.table[0, 3].item()
        for s in (st.scales, st.dev["scales"]):
            s[blk, :, 1] *= 2.0 ** 40
        # keys of that block point away from the queries: score below -100
        st.q = (st.q.abs() * 8).to(dtype)
        st.dev["q"] = st.q.cuda()
        st.kc[blk] = 0x80 | 0x78   # -256
        st.k = st.kc.cuda().view(torch.float8_e4m3fn)
        for out_dtype in (dtype, F32):
            want, bound = st.reference(out_dtype)
            got = st.decode(out_dtype) if qn == [1] else st.prefill(out_dtype)
            # (the bound's term for subnormal weights counts that block's values too; the others' are below 8)
            ref.assert_within(got, want, bound.clamp(max=0.05))


def test_extreme_queries_and_scales(cuda_lib):
    """Queries of a few hundred binades' range in bf16, key scales that bring the scores back."""
    for mag in (2.0 ** 60, 2.0 ** -60):
        for qn in ([1, 1], [20, 1]):
            st = Step([100, 40], qn, 4, 2, 64, BF16, WHOLE, 0, seed=6, poison=False)
            st.q = st.q * mag
            st.dev["q"] = st.q.cuda()
            for s in (st.scales, st.dev["scales"]):
                s[..., 0] /= mag
            got = st.decode(F32) if qn == [1, 1] else st.prefill(F32)
            ref.assert_within(got, *st.reference(F32))


def test_rows_within_a_query_differ(cuda_lib):
    """Heads of one group, and rows of one tile, with queries of very different magnitude; a row of zeros."""
    for qn in ([1], [40]):
        st = Step([90], qn, 8, 1, 128, BF16, WHOLE, 0, seed=7, poison=False)
        st.q[:, 0] *= 1e-6
        st.q[:, 1] *= 30
        st.q[:, 2] = 0
        st.q[:, 3, ::2] *= 1e-5
        st.dev["q"] = st.q.cuda()
        got = st.decode(F32) if qn == [1] else st.prefill(F32)
        ref.assert_within(got, *st.reference(F32))


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_equal_values_reproduce_themselves(cuda_lib, dtype):
    """Every value the same code and scale: the weighted mean is that value, off by at most the weights' 2^-11 before it is
    stored (2^-9 or, with the residual, far below 2^-12 of it): its bits, or for bf16 half a step away."""
    for chunks in (1, 40):
        st = Step([300] * chunks, [200] * chunks, 8, 2, 128, dtype, 30, 2, poison=False)
        st.v.view(torch.uint8).fill_(0x39)
        st.dev["scales"][..., 1] = 1.0
        for got in (st.prefill(dtype), ):
            assert (got == 1.125).all()


def test_reports(cuda_lib):
    """Bad table entries, lengths and chunks set their status bit, and the other sequences are unharmed."""
    st = Step([64, 40, 100], [1, 1, 1], 4, 2, 64, BF16, WHOLE, 0, poison=False)
    want, bound = st.reference(F32)
    st.dev["table"][1, 1] = 10 ** 6
    got = st.decode(F32)
    assert st.status.item() == BAD_BLOCK and got.isfinite().all()
    ref.assert_within(got[[0, 2]], want[[0, 2]], bound[[0, 2]])
    st.status.zero_()
    st.dev["table"][1, 1] = st.table[1, 1].item()
    st.dev["ctx"][1] = -5
    got = st.decode(F32)
    assert st.status.item() == BAD_CONTEXT and (got[1] == 0).all()
    ref.assert_within(got[[0, 2]], want[[0, 2]], bound[[0, 2]])
    st = Step([64, 40, 100], [10, 41, 30], 4, 2, 64, BF16, WHOLE, 0, poison=False)
    st.ctx[1] = 41
    keep = list(range(10)) + list(range(51, 81))
    want, bound = [x[keep] for x in st.reference(F32)]
    got = st.prefill(F32)
    assert st.status.item() == BAD_CHUNK and got[10:51].isnan().all()
    ref.assert_within(got[keep], want, bound)
    for change, bit in ((dict(max_q=29), BAD_CHUNK), (dict(), BAD_BLOCK), (dict(), BAD_CONTEXT)):
        st = Step([64, 100], [10, 30], 4, 2, 64, BF16, WHOLE, 0, poison=False)
        want, bound = [x[:10] for x in st.reference(F32)]
        if bit == BAD_BLOCK:
            st.dev["table"][1, 2] = -4
        if bit == BAD_CONTEXT:
            st.dev["ctx"][1] = 10 ** 6
        got = st.prefill(F32, **change)
        assert st.status.item() == bit
        ref.assert_within(got[:10], want, bound)


def test_refusals(cuda_lib):
    st = Step([64], [1], 4, 2, 64, BF16, WHOLE, 0)
    with pytest.raises(PkvError):
        st.decode(F32, scale=-1.0)
    with pytest.raises(PkvError):
        st.decode(F16)
    st.k = st.k.view(torch.uint8)
    with pytest.raises(TypeError):
        st.decode(F32)
