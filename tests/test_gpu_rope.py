"""pkv_qk_rope and pkv_qk_rope_append against the formula in 64 bits.

Bound on a stored value, from the arithmetic: y_i cos a - y_j sin a takes three
fp32 roundings (2^-24 each) and the error of cos and sin: the angle as a number
of half turns is rounded to 2^-25 (pi 2^-25 < 2^-23 radians) and sincospi is
good to 2^-23, so 2^-21 m (|y_i| + |y_j|) covers them.  A norm adds a relative
(d + 8) 2^-24 (the sum of squares' d additions, division, root, two products).
The store then rounds by half a step.
"""
import math

import pytest
import torch

import window_ref as ref
from paged_kv_cache_tables_gb300 import (ROPE_BANDS, ROPE_LINEAR, ROPE_NTK, ROPE_PLAIN, ROPE_YARN, PkvError, qk_rope,
                                         qk_rope_append, rope_frequencies)

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
SCALINGS = {"plain": dict(scaling=ROPE_PLAIN), "linear": dict(scaling=ROPE_LINEAR, factor=4.0),
            "ntk": dict(scaling=ROPE_NTK, factor=8.0),
            "bands": dict(base=500000.0, scaling=ROPE_BANDS, factor=8.0, original_context=8192, low=1.0, high=4.0),
            "yarn": dict(scaling=ROPE_YARN, factor=16.0, original_context=4096, low=1.0, high=32.0)}


def turned(x, positions, freqs, mscale, rot, interleaved, weight, eps):
    """(value, bound before the store's rounding) of the rows x [T, H, d], 64 bits on the CPU."""
    x = x.double().cpu()
    T, H, d = x.shape
    extra = 0.0
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.double().cpu()
        extra = (d + 8) * 2.0 ** -24
    # whole turns dropped exactly, as integers
    turn = torch.tensor([[(int(p) * int(f)) % 2 ** 64 / 2.0 ** 64 for f in freqs.tolist()] for p in positions.tolist()],
                        dtype=torch.float64).reshape(T, 1, rot // 2) * 2 * math.pi
    c, s = mscale * torch.cos(turn), mscale * torch.sin(turn)
    i = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    j = i + 1 if interleaved else i + rot // 2
    y, err = x.clone(), x.abs() * (extra + 2.0 ** -23)
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., i] * s + x[..., j] * c
    both = mscale * (x[..., i].abs() + x[..., j].abs()) * (extra + 2.0 ** -21)
    err[..., i] = both
    err[..., j] = both
    return y, err


def check(got, x, positions, freqs, m, rot, interleaved, weight, eps, what):
    y, err = turned(x, positions, freqs, m, rot, interleaved, weight, eps)
    ref.assert_within(got, y, err + ref.rounding(y, err, got.dtype), what)


def rows(T, H, d, dtype, g, scale=1.0):
    return (torch.randn(T, H, d, generator=g) * scale).to(dtype).cuda()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T,Hq,Hkv,d,rot", [(1, 1, 1, 64, 64), (1, 32, 8, 128, 128), (3, 5, 1, 64, 16), (7, 8, 2, 64, 48),
                                            (33, 32, 8, 64, 32), (129, 6, 2, 128, 64), (17, 3, 3, 128, 112),
                                            (700, 4, 4, 128, 128), (2500, 2, 1, 64, 64)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("normed", ["none", "both", "q", "k"])
def test_qk_rope(cuda_lib, T, Hq, Hkv, d, rot, dtype, interleaved, normed):
    g = torch.Generator().manual_seed(T * 131 + rot)
    q, k = rows(T, Hq, d, dtype, g), rows(T, Hkv, d, dtype, g, 3.0)
    pos = torch.randint(0, 5000, (T,), generator=g, dtype=torch.int32).cuda()
    freqs, m = rope_frequencies(rot)
    w = {n: (1 + 0.2 * torch.randn(d, generator=g)).to(dtype).cuda() if normed in (n, "both") else None for n in "qk"}
    qo, ko = torch.full_like(q, float("nan")), torch.full_like(k, float("nan"))
    q0, k0 = q.clone(), k.clone()
    qk_rope(qo, ko, q, k, pos, freqs, interleaved=interleaved, mscale=m, q_weight=w["q"], k_weight=w["k"], eps=1e-5)
    assert torch.equal(q, q0) and torch.equal(k, k0)
    check(qo, q, pos, freqs, m, rot, interleaved, w["q"], 1e-5, "q")
    check(ko, k, pos, freqs, m, rot, interleaved, w["k"], 1e-5, "k")


@pytest.mark.parametrize("name", sorted(SCALINGS))
@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions_and_scalings(cuda_lib, name, interleaved):
    g = torch.Generator().manual_seed(5)
    freqs, m = rope_frequencies(64, **SCALINGS[name])
    pos = torch.tensor([0, 1, 2 ** 31 - 1, -2 ** 31, -1, 1 << 20, 524287, 131071, 99999999], dtype=torch.int32).cuda()
    q, k = rows(9, 4, 128, BF16, g), rows(9, 2, 128, BF16, g)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    qk_rope(qo, ko, q, k, pos, freqs, interleaved=interleaved, mscale=m)
    check(qo, q, pos, freqs, m, 64, interleaved, None, 0, "q")
    check(ko, k, pos, freqs, m, 64, interleaved, None, 0, "k")
    if m == 1.0:
        assert torch.equal(qo[0], q[0])   # position 0 turns nothing


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_extreme_values(cuda_lib, dtype):
    """Rows of zeros, of the type's largest values and of subnormals, with and without a norm; infinities and NaN stay in their row."""
    big = torch.finfo(dtype).max
    freqs, m = rope_frequencies(64)
    q = torch.zeros(6, 2, 64, dtype=dtype)
    q[1] = 1.0
    q[2] = torch.finfo(dtype).tiny / 4
    q[3] = 100.0
    q[4, 0, 3] = float("inf")
    q[5, 1, 7] = float("nan")
    q, k = q.cuda(), torch.full((6, 1, 64), big / 2, dtype=dtype).cuda()
    pos = torch.arange(6, dtype=torch.int32).cuda()
    w = torch.full((64,), 0.5).cuda()   # a weight in 32 bits
    for weight, eps in ((None, 0.0), (w, 1e-6)):
        qo, ko = torch.empty_like(q), torch.empty_like(k)
        qk_rope(qo, ko, q, k, pos, freqs, q_weight=weight, eps=eps)
        for r, h in ((0, 0), (0, 1), (1, 0), (2, 1), (3, 0), (4, 1), (5, 0)):
            check(qo[r:r + 1, h:h + 1], q[r:r + 1, h:h + 1], pos[r:r + 1], freqs, m, 64, False, weight, eps, (r, h))
        assert not torch.isfinite(qo[4, 0].float()).all() and torch.isnan(qo[5, 1].float()).any()
    # half the largest value, normed: the squares stay in range of fp32 for fp16, and overflow it for bf16
    qk_rope(qo, ko, q, k, pos, freqs, k_weight=w, eps=1e-6)
    if dtype == F16:
        check(ko, k, pos, freqs, m, 64, False, w, 1e-6, "large")


def test_in_place_on_slices_of_fused_rows(cuda_lib):
    g = torch.Generator().manual_seed(1)
    T, Hq, Hkv, d = 301, 6, 2, 128
    fused = (torch.randn(T, (Hq + 2 * Hkv) * d + 24, generator=g)).to(BF16).cuda()
    before = fused.clone()

    def parts(x):
        return (x[:, :Hq * d].view(T, Hq, d), x[:, Hq * d:(Hq + Hkv) * d].view(T, Hkv, d),
                x[:, (Hq + Hkv) * d:(Hq + 2 * Hkv) * d].view(T, Hkv, d))

    q, k, _ = parts(fused)
    pos = torch.randint(0, 9000, (T,), generator=g, dtype=torch.int32).cuda()
    freqs, m = rope_frequencies(64)
    qk_rope(q, k, q, k, pos, freqs, interleaved=True)
    q0, k0, v0 = parts(before)
    check(q, q0, pos, freqs, m, 64, True, None, 0, "q")
    check(k, k0, pos, freqs, m, 64, True, None, 0, "k")
    assert torch.equal(fused[:, (Hq + Hkv) * d:], before[:, (Hq + Hkv) * d:])
    # an input repeated for every token (stride 0)
    one = before[:1, :Hq * d].view(1, Hq, d).expand(T, Hq, d)
    qo, ko = torch.empty(T, Hq, d, dtype=BF16, device="cuda"), torch.empty(T, Hkv, d, dtype=BF16, device="cuda")
    qk_rope(qo, ko, one, k0, pos, freqs)
    check(qo, one, pos, freqs, m, 64, False, None, 0, "broadcast q")


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T,Hq,Hkv,d,rot,inter,normed", [(1, 4, 4, 64, 64, False, True), (64, 32, 8, 64, 64, False, False),
                                                         (333, 20, 4, 128, 64, True, True), (1500, 8, 1, 128, 128, False, True)])
def test_append(cuda_lib, T, Hq, Hkv, d, rot, inter, normed, dtype):
    g = torch.Generator().manual_seed(T)
    fused = torch.randn(T, (Hq + 2 * Hkv) * d + 64, generator=g).to(dtype).cuda()
    q, k, v = (x.view(T, -1, d) for x in fused.split([Hq * d, Hkv * d, Hkv * d, 64], dim=1)[:3])
    pos = torch.randint(0, 1 << 20, (T,), generator=g, dtype=torch.int32).cuda()
    NB = T // 16 + 3
    slots = torch.randperm(NB * 16, generator=g)[:T]
    bad = 0
    if T > 10:
        slots[3], slots[7], slots[9] = -1, -(2 ** 40), NB * 16
        slots[10] = 2 ** 45
        bad = 8
    w = (1 + 0.2 * torch.randn(d, generator=g)).to(dtype).cuda() if normed else None
    freqs, m = rope_frequencies(rot, **SCALINGS["yarn"])
    kc = torch.full((NB, Hkv, 16, d), -3.0, dtype=dtype, device="cuda")
    vc = torch.full((NB, Hkv, 16, d), -5.0, dtype=dtype, device="cuda")
    qo = torch.full((T, Hq, d), float("nan"), dtype=dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    qk_rope_append(qo, q, k, v, pos, slots.cuda(), freqs, kc, vc, interleaved=inter, mscale=m, q_weight=w, k_weight=w,
                   eps=1e-6, dev_status=status)
    check(qo, q, pos, freqs, m, rot, inter, w, 1e-6, "q")
    ok = (slots >= 0) & (slots < NB * 16)
    at = slots[ok].cuda()
    check(kc[at // 16, :, at % 16], k[ok.cuda()], pos[ok.cuda()], freqs, m, rot, inter, w, 1e-6, "k")
    assert torch.equal(vc[at // 16, :, at % 16], v[ok.cuda()])
    rest = torch.ones(NB * 16, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert (kc.transpose(1, 2).reshape(NB * 16, -1)[rest] == -3).all()
    assert (vc.transpose(1, 2).reshape(NB * 16, -1)[rest] == -5).all()
    assert status.item() == bad


def test_no_tokens(cuda_lib):
    e = torch.empty(0, 4, 64, dtype=BF16, device="cuda")
    i = torch.empty(0, dtype=torch.int32, device="cuda")
    freqs, _ = rope_frequencies(64)
    c = torch.zeros(2, 4, 16, 64, dtype=BF16, device="cuda")
    qk_rope(e, e, e, e, i, freqs)
    qk_rope_append(e, e, e, e, i, i.long(), freqs, c, c)
    assert (c == 0).all()


def test_captured_on_a_side_stream(cuda_lib):
    g = torch.Generator().manual_seed(2)
    q, k = rows(40, 8, 64, BF16, g), rows(40, 2, 64, BF16, g)
    pos = torch.randint(0, 4000, (40,), generator=g, dtype=torch.int32).cuda()
    freqs, m = rope_frequencies(64)
    qo, ko = torch.zeros_like(q), torch.zeros_like(k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        qk_rope(qo, ko, q, k, pos, freqs)
    for shift in (0, 77):
        pos += shift
        q.mul_(-1)
        graph.replay()
        check(qo, q, pos, freqs, m, 64, False, None, 0, shift)
        check(ko, k, pos, freqs, m, 64, False, None, 0, shift)


def test_refusals(cuda_lib):
    g = torch.Generator().manual_seed(2)
    q, k = rows(4, 8, 64, BF16, g), rows(4, 2, 64, BF16, g)
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    freqs, _ = rope_frequencies(64)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    with pytest.raises(ValueError):
        qk_rope(qo, ko, q, k, pos[:3], freqs)
    with pytest.raises(TypeError):
        qk_rope(qo, ko, q, k, pos.long(), freqs)
    with pytest.raises(TypeError):
        qk_rope(qo.half(), ko, q, k, pos, freqs)
    with pytest.raises(ValueError):   # heads of a token apart
        qk_rope(qo, ko, q.transpose(0, 1).contiguous().transpose(0, 1), k, pos, freqs)
    with pytest.raises(ValueError):
        qk_rope(qo, ko, q, k, pos, freqs.cpu())
    with pytest.raises(TypeError):
        qk_rope(qo, ko, q, k, pos, freqs, q_weight=torch.ones(64, device="cuda"),
                k_weight=torch.ones(64, device="cuda", dtype=BF16))
    with pytest.raises(PkvError):     # the output over the next token's input
        qk_rope(q[1:], ko[:3], q[:3], k[:3], pos[:3], freqs)
    with pytest.raises(PkvError):     # 128 dimensions turned of 64
        qk_rope(qo, ko, q, k, pos, rope_frequencies(128)[0])
    with pytest.raises(PkvError):     # rows that start between 16-byte boundaries
        buf = torch.zeros(4 * 512 + 4, dtype=BF16, device="cuda")
        qk_rope(buf[4:].view(4, 8, 64), ko, q, k, pos, freqs)
