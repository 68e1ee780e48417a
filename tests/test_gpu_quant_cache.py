"""Writing the cache held in 8 bits and reading it back, against the definition in 64 bits: codes and scales are equal
bit for bit, rows read back are within half a step of the output's type."""
import pytest
import torch

import quant_ref as qr
import window_ref as ref
from paged_kv_cache_tables_gb300 import kv_append_e4m3, kv_gather_e4m3
from quant_ref import BF16, CODE, F16, F32

pytestmark = pytest.mark.gpu
BAD_BLOCK, BAD_CONTEXT, BAD_SLOT = 1, 2, 8


def rows(g, T, Hkv, d, dtype, spread=1.0):
    x = torch.randn(T, Hkv, d, generator=g) * torch.exp(spread * torch.randn(T, 1, 1, generator=g))
    return x.to(dtype)


class Cache:
    """A cache on the GPU and its twin in 64 bits."""

    def __init__(self, NB, Hkv, d, seed=0):
        g = torch.Generator().manual_seed(seed)
        (k, ks), (v, vs) = qr.pool(g, NB, Hkv, d), qr.pool(g, NB, Hkv, d)
        self.codes = [k, v]
        self.scales = torch.stack([ks, vs], 2).double()
        self.dev = [k.cuda().view(CODE), v.cuda().view(CODE)]
        self.dev_scales = self.scales.float().cuda()
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def append(self, k, v, slots, **kw):
        kv_append_e4m3(k.cuda() if not k.is_cuda else k, v.cuda() if not v.is_cuda else v,
                       torch.tensor(slots, dtype=torch.int64).cuda(), *self.dev, self.dev_scales, dev_status=self.status, **kw)
        for i, x in enumerate((k, v)):
            qr.append(x.cpu().double(), slots, self.codes[i], self.scales, i)

    def check(self):
        got = [c.view(torch.uint8).cpu() for c in self.dev]
        assert torch.equal(self.dev_scales.cpu().double(), self.scales)
        for g, want in zip(got, self.codes):
            same = (g == want) | ((g & 127 == 127) & (want & 127 == 127))   # a NaN of either sign
            assert same.all(), (~same).nonzero()[:5]


@pytest.mark.parametrize("Hkv,d,dtype", [(1, 64, BF16), (2, 128, F16), (3, 64, F16), (8, 128, BF16)])
def test_append(cuda_lib, Hkv, d, dtype):
    """Chunks that start, end and cross blocks at every offset, single rows, padding rows, in one call; then more rows on
    the same blocks, whose scales grow."""
    g = torch.Generator().manual_seed(d + Hkv)
    c = Cache(120, Hkv, d)
    slots, free = [], torch.randperm(120, generator=g).tolist()
    ends = []
    for start, n in [(o, m) for o in range(0, 16, 3) for m in (1, 2, 15, 16, 17, 33)]:
        blocks = [free.pop() for _ in range(-(-(start + n) // 16))] if len(free) > 8 else []
        slots += [blocks[p // 16] * 16 + p % 16 for p in range(start, start + n)] if blocks else []
        slots += [-1] * (n % 2)
        if blocks and (start + n) % 16:
            ends.append(blocks[-1] * 16 + (start + n) % 16)
    slots += [-7, -1]
    c.append(rows(g, len(slots), Hkv, d, dtype), rows(g, len(slots), Hkv, d, dtype), slots)
    c.check()
    for scale in (1.0, 8.0, 0.1, 100.0):
        c.append((rows(g, len(ends), Hkv, d, dtype) * scale), (rows(g, len(ends), Hkv, d, dtype) / scale), ends)
        c.check()
        ends = [s + 1 for s in ends if s % 16 < 15]
    assert c.status.item() == 0


@pytest.mark.parametrize("T", [1, 7, 300, 5000])
@pytest.mark.parametrize("Hkv", [1, 8])
def test_append_prompts(cuda_lib, T, Hkv):
    g = torch.Generator().manual_seed(T)
    c = Cache(T // 16 + 3, Hkv, 128)
    ids = torch.randperm(T // 16 + 3, generator=g).tolist()
    slots = [ids[p // 16] * 16 + p % 16 for p in range(T)]
    c.append(rows(g, T, Hkv, 128, BF16), rows(g, T, Hkv, 128, BF16), slots)
    c.check()


def test_append_token_by_token(cuda_lib):
    """A block filled a row at a time, magnitudes rising, falling and none."""
    g = torch.Generator().manual_seed(5)
    for mags in ([2.0 ** i for i in range(16)], [2.0 ** -i for i in range(16)], [0.0] * 16, [0.0, 1, 0, 1e-25, 3e4, 0, 1, 2] * 2):
        c = Cache(4, 2, 64)
        for off, m in enumerate(mags):
            k, v = rows(g, 3, 2, 64, BF16, 0.1) * m, rows(g, 3, 2, 64, BF16, 0.1) * m
            c.append(k, v, [2 * 16 + off, -1, 0 * 16 + off])
            c.check()


def test_append_not_finite(cuda_lib):
    """Infinities saturate and, like NaN, do not enter the scale; a scale that is none counts as 0."""
    g = torch.Generator().manual_seed(6)
    for dtype in (BF16, F16):
        c = Cache(6, 2, 64)
        k, v = rows(g, 20, 2, 64, dtype), rows(g, 20, 2, 64, dtype)
        k[0], k[3, 1, 5], k[4, :, 7], v[19], v[2, 0, 0] = float("nan"), float("inf"), float("-inf"), float("inf"), float("nan")
        k[5, 0, :] = torch.finfo(dtype).max
        c.dev_scales[3] = c.scales[3] = float("nan")
        c.dev_scales[4] = c.scales[4] = -1.0
        c.append(k, v, [16 + i for i in range(16)] + [3 * 16 + 2, 4 * 16 + 9, 0, 1])
        c.check()


def test_append_strided_rows(cuda_lib):
    """k and v as slices of one projection's rows, K and V of different strides, one token of any stride."""
    g = torch.Generator().manual_seed(7)
    for T in (1, 40):
        c = Cache(6, 2, 128)
        qkv = rows(g, T, 1, 8 * 128 + 2 * 256 + 24, BF16)[:, 0].cuda()
        k, v = qkv[:, 1024:1280].view(T, 2, 128), qkv[:, 1280:1536].view(T, 2, 128)
        c.append(k, v.contiguous(), [16 + i for i in range(T)])
        c.check()
        c.append(k, v, [3 + i for i in range(T)])
        c.check()


def test_append_bad_slots_and_nothing(cuda_lib):
    c = Cache(4, 2, 64)
    g = torch.Generator().manual_seed(8)
    x = rows(g, 5, 2, 64, BF16)
    c.append(x, x, [4 * 16, 17, 2 ** 40, 4 * 16 + 3, -1])
    c.check()
    assert c.status.item() == BAD_SLOT
    c.append(x[:0], x[:0], [])
    c.check()


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("Hkv,d", [(1, 64), (8, 128), (3, 128), (5, 64)])
def test_gather(cuda_lib, dtype, Hkv, d):
    g = torch.Generator().manual_seed(d)
    lens, first = [0, 1, 15, 16, 17, 100, 0, 333, 3, 0], [0, 5, 0, 16, 31, 7, 3, 1, 200, 1]
    for with_first in (False, True):
        starts = first if with_first else [0] * len(lens)
        nb = [-(-(a + n) // 16) for a, n in zip(starts, lens)]
        NB = sum(nb) + 2
        (k, ks), (v, vs) = qr.pool(g, NB, Hkv, d), qr.pool(g, NB, Hkv, d, odd_scales=True)
        ids = torch.randperm(NB, generator=g).int()
        table = torch.full((len(lens), max(nb) + 1), -1, dtype=torch.int32)
        at = 0
        for s, n in enumerate(nb):
            table[s, :n] = ids[at:at + n]
            at += n
        cu = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32)
        T = sum(lens)
        out = [torch.full((T + 21, Hkv, d), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        scales = torch.stack([ks, vs], 2).contiguous()
        kv_gather_e4m3(*out, k.cuda().view(CODE), v.cuda().view(CODE), scales.cuda(), table.cuda(), cu.cuda(),
                       first=torch.tensor(first, dtype=torch.int32).cuda() if with_first else None, dev_status=status)
        for i, codes in enumerate((k, v)):
            want = torch.cat([qr.gathered(codes, scales[..., i], table[s], a + n)[a:] for s, (a, n) in enumerate(zip(starts, lens))])
            # code times scale has up to 28 bits: rounded to fp32 and then to 16 bits, which can move a tie by half a step of fp32
            err = want.abs() * 2.0 ** -24
            ref.assert_within(out[i][:T], want, (0 if dtype == F32 else err) + ref.rounding(want, err, dtype))
            assert (out[i][T:] == 7).all()
        assert status.item() == 0


def test_gather_many_sequences(cuda_lib):
    """More sequences than a search of a few steps covers, empty ones among them."""
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 4, (3000,), generator=g).tolist()
    NB = 3000
    k, ks = qr.pool(g, NB, 1, 64)
    table = torch.randperm(NB, generator=g).int().view(NB, 1)
    cu = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32)
    scales = torch.stack([ks, ks], 2).contiguous()
    out = [torch.zeros((sum(lens), 1, 64), dtype=F32, device="cuda") for _ in range(2)]
    kv_gather_e4m3(*out, k.cuda().view(CODE), k.cuda().view(CODE), scales.cuda(), table.cuda(), cu.cuda())
    want = torch.cat([qr.gathered(k, ks, table[s], n) for s, n in enumerate(lens)])
    for o in out:
        assert torch.equal(o.cpu().double(), want)


def test_gather_reports_what_it_cannot_read(cuda_lib):
    g = torch.Generator().manual_seed(4)
    k, ks = qr.pool(g, 4, 2, 64)
    scales = torch.stack([ks, ks], 2).contiguous().cuda()
    dev = k.cuda().view(CODE)

    def call(table, cu, first=None):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = [torch.full((24, 2, 64), 7.0, dtype=F32, device="cuda") for _ in range(2)]
        kv_gather_e4m3(*out, dev, dev, scales, torch.tensor(table, dtype=torch.int32).cuda(),
                       torch.tensor(cu, dtype=torch.int32).cuda(),
                       first=None if first is None else torch.tensor(first, dtype=torch.int32).cuda(), dev_status=status)
        return out[0], status.item()

    out, status = call([[1, 9], [-3, 2]], [0, 20, 24])
    assert status == BAD_BLOCK and (out[16:24] == 0).all() and (out[:16] != 0).any()
    out, status = call([[1], [2]], [0, 17, 18])
    assert status == BAD_CONTEXT and (out[16] == 0).all() and (out[17] != 0).any() and (out[18:] == 7).all()
    out, status = call([[1], [2]], [0, 2, 4], [-1, 15])
    assert status == BAD_CONTEXT and (out[0] == 0).all() and (out[3] == 0).all() and (out[1:3] != 0).any(-1).all()


def test_written_and_read_back(cuda_lib):
    """A row read back is within half a step of e4m3 at its block's scale."""
    g = torch.Generator().manual_seed(9)
    T, Hkv, d = 500, 4, 128
    c = Cache(40, Hkv, d)
    ids = torch.randperm(40, generator=g)
    x = [rows(g, T, Hkv, d, BF16, 0.3) for _ in range(2)]
    c.append(*x, [ids[p // 16].item() * 16 + p % 16 for p in range(T)])
    out = [torch.zeros((T, Hkv, d), dtype=F32, device="cuda") for _ in range(2)]
    kv_gather_e4m3(*out, *c.dev, c.dev_scales, ids.int().view(1, -1).cuda(), torch.tensor([0, T], dtype=torch.int32).cuda())
    b = ids[torch.arange(T) // 16]
    for i in range(2):
        step = x[i].double().abs() / 16 + 2.0 ** -10 * c.scales[b, :, i].unsqueeze(-1)
        ref.assert_within(out[i], x[i].double(), step)
