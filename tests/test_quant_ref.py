"""The references for the cache held in 8 bits against a second way of computing
them, and refusals of its entry points: every bad argument is turned down on the
host before anything is enqueued (no GPU needed: the pointers are never followed)."""
import math

import pytest
import torch

import paged_kv_cache_tables_gb300 as pkv
import quant_ref as qr
from paged_kv_cache_tables_gb300 import _binding as B

FAKE = 1 << 20
INVALID, UNSUPPORTED = -1, -2


def test_codes_agree_with_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(qr.CODE).double()
    assert torch.equal(qr.decode(codes).nan_to_num(1e9), want.nan_to_num(1e9))
    g = torch.Generator().manual_seed(1)
    x = torch.randn(200000, generator=g, dtype=torch.float64) * torch.exp(4 * torch.randn(200000, generator=g, dtype=torch.float64))
    mids = torch.cat([qr._MID, -qr._MID, qr.VALUES[:127], torch.tensor([448.0, 449, 463.9, 1e9, -1e9, 2.0 ** -10, 2.0 ** -11])])
    x = torch.cat([x, mids]).float()
    assert torch.equal(qr.encode(x.double()), x.clamp(-448, 448).to(qr.CODE).view(torch.uint8))
    assert qr.encode(torch.tensor([math.inf, -math.inf, math.nan], dtype=torch.float64)).tolist() == [126, 254, 127]


def test_scale():
    assert [qr.scale_of(a) for a in (0.0, 448.0, 448.1, 224.0, 1.0, 1e-30)] == [2.0 ** -60, 1.0, 2.0, 0.5, 2.0 ** -8, 2.0 ** -60]


def call(name, defaults, **change):
    args = dict(defaults)
    assert not set(change) - set(args), change
    args.update(change)
    return getattr(B.lib(), name)(*args.values())


APPEND = dict(k=FAKE, k_stride=128, v=FAKE, v_stride=128, slots=FAKE, T=16, k_cache=FAKE, v_cache=FAKE, scales=FAKE,
              num_blocks=8, bs=16, hkv=2, d=64, dtype=1, status=None, stream=None)


@pytest.mark.parametrize("change,rc", [
    (dict(T=-1), INVALID), (dict(num_blocks=0), INVALID), (dict(hkv=0), INVALID), (dict(dtype=2), UNSUPPORTED),
    (dict(dtype=7), UNSUPPORTED), (dict(bs=32), UNSUPPORTED), (dict(d=96), UNSUPPORTED), (dict(k=None), INVALID),
    (dict(v=None), INVALID), (dict(slots=None), INVALID), (dict(k_cache=None), INVALID), (dict(v_cache=None), INVALID),
    (dict(scales=None), INVALID), (dict(k=FAKE + 8), INVALID), (dict(v=FAKE + 2), INVALID), (dict(slots=FAKE + 4), INVALID),
    (dict(k_cache=FAKE + 8), INVALID), (dict(v_cache=FAKE + 8), INVALID), (dict(scales=FAKE + 4), INVALID),
    (dict(k_stride=129), INVALID), (dict(v_stride=4), INVALID), (dict(k_stride=-128), INVALID), (dict(v_stride=-128), INVALID),
    (dict(T=1 << 29, hkv=2), UNSUPPORTED), (dict(T=0, k=None, v=None, slots=None, k_cache=None, v_cache=None, scales=None), 0)])
def test_append_refusals(change, rc):
    assert call("pkv_kv_append_e4m3", APPEND, **change) == rc


GATHER = dict(k=FAKE, v=FAKE, k_cache=FAKE, v_cache=FAKE, scales=FAKE, tables=FAKE, max_blocks=4, cu=FAKE, first=None,
              num_seqs=2, total=20, num_blocks=8, bs=16, hkv=2, d=64, out_dtype=1, status=None, stream=None)


@pytest.mark.parametrize("change,rc", [
    (dict(num_seqs=-1), INVALID), (dict(total=-1), INVALID), (dict(num_blocks=0), INVALID), (dict(hkv=0), INVALID),
    (dict(max_blocks=0), INVALID), (dict(bs=8), UNSUPPORTED), (dict(d=80), UNSUPPORTED), (dict(out_dtype=3), UNSUPPORTED),
    (dict(hkv=(1 << 16) + 1), UNSUPPORTED), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k_cache=None), INVALID),
    (dict(v_cache=None), INVALID), (dict(scales=None), INVALID), (dict(tables=None), INVALID), (dict(cu=None), INVALID),
    (dict(k=FAKE + 8), INVALID), (dict(v=FAKE + 4), INVALID), (dict(k_cache=FAKE + 1), INVALID), (dict(v_cache=FAKE + 8), INVALID),
    (dict(scales=FAKE + 4), INVALID), (dict(tables=FAKE + 2), INVALID), (dict(cu=FAKE + 1), INVALID), (dict(first=FAKE + 2), INVALID),
    (dict(total=0, k=None, v=None), 0), (dict(num_seqs=0, tables=None, cu=None), 0)])
def test_gather_refusals(change, rc):
    assert call("pkv_kv_gather_e4m3", GATHER, **change) == rc


DECODE = dict(out=FAKE, q=FAKE, k_cache=FAKE, v_cache=FAKE, scales=FAKE, block_tables=FAKE, max_blocks=4, context_lens=FAKE,
              num_seqs=2, num_blocks=8, hq=8, hkv=8, d=64, bs=16, window=32, sinks=4, scale=0.125, dtype=1, out_dtype=1,
              status=None, stream=None)
PREFILL = dict(out=FAKE, q=FAKE, cu=FAKE, num_seqs=1, max_q=16, total_q=16, k_cache=FAKE, v_cache=FAKE, scales=FAKE,
               block_tables=FAKE, max_blocks=4, context_lens=FAKE, num_blocks=8, hq=8, hkv=8, d=64, bs=16, window=32, sinks=4,
               scale=0.125, dtype=1, out_dtype=1, status=None, stream=None)
ATTENTION = [
    (dict(window=0), INVALID), (dict(window=-1), INVALID), (dict(sinks=-1), INVALID), (dict(scale=0.0), INVALID),
    (dict(scale=-1.0), INVALID), (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID), (dict(hq=6, hkv=4), INVALID),
    (dict(hq=34, hkv=2), UNSUPPORTED), (dict(hq=(1 << 16) + 16, hkv=(1 << 12) + 1), UNSUPPORTED), (dict(d=96), UNSUPPORTED), (dict(bs=32), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED),
    (dict(out_dtype=0), UNSUPPORTED), (dict(num_blocks=0), INVALID), (dict(hkv=0), INVALID), (dict(max_blocks=0), INVALID),
    (dict(num_seqs=-1), INVALID), (dict(num_blocks=1 << 27), UNSUPPORTED), (dict(max_blocks=(1 << 26) + 1), UNSUPPORTED),
    (dict(out=None), INVALID), (dict(q=None), INVALID), (dict(k_cache=None), INVALID), (dict(v_cache=None), INVALID),
    (dict(scales=None), INVALID), (dict(scales=FAKE + 4), INVALID),
    (dict(block_tables=None), INVALID), (dict(context_lens=None), INVALID), (dict(k_cache=FAKE + 8), INVALID),
    (dict(v_cache=FAKE + 2), INVALID), (dict(q=FAKE + 2), INVALID), (dict(out=FAKE + 2), INVALID),
    (dict(q=FAKE + 8), INVALID), (dict(out=FAKE + 8), INVALID),
    (dict(block_tables=FAKE + 1), INVALID), (dict(context_lens=FAKE + 2), INVALID),
    (dict(num_seqs=0, out=None, q=None, k_cache=None, v_cache=None, scales=None, block_tables=None, context_lens=None), 0)]


@pytest.mark.parametrize("change,rc", ATTENTION + [(dict(num_seqs=1 << 24, max_blocks=128), UNSUPPORTED),
                                                   (dict(num_seqs=1 << 24), UNSUPPORTED)])
def test_decode_refusals(change, rc):
    assert call("pkv_paged_decode_attention_e4m3", DECODE, **change) == rc


@pytest.mark.parametrize("change,rc", ATTENTION + [
    (dict(max_q=-1), INVALID), (dict(total_q=-1), INVALID), (dict(cu=None), INVALID), (dict(cu=FAKE + 2), INVALID),
    (dict(total_q=0, q=None, out=None), 0), (dict(max_q=0), 0)])
def test_prefill_refusals(change, rc):
    assert call("pkv_paged_prefill_attention_e4m3", PREFILL, **change) == rc


def test_python_refuses_before_the_library():
    t = torch.zeros(4, 2, 64)
    for call in (lambda: pkv.kv_append_e4m3(t, t, t, t, t, t), lambda: pkv.kv_gather_e4m3(t, t, t, t, t, t, t),
                 lambda: pkv.paged_decode_attention_e4m3(t, t, t, t, t, t, t),
                 lambda: pkv.paged_prefill_attention_e4m3(t, t, t, 4, t, t, t, t, t)):
        with pytest.raises((TypeError, ValueError)):
            call()
