"""Refusals of the window, rotation and table entry points: every bad argument
is turned down on the host before anything is enqueued (no GPU needed: the
pointers are never followed)."""
import ctypes
import math

import pytest
import torch

import paged_kv_cache_tables_gb300 as pkv
from paged_kv_cache_tables_gb300 import _binding as B

FAKE = 1 << 20
INVALID, UNSUPPORTED = -1, -2
NAN = float("nan")


def call(name, defaults, **change):
    args = dict(defaults)
    assert not set(change) - set(args), change
    args.update(change)
    return getattr(B.lib(), name)(*args.values())


DECODE = dict(out=FAKE, q=FAKE, k_cache=FAKE, v_cache=FAKE, block_tables=FAKE, max_blocks=4, context_lens=FAKE, num_seqs=2,
              num_blocks=8, hq=8, hkv=8, d=64, bs=16, window=32, sinks=4, scale=0.125, dtype=1, out_dtype=1, status=None,
              stream=None)
PREFILL = dict(out=FAKE, q=FAKE, cu=FAKE, num_seqs=1, max_q=16, total_q=16, k_cache=FAKE, v_cache=FAKE, block_tables=FAKE,
               max_blocks=4, context_lens=FAKE, num_blocks=8, hq=8, hkv=8, d=64, bs=16, window=32, sinks=4, scale=0.125,
               dtype=1, out_dtype=1, status=None, stream=None)
ATTENTION = [
    (dict(window=0), INVALID), (dict(window=-1), INVALID), (dict(sinks=-1), INVALID), (dict(scale=0.0), INVALID),
    (dict(scale=-1.0), INVALID), (dict(scale=NAN), INVALID), (dict(scale=math.inf), INVALID), (dict(hq=6, hkv=4), INVALID),
    (dict(hq=34, hkv=2), UNSUPPORTED), (dict(d=96), UNSUPPORTED), (dict(bs=32), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED),
    (dict(out_dtype=0), UNSUPPORTED), (dict(num_blocks=0), INVALID), (dict(hkv=0), INVALID), (dict(max_blocks=0), INVALID),
    (dict(num_seqs=-1), INVALID), (dict(num_blocks=1 << 27), UNSUPPORTED), (dict(max_blocks=(1 << 26) + 1), UNSUPPORTED),
    (dict(out=None), INVALID), (dict(q=None), INVALID), (dict(k_cache=None), INVALID), (dict(v_cache=None), INVALID),
    (dict(block_tables=None), INVALID), (dict(context_lens=None), INVALID), (dict(k_cache=FAKE + 8), INVALID),
    (dict(v_cache=FAKE + 2), INVALID), (dict(q=FAKE + 2), INVALID), (dict(out=FAKE + 2), INVALID),
    (dict(q=FAKE + 8), INVALID), (dict(out=FAKE + 8), INVALID),
    (dict(block_tables=FAKE + 1), INVALID), (dict(context_lens=FAKE + 2), INVALID),
    (dict(num_seqs=0, out=None, q=None, k_cache=None, v_cache=None, block_tables=None, context_lens=None), 0)]


@pytest.mark.parametrize("change,rc", ATTENTION + [(dict(num_seqs=1 << 24, max_blocks=128), UNSUPPORTED),
                                                   (dict(num_seqs=1 << 24), UNSUPPORTED)])
def test_window_decode(change, rc):
    assert call("pkv_paged_window_decode_attention", DECODE, **change) == rc


@pytest.mark.parametrize("change,rc", ATTENTION + [
    (dict(max_q=-1), INVALID), (dict(total_q=-1), INVALID), (dict(cu=None), INVALID), (dict(cu=FAKE + 2), INVALID),
    (dict(q=FAKE + 4), INVALID), (dict(out=FAKE + 8), INVALID), (dict(total_q=0, q=None, out=None), 0),
    (dict(max_q=0), 0)])
def test_window_prefill(change, rc):
    assert call("pkv_paged_window_prefill_attention", PREFILL, **change) == rc


Q, K, V, QO, KO = (FAKE + i * (1 << 20) for i in range(5))
ROPE = dict(q_out=QO, q_out_stride=512, k_out=KO, k_out_stride=128, q=Q, q_stride=512, k=K, k_stride=128, positions=FAKE,
            freqs=FAKE, rot=64, interleaved=0, mscale=1.0, q_weight=None, k_weight=None, weight_dtype=1, eps=1e-6, T=16,
            hq=8, hkv=2, d=64, dtype=1, stream=None)
APPEND = dict(q_out=QO, q_out_stride=512, q=Q, q_stride=512, k=K, k_stride=128, v=V, v_stride=128, positions=FAKE,
              slots=FAKE, freqs=FAKE, rot=64, interleaved=0, mscale=1.0, q_weight=None, k_weight=None, weight_dtype=1,
              eps=1e-6, T=16, k_cache=FAKE, v_cache=FAKE, num_blocks=8, bs=16, hq=8, hkv=2, d=64, dtype=1, status=None,
              stream=None)
W = FAKE + (1 << 26)   # a weight's address
ROTATE = [
    (dict(rot=0), UNSUPPORTED), (dict(rot=8), UNSUPPORTED), (dict(rot=40), UNSUPPORTED), (dict(rot=80), UNSUPPORTED),
    (dict(d=96), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED), (dict(hq=0), INVALID), (dict(hkv=0), INVALID),
    (dict(T=-1), INVALID), (dict(mscale=NAN), INVALID), (dict(q_weight=W, eps=NAN), INVALID),
    (dict(q_weight=W, eps=-1.0), INVALID), (dict(q_weight=W, weight_dtype=0), UNSUPPORTED),
    (dict(q_weight=W + 4), INVALID), (dict(k_weight=W + 8), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID),
    (dict(q_out=None), INVALID), (dict(positions=None), INVALID), (dict(freqs=None), INVALID), (dict(freqs=FAKE + 4), INVALID),
    (dict(q=Q + 8), INVALID), (dict(k=K + 2), INVALID), (dict(q_out=QO + 4), INVALID), (dict(q_stride=516), INVALID),
    (dict(k_stride=130), INVALID), (dict(q_stride=-512), INVALID), (dict(k_stride=-128), INVALID),
    (dict(q_out_stride=504), INVALID), (dict(q_out_stride=516), INVALID),
    # an output over another input, or over its own input shifted by a row, part of a row or with another stride
    (dict(q_out=K), INVALID), (dict(q_out=Q + 1024), INVALID), (dict(q_out=Q + 512), INVALID),
    (dict(q_out=Q, q_out_stride=1024), INVALID),
    (dict(T=0, q=None, k=None, q_out=None, positions=None, freqs=None), 0)]


@pytest.mark.parametrize("change,rc", ROTATE + [
    (dict(k_out=None), INVALID), (dict(k_out=KO + 2), INVALID), (dict(k_out_stride=120), INVALID),
    (dict(k_out_stride=132), INVALID), (dict(k_out=Q), INVALID), (dict(k_out=QO + 512), INVALID),
    (dict(k_out=K + 256), INVALID)])
def test_qk_rope(change, rc):
    assert call("pkv_qk_rope", ROPE, **change) == rc


@pytest.mark.parametrize("change,rc", ROTATE + [
    (dict(v=None), INVALID), (dict(slots=None), INVALID), (dict(k_cache=None), INVALID), (dict(v_cache=None), INVALID),
    (dict(v=V + 8), INVALID), (dict(v_stride=-8), INVALID), (dict(v_stride=129), INVALID), (dict(slots=FAKE + 4), INVALID),
    (dict(k_cache=FAKE + 8), INVALID), (dict(v_cache=FAKE + 8), INVALID), (dict(num_blocks=0), INVALID),
    (dict(bs=8), UNSUPPORTED), (dict(q_out=V), INVALID)])
def test_qk_rope_append(change, rc):
    assert call("pkv_qk_rope_append", APPEND, **change) == rc


def test_fused_rows_in_place_pass_the_overlap_check():
    """q, k and v slices of one buffer's rows, q rotated in place: accepted up
    to the launch (which needs a device)."""
    if torch.cuda.is_available():
        pytest.skip("the fake pointers must not reach a device")
    rows = dict(q=FAKE, k=FAKE + 1024, v=FAKE + 1024 + 256, q_out=FAKE, q_stride=768, k_stride=768, v_stride=768,
                q_out_stride=768)
    assert call("pkv_qk_rope_append", APPEND, **rows) not in (0, INVALID, UNSUPPORTED)
    # the same slices, the output one head further: over k
    assert call("pkv_qk_rope_append", APPEND, **dict(rows, q_out=FAKE + 128)) == INVALID


TABLES = dict(seq_lens=FAKE, new_lens=FAKE, num_seqs=4, tables=FAKE, max_blocks=8, free_list=FAKE, capacity=16, count=FAKE,
              count_out=FAKE, num_blocks=16, bs=16, ctx=FAKE, cu=FAKE, slots=FAKE, pos=FAKE, max_tokens=8, status=None,
              stream=None)


@pytest.mark.parametrize("change,rc", [
    (dict(num_seqs=-1), INVALID), (dict(num_seqs=B.TABLES_MAX_SEQS + 1), UNSUPPORTED), (dict(max_blocks=0), INVALID),
    (dict(max_blocks=(1 << 26) + 1), UNSUPPORTED), (dict(capacity=-1), INVALID), (dict(num_blocks=0), INVALID),
    (dict(bs=8), UNSUPPORTED), (dict(max_tokens=-1), INVALID), (dict(seq_lens=None), INVALID), (dict(new_lens=None), INVALID),
    (dict(tables=None), INVALID), (dict(free_list=None), INVALID), (dict(count=None), INVALID), (dict(count_out=None), INVALID),
    (dict(ctx=None), INVALID), (dict(cu=None), INVALID), (dict(slots=None), INVALID), (dict(pos=None), INVALID),
    (dict(slots=FAKE + 4), INVALID), (dict(pos=FAKE + 2), INVALID), (dict(tables=FAKE + 1), INVALID)])
def test_step_tables(change, rc):
    assert call("pkv_step_tables", TABLES, **change) == rc


RELEASE = dict(tables=FAKE, max_blocks=8, seq_lens=FAKE, finished=FAKE, num_seqs=4, window=0, sinks=0, free_list=FAKE,
               capacity=16, count=FAKE, num_blocks=16, bs=16, workspace=FAKE, workspace_bytes=20, status=None, stream=None)


@pytest.mark.parametrize("change,rc", [
    (dict(num_seqs=-1), INVALID), (dict(num_seqs=B.TABLES_MAX_SEQS + 1), UNSUPPORTED), (dict(max_blocks=0), INVALID),
    (dict(window=-1), INVALID), (dict(sinks=-1), INVALID), (dict(capacity=-1), INVALID), (dict(num_blocks=0), INVALID),
    (dict(bs=8), UNSUPPORTED), (dict(tables=None), INVALID), (dict(seq_lens=None), INVALID), (dict(free_list=None), INVALID),
    (dict(count=None), INVALID), (dict(finished=FAKE + 2), INVALID), (dict(num_seqs=16384, max_blocks=1 << 17), UNSUPPORTED),
    (dict(num_seqs=257, workspace=None, workspace_bytes=2000), -3), (dict(num_seqs=257, workspace_bytes=1031), -3),
    (dict(num_seqs=257, workspace=FAKE + 2, workspace_bytes=2000), -3),
    (dict(num_seqs=0, tables=None, seq_lens=None, free_list=None, count=None, workspace=None, workspace_bytes=0), 0)])
def test_release_blocks(change, rc):
    assert call("pkv_release_blocks", RELEASE, **change) == rc


def test_release_workspace_size():
    assert [pkv.release_workspace_size(n) for n in (-1, 0, 256, 257, B.TABLES_MAX_SEQS)] == \
        [0, 0, 0, 1032, 4 * B.TABLES_MAX_SEQS + 4]


def test_bindings_refuse_cpu_tensors():
    x = torch.zeros(2, 2, 64, dtype=torch.float16)
    c = torch.zeros(4, 2, 16, 64, dtype=torch.float16)
    i = torch.zeros(2, dtype=torch.int32)
    t = torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(TypeError):
        pkv.paged_window_decode_attention(x, x, c, c, t, i, 16)
    with pytest.raises(TypeError):
        pkv.paged_window_prefill_attention(x, x, torch.zeros(3, dtype=torch.int32), 1, c, c, t, i, 16)
    with pytest.raises(TypeError):
        pkv.qk_rope(x, x, x, x, i, torch.zeros(32, dtype=torch.int64))
    with pytest.raises(TypeError):
        pkv.qk_rope_append(x, x, x, x, i, i.long(), torch.zeros(32, dtype=torch.int64), c, c)
    with pytest.raises(TypeError):
        pkv.step_tables(i, i, t, i, i[:1], 4, i, torch.zeros(3, dtype=torch.int32), i.long(), i)
    with pytest.raises(TypeError):
        pkv.release_blocks(t, i, i, i[:1], 4)
