"""Append to the cache in 8 bits where a token's rows are wide: 16 tokens a CTA from 4,096 elements on, whatever the
number of rows, and 8 of few rows below that; codes and scales bit for bit on both sides of the border."""
import pytest
import torch

from quant_ref import BF16, F16
from test_gpu_quant_cache import Cache, rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hkv,d,dtype", [(31, 128, BF16), (32, 128, BF16), (33, 128, F16), (63, 64, F16), (64, 64, BF16)])
@pytest.mark.parametrize("chunk,singles", [(1, 0), (0, 17), (70, 0), (33, 25)])
def test_append_of_wide_rows(cuda_lib, Hkv, d, dtype, chunk, singles):
    g = torch.Generator().manual_seed(Hkv + chunk)
    c = Cache(40, Hkv, d)
    ids = torch.randperm(40, generator=g).tolist()
    of_chunk, of_singles = ids[:10], ids[10:]
    at, offs = 5, [3 * i % 15 for i in range(singles)]
    for turn in range(3):      # rows behind those before: a block's scale starts, stays or grows
        slots = [of_chunk[p // 16] * 16 + p % 16 for p in range(at, min(at + chunk, 160))]
        slots += [-1] * turn + [of_singles[i] * 16 + o + turn for i, o in enumerate(offs) if o + turn < 16]
        scale = (1.0, 30.0, 0.2)[turn]
        c.append(rows(g, len(slots), Hkv, d, dtype) * scale, rows(g, len(slots), Hkv, d, dtype) / scale, slots)
        c.check()
        at = min(at + chunk, 160)
    assert c.status.item() == 0
