"""Sizes that append to the cache in 8 bits turns down on the host, before anything is enqueued (no GPU needed: the
pointers are never followed)."""
import pytest

from test_quant_ref import APPEND, UNSUPPORTED, call


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads", [(1 << 16) + 1, 1 << 24, 1 << 25])
def test_append_of_too_many_heads(heads, d):
    """Offsets within a token's row, head times head_dim, are 32-bit in the kernel; read back and attention end at 65,536
    heads too."""
    assert call("pkv_kv_append_e4m3", APPEND, hkv=heads, T=16, num_blocks=4, d=d, k_stride=heads * d, v_stride=heads * d) == UNSUPPORTED
    assert call("pkv_kv_append_e4m3", APPEND, hkv=1 << 16, T=0, d=d) == 0
