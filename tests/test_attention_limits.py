"""CPU checks of the sizes that one attention call refuses as a whole."""
import ctypes

import pytest

import nvfp4_w4a4_quantized_02_b200 as nv
from nvfp4_w4a4_quantized_02_b200 import build as nvbuild

P = 1 << 20  # never dereferenced: validation fails first


@pytest.mark.parametrize("tokens,n_seqs,heads", [
    (65535, 65535, 65535),     # 4.8e9 units of single tokens
    (16_000_000, 1, 65535),    # 4.1e9 row blocks of a prompt
])
def test_more_ctas_than_a_grid_has(tokens, n_seqs, heads):
    nvbuild.build()
    cache = nv.BlockCache(P, P, P, P, 1, 64, heads, 64)
    batch = nv.Batch(P, P, P, n_seqs, tokens, 3, 3)
    ld = heads * 64
    assert nv.attention_workspace_bytes(tokens, n_seqs, heads, heads, 64) == 0
    assert nv.lib().nvfp4_attention(P, ld, heads, batch, cache, 0.1, 1, P, 0, ld, P, ctypes.c_size_t(-1), None) == 2


def test_large_calls_that_do_fit():
    nvbuild.build()
    assert nv.attention_workspace_bytes(1 << 20, 65535, 96, 8, 128) > 0
    assert nv.attention_workspace_bytes(1 << 20, 1, 96, 8, 256) > 0
