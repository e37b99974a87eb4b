"""Refusals of the calls around the cache that need no GPU: the C entries answer a null handle
before any CUDA call, and the binding refuses tensors that are not on a GPU."""
import pytest

import bit_paged_kv_diag_b200 as kvq


def test_null_handle_is_refused():
    L = kvq.lib()
    ok = 0x10000
    assert L.kvq_rope_quant_append(None, 0, 0, ok, 1024, ok, 256, ok, 256, ok, ok, None, ok, 1, 1, ok, 128, 0, 1.0, ok,
                                   None) == kvq.KVQ_EINVAL
    assert L.kvq_gather_rows(None, 0, ok, ok, ok, 1, 1, 0, ok, ok, None) == kvq.KVQ_EINVAL
    assert L.kvq_update_block_bounds(None, 0, ok, ok, ok, ok, ok, 1, 1, None) == kvq.KVQ_EINVAL
    assert L.kvq_select_blocks(None, 0, ok, ok, ok, ok, ok, ok, 1, 1, 4, 1, 1, ok, None) == kvq.KVQ_EINVAL
    assert L.kvq_sparse_attention(None, 0, ok, ok, ok, ok, ok, 4, 1, 1, 0.0, ok, None) == kvq.KVQ_EINVAL


def test_host_tensors_are_refused():
    import torch
    cache = kvq.Cache(None, kvq.Desc(1, 2, 4, 128, 64, 16, 4, 1, 4), None, 0)
    x, q = torch.zeros(1, 2, 128, dtype=torch.float16), torch.zeros(1, 4, 128, dtype=torch.float16)
    i, t = torch.zeros(1, dtype=torch.int32), torch.zeros(1, 4, dtype=torch.int32)
    cu, blocks = torch.zeros(2, dtype=torch.int32), torch.zeros(1, 2, 3, dtype=torch.int32)
    with pytest.raises(TypeError):
        kvq.Rope(torch.ones(64))
    with pytest.raises(TypeError):
        kvq.BlockBounds(torch.zeros(1, 4, 2, 2, 128, dtype=torch.int8), torch.zeros(1, 4, 2))
    rope = kvq.Rope.__new__(kvq.Rope)
    rope.rotary_dim, rope.interleaved, rope.factor = 128, False, 1.0
    with pytest.raises(TypeError):
        kvq.rope_quant_append(cache, 0, x, x, cu, i, t, rope, q=q)
    with pytest.raises(TypeError):
        kvq.gather_rows(cache, 0, cu, i, t, 1)
    with pytest.raises(TypeError):
        kvq.sparse_attention(cache, 0, q, i, t, blocks)
