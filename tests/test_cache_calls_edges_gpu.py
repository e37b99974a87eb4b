"""Calls around the cache that the documentation allows and that are easily answered wrongly (GPU)."""
import pytest

from test_sparse_ops_gpu import D, Setup

pytestmark = pytest.mark.gpu


def test_tensors_set_again_between_calls():
    """The append and the bounds of tensors that were set again are those of new objects."""
    import torch
    s = Setup([0, 30], [50, 20], 2, 4, 64, 16, 0)
    kvq, cu, lens = s.kvq, s.dev(s.cu), s.dev(s.before)
    q, k, v = (torch.randn(s.T, n, D, device="cuda").half() for n in (8, 2, 2))
    freqs = [(1e4 ** -(torch.arange(0, rd, 2, device="cuda") / rd)).float() for rd in (128, 64, 96)]
    rope, bounds = kvq.Rope(freqs[0].clone()), kvq.BlockBounds.alloc(s.cache)
    for i, f in enumerate(freqs):
        want_q = kvq.rope_quant_append(s.cache, 0, k, v, cu, lens, s.pt, kvq.Rope(f), q=q)
        want, fresh = s.pool.clone(), kvq.BlockBounds.alloc(s.cache)
        kvq.update_block_bounds(s.cache, 0, fresh, cu, lens, s.pt, s.T)
        s.pool.zero_()
        if i == 1:
            rope.inv_freq = f.clone()
            bounds.codes = torch.zeros_like(bounds.codes)
            bounds.scale = torch.zeros_like(bounds.scale)
        elif i == 2:  # in place
            rope.inv_freq.set_(f.clone())
            bounds.codes.set_(torch.zeros_like(bounds.codes))
        got_q = kvq.rope_quant_append(s.cache, 0, k, v, cu, lens, s.pt, rope, q=q)
        kvq.update_block_bounds(s.cache, 0, bounds, cu, lens, s.pt, s.T)
        assert torch.equal(got_q, want_q) and torch.equal(s.pool, want)
        assert torch.equal(bounds.codes, fresh.codes) and torch.equal(bounds.scale, fresh.scale)
    assert s.status() == 0
