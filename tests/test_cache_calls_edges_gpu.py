"""Calls around the cache that the documentation allows and that are easily answered wrongly (GPU)."""
import numpy as np
import pytest

from test_sparse_ops_gpu import D, Setup, _filled_bounds

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


@pytest.mark.parametrize("n,fused", [(1, True), (1, False), (19, False), (700, False)])
@pytest.mark.parametrize("fmt", [0, 1])
def test_outputs_of_a_call_feed_an_append(n, fused, fmt):
    """q' of the rotating append, attention outputs and rows read back are the k and v of an append
    or of a fused step that follows at once on the stream."""
    import torch
    B, hkv = 6, 4
    s = Setup([900, 40, 0, 333, 2000, 17], [n] * B, hkv, 1, 64, 64, fmt, layers=2, layer=0).fill()
    kvq, cu, lens, after = s.kvq, s.dev(s.cu), s.dev(s.before), s.dev(s.after)
    x, y = (torch.randn(s.T, hkv, D, device="cuda").half() for _ in range(2))
    rope = kvq.Rope((1e4 ** -(torch.arange(0, 128, 2, device="cuda") / 128)).float())
    blocks = torch.zeros(s.T, hkv, 8, dtype=torch.int32, device="cuda")
    blocks[:] = torch.arange(8, dtype=torch.int32, device="cuda")
    k, v, q = torch.empty_like(x), torch.empty_like(x), torch.ones(B, hkv, D, device="cuda").half()
    out = torch.empty_like(q)

    def rotated():
        kvq.rope_quant_append(s.cache, 0, x, y, cu, lens, s.pt, rope, q=x, q_out=k)
        v.copy_(y)
        kvq.rope_quant_append(s.cache, 0, x, y, cu, lens, s.pt, rope, q=y, q_out=v)

    def attended():
        kvq.sparse_attention(s.cache, 0, x, after, s.pt, blocks, cu_q=cu, out=k)
        kvq.prefill_attention(s.cache, 0, y, cu, after, s.pt, out=v)

    def read_back():
        kvq.gather_rows(s.cache, 0, cu, lens, s.pt, s.T, k_out=k, v_out=v)

    def append():
        if fused:
            kvq.append_decode_attention(s.cache, 1, k, v, q, lens, s.pt, out=out)
        else:
            kvq.rotate_quant_append(s.cache, 1, k, v, cu, lens, s.pt)

    for make in (rotated, attended, read_back):
        got = []
        for wait in (False, False, True):
            k.zero_(), v.zero_(), s.pool[s.pool.numel() // 2:].zero_()
            make()
            if wait:
                torch.cuda.synchronize()
            append()
            got.append((s.pool.clone(), out.clone()))
        for pool, o in got[:2]:
            assert torch.equal(pool, got[2][0]) and (not fused or torch.equal(o, got[2][1])), make.__name__
    assert s.status() == 0


@pytest.mark.parametrize("group,page", [(1, 16), (4, 64)])
def test_rows_of_a_bad_sequence_are_zeros(group, page):
    """A sequence shorter than its chunk, longer than its table or of a negative length: all of its
    rows are zeros, whatever their own positions and lists; the others' are what they are without it."""
    import torch
    s = Setup([30, 30, 30, 30, 30], [3, 4, 3, 3, 2], 2, group, 64, page, 0).fill()
    kvq, cap = s.kvq, s.width * page
    cu, q = s.dev(s.cu), torch.randn(s.T, s.hq, D, device="cuda").half()
    blocks = torch.zeros(s.T, s.hkv, 2, dtype=torch.int32, device="cuda")
    blocks[:, :, 1] = 1
    want = kvq.sparse_attention(s.cache, 0, q, s.dev(s.after), s.pt, blocks, cu_q=cu)
    assert s.status() == 0 and want.any(-1).all()
    lens = s.after.copy()
    lens[0], lens[1], lens[3] = 2, cap + 2, -1  # (2: a row of it has a position; cap + 2: two rows are inside)
    bad = np.isin(s.seq, (0, 1, 3))
    out = kvq.sparse_attention(s.cache, 0, q, s.dev(lens), s.pt, blocks, cu_q=cu).cpu()
    assert s.status() == kvq.KVQ_DEV_BAD_POS
    assert not out[bad].any() and torch.equal(out[~bad], want.cpu()[~bad])
    # One query per sequence: an empty sequence is not a bad one.
    lens = np.array([0, cap + 1, -5, cap, 1], np.int32)
    full = np.array([33, 33, 33, cap, 1], np.int32)
    want = kvq.sparse_attention(s.cache, 0, q[:5].contiguous(), s.dev(full), s.pt, blocks[:5].contiguous()).cpu()
    assert s.status() == 0
    out = kvq.sparse_attention(s.cache, 0, q[:5].contiguous(), s.dev(lens), s.pt, blocks[:5].contiguous()).cpu()
    assert s.status() == kvq.KVQ_DEV_BAD_POS
    assert not out[:3].any() and torch.equal(out[3:], want[3:]) and out[3:].any(-1).all()


@pytest.mark.parametrize("hkv,group,before,new,chunk", [
    (1, 1, [4000, 900], [1, 1], False), (2, 4, [4000, 900], [1, 1], False), (1, 8, [30000], [1], False),
    (2, 2, [4000, 900], [20, 30], True), (1, 4, [600], [5], True)])
def test_queries_without_a_score_keep_the_first_and_last_pages(hkv, group, before, new, chunk):
    """No score of a query with a NaN in every head is a number: its pages are the first, the last
    and, all others being equal, the lowest.  The other queries' do not change."""
    import torch
    s = Setup(before, new, hkv, group, 64, 16, 0).fill()
    bounds, *_ = _filled_bounds(s, s.host())
    q = torch.randn(s.T, s.hq, D, device="cuda").half()

    def choose(q):
        return s.kvq.select_blocks(s.cache, 0, q, s.dev(s.after), s.pt, bounds, 10, cu_q=s.dev(s.cu) if chunk else None,
                                   sink=2, recent=3).cpu().numpy()

    want, nan = choose(q), np.arange(s.T) % 3 == 0
    bad = q.clone()
    bad[torch.from_numpy(nan).cuda(), :, 17] = float("nan")
    got = choose(bad)
    for t in range(s.T):
        n = int(s.pos[t]) // 16 + 1
        if nan[t]:
            assert (got[t] == [0, 1, 2, 3, 4, 5, 6, n - 3, n - 2, n - 1]).all(), (t, got[t])
        else:
            assert np.array_equal(got[t], want[t])
    assert s.status() == 0


def test_widest_page_table():
    """The last accepted width of a page table chooses as an exact one does; the next is refused."""
    import torch
    widest = 50048
    s = Setup([3000], [1], 1, 4, 64, 16, 0).fill()
    bounds, *_ = _filled_bounds(s, s.host())
    q, after = torch.randn(1, 4, D, device="cuda").half(), s.dev(s.after)
    want = s.kvq.select_blocks(s.cache, 0, q, after, s.pt, bounds, 9)
    for width in (widest, widest + 1):
        d = s.kvq.Desc(1, 1, 4, D, 64, 16, s.pages, 1, width, 0)
        cache, _ = s.kvq.alloc_pages(d, pool=s.pool)
        table = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
        table[:, :s.width] = s.pt
        if width == widest:
            assert torch.equal(s.kvq.select_blocks(cache, 0, q, after, table, bounds, 9), want)
            cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
            assert torch.equal(s.kvq.select_blocks(cache, 0, q, after, table, bounds, 9, cu_q=cu), want)
        else:
            with pytest.raises(s.kvq.KVQError) as e:
                s.kvq.select_blocks(cache, 0, q, after, table, bounds, 9)
            assert e.value.status == s.kvq.KVQ_EUNSUPPORTED
        assert s.kvq.get_device_status(cache) == 0
        cache.close()
