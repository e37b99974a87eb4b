"""The position-rotating append, the read-back of rows, page bounds, page choice and attention
over chosen pages against plain numpy implementations (sparse_ref.py), and a run of them together
(GPU)."""
import math

import numpy as np
import pytest

import sparse_ref as ref

pytestmark = pytest.mark.gpu
D = 128
MAX_FLIP_FRACTION = 1e-5  # codes a step away: an angle's cosine may round apart by one fp32 step


class Setup:
    """A cache with shuffled pages and ragged sequences; `before` tokens are cached already."""

    def __init__(self, before, new, hkv=2, group=4, block=128, page=16, fmt=0, layers=1, layer=0, seed=0,
                 extra=0, spare=3):
        import torch
        import bit_paged_kv_diag_b200 as kvq
        self.kvq, self.torch = kvq, torch
        self.rng = np.random.default_rng(seed)
        self.before, self.new = np.asarray(before, np.int32), np.asarray(new, np.int32)
        self.after = self.before + self.new
        self.hkv, self.group, self.hq, self.block, self.page, self.fmt = hkv, group, hkv * group, block, page, fmt
        self.layer, self.layers, self.batch = layer, layers, len(self.before)
        need = (self.after + page - 1) // page
        self.pages = int(need.sum()) + spare
        self.width = max(1, int(need.max())) + extra
        self.desc = kvq.Desc(layers, hkv, self.hq, D, block, page, self.pages, self.batch, self.width, fmt)
        self.pool = torch.zeros(kvq.pool_bytes(self.desc), dtype=torch.uint8, device="cuda")
        self.cache, self.table = kvq.alloc_pages(self.desc, self.after, self.rng.permutation(self.pages),
                                                 pool=self.pool)
        self.pt = torch.from_numpy(self.table).cuda()
        self.cu = np.concatenate(([0], np.cumsum(self.new))).astype(np.int32)
        self.T = int(self.cu[-1])
        self.H = ref.hadamard(block)
        self.seq = np.repeat(np.arange(self.batch), self.new)
        self.pos = np.concatenate([np.arange(b, a) for b, a in zip(self.before, self.after)] + [[]]).astype(np.int64)

    def dev(self, a):
        return self.torch.as_tensor(np.ascontiguousarray(a)).cuda()

    def rows(self, n, heads):
        x = self.rng.standard_normal((n, heads, D)).astype(np.float32)
        x[:, :, 5] *= 30
        return x * np.exp(0.5 * self.rng.standard_normal((n, heads, 1))).astype(np.float32)

    def fill(self):
        """Every slot of the layer holds a quantised row (written by hand, not by the append)."""
        lb = self.pool.numel() // self.layers
        raw = np.zeros((self.pages, self.hkv, lb // self.pages // self.hkv), np.uint8)
        P = ref.Pool(raw, self.hkv, self.page, self.fmt)
        for kv in range(2):
            y = ref.butterfly32(self.rows(self.pages * self.page, self.hkv), self.block)
            c, s = ref.quantise(y, self.fmt)
            shape = (self.pages, self.page, self.hkv, -1)
            P.parts[kv][...] = (c[..., 0::2] | (c[..., 1::2] << 4)).astype(np.uint8).reshape(shape).transpose(0, 2, 1, 3)
            P.parts[2 + kv][...] = s.reshape(shape).transpose(0, 2, 1, 3)
        w = 8 if self.fmt else 2
        raw = np.concatenate([x.reshape(self.pages, self.hkv, -1) for x in P.parts], -1)
        assert raw.shape[-1] == self.page * (D + 2 * w)
        self.pool[self.layer * lb:(self.layer + 1) * lb] = self.dev(raw.reshape(-1))
        return self

    def host(self):
        lb = self.pool.numel() // self.layers
        return ref.Pool(self.pool[self.layer * lb:(self.layer + 1) * lb].cpu().numpy(), self.hkv, self.page, self.fmt)

    def status(self):
        return self.kvq.get_device_status(self.cache)


def _filled_bounds(s, P):
    """Bounds of every page of the sequences after the call, written to a BlockBounds."""
    bd = s.kvq.BlockBounds.alloc(s.cache)
    lo = np.zeros((s.pages, s.hkv, D), int)
    hi, sg = np.zeros_like(lo), np.zeros((s.pages, s.hkv))
    k = P.values(0)
    for b in range(s.batch):
        for i in range((int(s.after[b]) + s.page - 1) // s.page):
            pg = s.table[b, i]
            for h in range(s.hkv):
                lo[pg, h], hi[pg, h], sg[pg, h] = ref.bounds(k[pg, h], min(s.page, int(s.after[b]) - i * s.page))
    bd.codes[s.layer] = s.dev(np.stack((lo, hi), 2).astype(np.int8))
    bd.scale[s.layer] = s.dev(sg.astype(np.float32))
    return bd, lo, hi, sg


# ------------------------------------------------------------------------------- append --
APPENDS = [
    # before, new, hkv, group, block, page, fmt, dtype, rd, interleaved, factor, with q
    ([0], [1], 1, 1, 128, 16, 0, "float16", 128, False, 1.0, True),
    ([5, 0, 130000, 31], [1, 0, 1, 1], 8, 4, 128, 16, 0, "float16", 128, False, 1.0, True),
    ([0, 17, 63], [37, 1, 90], 2, 8, 64, 32, 1, "bfloat16", 64, True, 1.25, True),
    ([3, 250], [260, 5], 3, 2, 32, 64, 0, "bfloat16", 96, False, 1.0, True),
    ([0, 0], [129, 64], 5, 4, 1, 128, 1, "float16", 16, True, 1.0, True),
    ([100, 7], [33, 200], 4, 1, 1, 256, 0, "float16", 32, False, 0.5, False),
    ([64] * 9, [3] * 9, 1, 8, 128, 16, 1, "float16", 112, True, 1.0, True),
    ([0], [2048], 2, 4, 64, 64, 0, "float16", 128, True, 1.0, True),
]


@pytest.mark.parametrize("case", APPENDS)
@pytest.mark.parametrize("packed", [True, False])
def test_rope_append(case, packed):
    before, new, hkv, group, block, page, fmt, dtype, rd, inter, factor, with_q = case
    s = Setup(before, new, hkv, group, block, page, fmt, layers=2, layer=1, extra=2)
    torch, kvq = s.torch, s.kvq
    pad = 3  # tokens behind the last sequence
    T = s.T + pad
    x = np.concatenate((s.rng.standard_normal((T, s.hq, D)).astype(np.float32), s.rows(T, hkv), s.rows(T, hkv)), 1)
    x = torch.from_numpy(x).to(getattr(torch, dtype))
    inv = (1e6 ** -(np.arange(0, rd, 2) / rd)).astype(np.float32)
    rope = kvq.Rope(s.dev(inv), interleaved=inter, factor=factor)
    d = x.cuda()
    q, k, v = d.split([s.hq, hkv, hkv], 1)  # slices of one buffer: tokens are a stride apart
    if not packed:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    positions = None
    pos = s.pos
    if packed and with_q:  # angles of other positions than the slots'
        pos = s.pos[::-1] * 3 % 70000
        positions = s.dev(np.concatenate((pos, [0] * pad)).astype(np.int32))
    out = torch.full((T, s.hq, D), 7.0, dtype=torch.float16, device="cuda") if with_q else None
    got = kvq.rope_quant_append(s.cache, 1, k, v, s.dev(s.cu), s.dev(s.before), s.pt, rope, q=q if with_q else None,
                                positions=positions, q_out=out)
    assert got is out and s.status() == 0
    xf = x.float().numpy()[: s.T]
    kk = ref.butterfly32(ref.rope32(xf[:, s.hq: s.hq + hkv], pos, inv, inter, factor), block)
    vv = ref.butterfly32(xf[:, s.hq + hkv:], block)
    P = s.host()
    touched = np.zeros((s.pages, s.page), bool)
    pg, sl = s.table[s.seq, s.pos // page], s.pos % page
    touched[pg, sl] = True
    flips = total = 0
    for kv, y in ((0, kk), (1, vv)):
        c, sc = ref.quantise(y, fmt)
        assert np.array_equal(P.parts[2 + kv][pg, :, sl], sc), "scales"
        dc = np.abs(P.codes(kv)[pg, :, sl] - c)
        flips, total = flips + np.count_nonzero(dc), total + dc.size
        if kv == 1:
            assert not dc.any(), "V has no angle: exact"
    assert flips <= MAX_FLIP_FRACTION * total
    for part in P.parts:  # nothing else of the layer is written
        assert not part.transpose(0, 2, 1, 3)[~touched].any()
    assert not s.pool[: s.pool.numel() // 2].any(), "the other layer"
    if with_q:
        o = out.float().cpu().numpy()
        assert (o[s.T:] == 7).all(), "rows behind the last sequence"
        xq = xf[:, : s.hq].astype(np.float64)
        want = ref.rope64(xq, pos, inv, inter, factor)
        # c, s, the products and the sum round by 2^-24 each in fp32; the store by 2^-11.
        a = np.abs(xq)
        half = rd // 2
        pair = a.copy()
        ia, ib = (slice(0, rd, 2), slice(1, rd, 2)) if inter else (slice(0, half), slice(half, rd))
        pair[..., ia], pair[..., ib] = a[..., ia] + a[..., ib], a[..., ia] + a[..., ib]
        tol = 2.0 ** -11 * np.abs(want) + 2.0 ** -25 + 3.1 * 2.0 ** -24 * pair * max(factor, 1)
        assert (np.abs(o[: s.T] - want) <= tol).all()


@pytest.mark.parametrize("fmt,block,page", [(0, 128, 16), (1, 64, 64), (0, 1, 256), (1, 32, 32)])
def test_rope_append_without_angles_is_the_plain_append(fmt, block, page):
    """Position 0 turns nothing: the pool is the one rotate_quant_append writes, bit for bit."""
    a, b = (Setup([9, 0, 40], [77, 1, 300], 4, 2, block, page, fmt) for _ in range(2))
    torch = a.torch
    k, v = (a.dev(a.rows(a.T, 4).astype(np.float16)) for _ in range(2))
    k[3], v[5] = 0, 0
    k[7] *= 1000
    rope = a.kvq.Rope(torch.ones(64, device="cuda"))
    zeros = torch.zeros(a.T, dtype=torch.int32, device="cuda")
    a.kvq.rope_quant_append(a.cache, 0, k, v, a.dev(a.cu), a.dev(a.before), a.pt, rope, positions=zeros)
    b.kvq.rotate_quant_append(b.cache, 0, k, v, b.dev(b.cu), b.dev(b.before), b.pt)
    assert torch.equal(a.pool, b.pool) and a.status() == 0


@pytest.mark.parametrize("fmt", [0, 1])
def test_rope_append_large_and_zero_rows(fmt):
    """bf16 rows beyond the scales' range (they saturate), tiny ones and zeros."""
    s = Setup([3], [40], 2, 2, 64, 16, fmt)
    torch = s.torch
    x = s.rng.standard_normal((40, 2, D)).astype(np.float32)
    x *= (10.0 ** s.rng.integers(-30, 30, (40, 2, 1))).astype(np.float32)
    x[7] = 0
    k = torch.from_numpy(x).bfloat16()
    s.kvq.rope_quant_append(s.cache, 0, k.cuda(), k.cuda(), s.dev(s.cu), s.dev(s.before), s.pt,
                            s.kvq.Rope(torch.ones(64, device="cuda")),
                            positions=torch.zeros(40, dtype=torch.int32, device="cuda"))
    c, sc = ref.quantise(ref.butterfly32(k.float().numpy(), 64), fmt)
    P = s.host()
    pg, sl = s.table[0, s.pos // 16], s.pos % 16
    for kv in range(2):
        assert np.array_equal(P.parts[2 + kv][pg, :, sl], sc) and np.array_equal(P.codes(kv)[pg, :, sl], c)


# --------------------------------------------------------------------------------- rows --
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("block,page,hkv,starts,lens", [
    (128, 16, 2, [0], [1]), (64, 64, 1, [5, 100, 0], [70, 0, 33]), (32, 32, 8, [31, 1], [2, 500]),
    (1, 256, 3, [250, 0], [20, 257]), (128, 128, 4, [0] * 5, [15, 16, 17, 1, 300])])
def test_gather_rows(dtype, fmt, block, page, hkv, starts, lens):
    s = Setup(starts, lens, hkv, 2, block, page, fmt, layers=2, layer=1).fill()
    torch, dt = s.torch, getattr(s.torch, dtype)
    shape = (s.T + 2, hkv, D)
    k, v = (torch.full(shape, 7.0, dtype=dt, device="cuda") for _ in range(2))
    got = s.kvq.gather_rows(s.cache, 1, s.dev(s.cu), s.dev(s.before), s.pt, s.T + 2, dtype=dt, k_out=k, v_out=v)
    assert got[0] is k and got[1] is v and s.status() == 0
    P = s.host()
    half = {"float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}[dtype]
    for kv, out in ((0, k), (1, v)):
        o = out.double().cpu().numpy()
        assert (o[s.T:] == 7).all(), "rows behind the last sequence"
        y = P.values(kv)[s.table[s.seq, s.pos // page], :, s.pos % page]
        want = y @ s.H
        # fp32 after the exact stages: at most 5 roundings of 2^-24 of the block's sum |y| / sqrt(b)
        spread = np.abs(y) @ np.abs(s.H)
        assert (np.abs(o[: s.T] - want) <= half * np.abs(want) + 5 * 2.0 ** -24 * spread + 2.0 ** -25).all()


def test_gather_rows_many_short_and_empty_sequences():
    """More sequences than one probe of the offsets holds, most of them empty."""
    rng = np.random.default_rng(5)
    lens = np.where(rng.random(300) < 0.8, 0, rng.integers(1, 4, 300))
    lens[100:170] = 0
    s = Setup(rng.integers(0, 40, 300), lens, 2, 1, 64, 16, 0).fill()
    k, v = s.kvq.gather_rows(s.cache, 0, s.dev(s.cu), s.dev(s.before), s.pt, s.T)
    P = s.host()
    for kv, out in ((0, k), (1, v)):
        want = P.values(kv)[s.table[s.seq, s.pos // 16], :, s.pos % 16] @ s.H
        assert np.abs(out.double().cpu().numpy() - want).max() <= 2.0 ** -10 * np.abs(want).max()
    # K alone, through the C entry: V is neither read nor written.
    only, cu, before = s.torch.empty_like(k), s.dev(s.cu), s.dev(s.before)
    rc = s.kvq.lib().kvq_gather_rows(s.cache.handle, 0, cu.data_ptr(), before.data_ptr(), s.pt.data_ptr(), 300,
                                     s.T, 0, only.data_ptr(), None,
                                     s.torch.cuda.current_stream().cuda_stream)
    assert rc == s.kvq.KVQ_OK and s.torch.equal(only, k) and s.status() == 0
    # The same sequences as an append and as chunks of queries.
    a, b = (Setup(rng.integers(0, 40, 300) * 0 + 17, lens, 2, 1, 64, 16, 0) for _ in range(2))
    x = a.dev(a.rows(a.T, 2).astype(np.float16))
    zeros = a.torch.zeros(a.T, dtype=a.torch.int32, device="cuda")
    a.kvq.rope_quant_append(a.cache, 0, x, x, a.dev(a.cu), a.dev(a.before), a.pt,
                            a.kvq.Rope(a.torch.ones(64, device="cuda")), positions=zeros)
    b.kvq.rotate_quant_append(b.cache, 0, x, x, b.dev(b.cu), b.dev(b.before), b.pt)
    assert a.torch.equal(a.pool, b.pool) and a.status() == 0


def test_gathered_rows_feed_an_append():
    """A prefix copied to another layer: read back and appended again, one call after the other (the
    append reads its k and v early, so the read-back must have completed)."""
    lens = [9000, 7001]
    s = Setup([0, 0], lens, 8, 1, 64, 64, 0, layers=2, layer=0).fill()
    cu, zero = s.dev(s.cu), s.dev(s.before)
    for _ in range(5):
        k, v = s.kvq.gather_rows(s.cache, 0, cu, zero, s.pt, s.T)
        k.zero_(), v.zero_()
        s.kvq.gather_rows(s.cache, 0, cu, zero, s.pt, s.T, k_out=k, v_out=v)
        s.kvq.rotate_quant_append(s.cache, 1, k, v, cu, zero, s.pt)
        got = s.pool.clone()
        s.torch.cuda.synchronize()
        s.kvq.rotate_quant_append(s.cache, 1, k, v, cu, zero, s.pt)
        assert s.torch.equal(got, s.pool)


# ------------------------------------------------------------------------------- bounds --
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("before,new,hkv", [([0], [1], 1), ([15, 16, 17, 0, 300], [1, 1, 1, 0, 700], 3),
                                            ([0, 255], [513, 2], 8)])
def test_update_block_bounds(fmt, page, before, new, hkv):
    s = Setup(before, new, hkv, 1, 64, page, fmt, layers=2, layer=1).fill()
    P = s.host()
    zero = s.table[0, 0]  # all-zero keys in one page and head: zero codes and scale
    for part in (0, 2):
        P.parts[part][zero, 0] = 0
    lb = s.pool.numel() // 2
    s.pool[lb:] = s.dev(np.concatenate([x.reshape(s.pages, hkv, -1) for x in P.parts], -1).reshape(-1))
    bd = s.kvq.BlockBounds.alloc(s.cache)
    bd.codes.fill_(99)
    bd.scale.fill_(-1.0)
    s.kvq.update_block_bounds(s.cache, 1, bd, s.dev(s.cu), s.dev(s.before), s.pt, s.T)
    assert s.status() == 0
    codes, scale = bd.codes.cpu().numpy(), bd.scale.cpu().numpy()
    assert (codes[0] == 99).all() and (scale[0] == -1).all()
    k, left = P.values(0), np.ones(s.pages, bool)
    for b in range(s.batch):
        if s.new[b] == 0:
            continue
        for i in range(int(s.before[b]) // page, (int(s.after[b]) - 1) // page + 1):
            pg = s.table[b, i]
            left[pg] = False
            for h in range(hkv):
                lo, hi, sg = ref.bounds(k[pg, h], min(page, int(s.after[b]) - i * page))
                assert scale[1, pg, h] == sg
                assert np.array_equal(codes[1, pg, h, 0], lo) and np.array_equal(codes[1, pg, h, 1], hi)
    assert (codes[1][left] == 99).all() and (scale[1][left] == -1).all(), "untouched pages"


# --------------------------------------------------------------------------------- select --
SELECTS = [
    # before, new (query rows), hkv, group, block, page, fmt, num_blocks, sink, recent, chunk call
    ([0], [1], 1, 1, 128, 16, 0, 4, 1, 1, False),
    ([1000, 62, 2, 5000], [1, 1, 1, 1], 2, 4, 64, 16, 1, 8, 1, 2, False),
    ([40000, 2047], [1, 1], 1, 8, 128, 16, 0, 32, 0, 1, False),
    ([4000, 100, 0, 777], [37, 5, 3, 1], 2, 2, 32, 32, 0, 9, 1, 2, True),
    ([900, 3000], [100, 28], 3, 1, 1, 16, 1, 16, 0, 0, True),
    ([3100], [9], 2, 8, 128, 256, 0, 5, 2, 3, True),
    ([2500, 0, 600], [40, 0, 61], 8, 4, 128, 16, 0, 1, 0, 1, True),
    ([6000], [130], 1, 4, 64, 64, 1, 300, 1, 1, True),
    ([9000, 700], [1, 1], 1, 1, 64, 16, 0, 20, 1, 1, False),
    ([4500], [1], 3, 2, 1, 16, 1, 13, 2, 0, False),
    ([1500, 90], [40, 33], 1, 8, 128, 16, 0, 12, 1, 2, True),
    ([1500], [50], 1, 2, 32, 16, 1, 20, 2, 1, True),
    ([1200], [64], 2, 1, 64, 16, 0, 7, 0, 3, True),
    ([70] * 40, [1] * 40, 2, 4, 64, 16, 0, 3, 1, 1, False),
    ([70] * 40, [2] * 40, 1, 2, 64, 16, 0, 3, 1, 1, True),
]


@pytest.mark.parametrize("case", SELECTS)
def test_select_blocks(case):
    before, new, hkv, group, block, page, fmt, nb, sink, recent, chunk = case
    s = Setup(before, new, hkv, group, block, page, fmt, layers=2, layer=1, extra=5).fill()
    P = s.host()
    bd, lo, hi, sg = _filled_bounds(s, P)
    # Ties: runs of pages with the same bounds.
    for b in range(s.batch):
        n = (int(s.after[b]) + page - 1) // page
        for i in range(3, n - 1, 7):
            a, c = s.table[b, i], s.table[b, i - 2]
            lo[a], hi[a], sg[a] = lo[c], hi[c], sg[c]
    bd.codes[1] = s.dev(np.stack((lo, hi), 2).astype(np.int8))
    bd.scale[1] = s.dev(sg.astype(np.float32))
    pad = 2 if chunk else 0
    q = s.rng.standard_normal((s.T + pad, s.hq, D)).astype(np.float16)
    q[0, 0] = 0
    blocks = s.torch.full((s.T + pad, hkv, nb), 77, dtype=s.torch.int32, device="cuda")
    got = s.kvq.select_blocks(s.cache, 1, s.dev(q), s.dev(s.after), s.pt, bd, nb, cu_q=s.dev(s.cu) if chunk else None,
                              sink=sink, recent=recent, blocks=blocks)
    assert got is blocks and s.status() == 0
    o = blocks.cpu().numpy()
    assert (o[s.T:] == 77).all()
    for t in range(s.T):
        b, n = s.seq[t], int(s.pos[t]) // page + 1
        for h in range(hkv):
            pg = s.table[b, :n]
            want = ref.choose(q[t, h * group:(h + 1) * group], block, lo[pg, h], hi[pg, h], sg[pg, h], n, nb, sink, recent)
            assert np.array_equal(o[t, h], want), (t, h, o[t, h], want)


@pytest.mark.parametrize("extra,new,chunk", [(20000, [19], True), (49000, [1], False)])
def test_select_blocks_wide_page_table(extra, new, chunk):
    """A page table far wider than the sequences: the scores of fewer queries fit at a time."""
    a, b = (Setup([3000], new, 1, 4, 64, 16, 0, extra=x).fill() for x in (extra, 0))
    q = a.rng.standard_normal((a.T, 4, D)).astype(np.float16)
    out = []
    for s in (a, b):
        bd, *_ = _filled_bounds(s, s.host())
        out.append(s.kvq.select_blocks(s.cache, 0, s.dev(q), s.dev(s.after), s.pt, bd, 9,
                                       cu_q=s.dev(s.cu) if chunk else None))
        assert s.status() == 0
    assert a.torch.equal(*out)


def test_select_blocks_all_scores_equal_takes_the_lowest_pages():
    for new, chunk in (([1, 1], False), ([20, 30], True)):
        s = Setup([4000, 900], new, 2, 2, 64, 16, 0)
        bd = s.kvq.BlockBounds.alloc(s.cache)  # zero bounds: every score 0
        q = s.torch.randn(s.T, s.hq, D, device="cuda").half()
        o = s.kvq.select_blocks(s.cache, 0, q, s.dev(s.after), s.pt, bd, 10, cu_q=s.dev(s.cu) if chunk else None,
                                sink=2, recent=3).cpu().numpy()
        for t in range(s.T):
            n = int(s.pos[t]) // 16 + 1
            want = list(range(7)) + [n - 3, n - 2, n - 1]
            assert (o[t] == want).all()


# --------------------------------------------------------------------------------- sparse --
def _check_sparse(s, P, q, blocks, out, scale=1 / math.sqrt(D)):
    k, v = P.values(0), P.values(1)
    o = out.double().cpu().numpy()
    worst = 0.0
    for t in range(s.T):
        b, p = s.seq[t], int(s.pos[t])
        for h in range(s.hkv):
            at = np.concatenate([np.arange(j * s.page, min((j + 1) * s.page, p + 1)) for j in blocks[t, h].tolist()
                                 if j >= 0 and j * s.page <= p] + [np.zeros(0, int)]).astype(int)
            got = o[t, h * s.group:(h + 1) * s.group]
            if at.size == 0:
                assert (got == 0).all()
                continue
            pg = s.table[b, at // s.page]
            want, tol = ref.attend(q[t, h * s.group:(h + 1) * s.group], s.H, k[pg, h, at % s.page], v[pg, h, at % s.page],
                                   scale)
            worst = max(worst, float((np.abs(got - want) / tol).max()))
    assert worst <= 1, worst


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("group", [1, 2, 4, 8])
@pytest.mark.parametrize("page,block", [(16, 128), (32, 64), (64, 32), (256, 1)])
def test_sparse_attention(fmt, group, page, block):
    """Lists in any order with empty, later and partly filled pages, rows without any page, a
    query at position 0; one query per sequence, and chunks."""
    hkv = 2
    for new, chunk in (([1] * 5, False), ([30, 1, 0, 7, 50], True)):
        s = Setup([3000, 0, 16, 700, 255], new, hkv, group, block, page, fmt, layers=2, layer=1, extra=3,
                  seed=group).fill()
        pad = 2 if chunk else 0
        nb = 11
        n = s.pos // page + 1
        blocks = np.full((s.T + pad, hkv, nb), -1, np.int32)
        for t in range(s.T):
            for h in range(hkv):
                kind = s.rng.integers(4)
                m = min(nb, int(n[t]))
                pick = s.rng.permutation(int(n[t]))[:m]
                if kind == 1:
                    pick = pick[: m // 2]
                elif kind == 2:  # pages behind the position, far pages, other negatives
                    pick = np.concatenate((pick[: nb - 4], [int(n[t]), 2 ** 30, -5, -2 ** 31]))
                elif kind == 3 and t % 3 == 0:
                    pick = pick[:0]
                row = np.full(nb, -1, np.int64)
                row[s.rng.permutation(nb)[: len(pick)]] = pick
                blocks[t, h] = row
        q = s.rng.standard_normal((s.T + pad, s.hq, D)).astype(np.float16)
        out = s.torch.full((s.T + pad, s.hq, D), 7.0, dtype=s.torch.float16, device="cuda")
        got = s.kvq.sparse_attention(s.cache, 1, s.dev(q), s.dev(s.after), s.pt, s.dev(blocks),
                                     cu_q=s.dev(s.cu) if chunk else None, out=out)
        assert got is out and s.status() == 0
        assert (out[s.T:] == 7).all()
        _check_sparse(s, s.host(), q, blocks, out)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("page,nb,before,new,hkv,group", [
    (64, 64, [9000, 4095], [1, 1], 2, 4),      # parts of a unit joined over CTAs
    (16, 300, [20000], [1], 1, 8),
    (128, 40, [6000], [1], 1, 1),
    (32, 1, [500, 31], [1, 1], 3, 2),
    (16, 1, [200], [40], 1, 8),
])
def test_sparse_attention_long_lists(fmt, page, nb, before, new, hkv, group):
    s = Setup(before, new, hkv, group, 128, page, fmt).fill()
    n = s.pos // page + 1
    blocks = np.full((s.T, hkv, nb), -1, np.int32)
    for t in range(s.T):
        for h in range(hkv):
            m = min(nb, int(n[t]))
            blocks[t, h, :m] = np.sort(s.rng.permutation(int(n[t]))[:m])
    q = (3 * s.rng.standard_normal((s.T, s.hq, D))).astype(np.float16)
    cu = None if max(new) == 1 else s.dev(s.cu)
    args = (s.cache, 0, s.dev(q), s.dev(s.after), s.pt, s.dev(blocks))
    out = s.kvq.sparse_attention(*args, cu_q=cu, softmax_scale=0.125)
    assert s.status() == 0
    _check_sparse(s, s.host(), q, blocks, out, 0.125)
    for _ in range(3):  # the joined parts do not depend on the order in which CTAs arrive
        assert s.torch.equal(out, s.kvq.sparse_attention(*args, cu_q=cu, softmax_scale=0.125))


def test_sparse_attention_ignores_rows_past_the_sequence():
    """Slots behind a sequence's end hold infinities and NaN: they must not reach an output."""
    for fmt in (0, 1):
        for page in (16, 64):
            s = Setup([page + 5], [1], 1, 4, 64, page, fmt).fill()
            P = s.host()
            pg = s.table[0, 1]
            for part in (2, 3):  # fp16 NaN / E4M3 NaN
                P.parts[part][pg, 0, 6:] = 0x7F
            s.pool[:] = s.dev(np.concatenate([x.reshape(s.pages, 1, -1) for x in P.parts], -1).reshape(-1))
            q = s.rng.standard_normal((1, 4, D)).astype(np.float16)
            blocks = np.array([[[1, 0]]], np.int32)
            out = s.kvq.sparse_attention(s.cache, 0, s.dev(q), s.dev(s.after), s.pt, s.dev(blocks))
            _check_sparse(s, s.host(), q, blocks, out)


# --------------------------------------------------------------------------------- together --
@pytest.mark.parametrize("fmt,page,block", [(0, 16, 128), (1, 64, 64)])
def test_run_together(fmt, page, block):
    """A prompt in two chunks, then decode steps: rope_quant_append, update_block_bounds,
    select_blocks and sparse_attention on a side stream; with lists that hold every page the
    outputs are those of the dense calls on the same cache; the steps captured into a graph and
    replayed give the same bytes."""
    import torch
    import bit_paged_kv_diag_b200 as kvq
    hkv, group, steps = 2, 4, 3
    prompt = [150, 67, 300]
    S = Setup([0, 0, 0], np.array(prompt) + steps + 1, hkv, group, block, page, fmt, seed=3)
    inv = S.dev((1e4 ** -(np.arange(0, D, 2) / D)).astype(np.float32))
    rope, bounds = kvq.Rope(inv), kvq.BlockBounds.alloc(S.cache)
    nb = S.width
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.Generator(device="cuda").manual_seed(1)

    def qkv(T):
        return torch.randn(T, S.hq + 2 * hkv, D, device="cuda", generator=g).half().split([S.hq, hkv, hkv], 1)

    with torch.cuda.stream(side):
        lens = torch.zeros(3, dtype=torch.int32, device="cuda")
        for cut in (50, None):
            new = torch.tensor([min(50, n) if cut else n - min(50, n) for n in prompt], dtype=torch.int32)
            cu = torch.cat((torch.zeros(1, dtype=torch.int32), new.cumsum(0).int())).cuda()
            T = int(new.sum())
            q, k, v = qkv(T)
            qr = kvq.rope_quant_append(S.cache, 0, k, v, cu, lens, S.pt, rope, q=q)
            kvq.update_block_bounds(S.cache, 0, bounds, cu, lens, S.pt, T)
            after = lens + new.cuda()
            blocks = kvq.select_blocks(S.cache, 0, qr, after, S.pt, bounds, nb, cu_q=cu)
            o = kvq.sparse_attention(S.cache, 0, qr, after, S.pt, blocks, cu_q=cu)
            dense = kvq.prefill_attention(S.cache, 0, qr, cu, after, S.pt)
            assert torch.allclose(o.float(), dense.float(), atol=2e-3, rtol=1e-2)
            few = kvq.select_blocks(S.cache, 0, qr, after, S.pt, bounds, 3, cu_q=cu)
            assert torch.equal(few[..., 0], torch.where(few[..., 0] >= 0, 0, -1)) and (few < S.width).all()
            lens = after
        one = torch.arange(4, dtype=torch.int32, device="cuda")
        q, k, v = (x.contiguous() for x in qkv(3))
        last = lens + 1

        def step():
            qr = kvq.rope_quant_append(S.cache, 0, k, v, one, lens, S.pt, rope, q=q)
            kvq.update_block_bounds(S.cache, 0, bounds, one, lens, S.pt, 3)
            blocks = kvq.select_blocks(S.cache, 0, qr, last, S.pt, bounds, 4, sink=1, recent=1)
            return qr, blocks, kvq.sparse_attention(S.cache, 0, qr, last, S.pt, blocks)

        first = [x.clone() for x in step()]
        pool, codes = S.pool.clone(), bounds.codes.clone()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            res = step()
        for n in range(steps):
            graph.replay()
            if n == 0:
                for a, b in zip(first, res):
                    assert torch.equal(a, b)
                assert torch.equal(pool, S.pool) and torch.equal(codes, bounds.codes)
            eager = step()
            graph.replay()
            for a, b in zip(eager, res):
                assert torch.equal(a, b)
            full = kvq.sparse_attention(S.cache, 0, res[0], last, S.pt,
                                        torch.arange(nb, dtype=torch.int32, device="cuda").expand(3, hkv, nb).contiguous())
            dense = kvq.decode_attention(S.cache, 0, res[0], last, S.pt)
            assert torch.allclose(full.float(), dense.float(), atol=2e-3, rtol=1e-2)
            lens += 1  # the graph reads the new lengths, keys and queries
            last += 1
            q.copy_(torch.randn(q.shape, device="cuda", generator=g))
            k.copy_(torch.randn(k.shape, device="cuda", generator=g))
        ko, vo = kvq.gather_rows(S.cache, 0, one, lens - 1, S.pt, 3)
    side.synchronize()
    assert S.status() == 0
    P = S.host()
    for b in range(3):
        p = int(lens[b]) - 1
        for kv, got in ((0, ko), (1, vo)):
            want = P.values(kv)[S.table[b, p // page], :, p % page] @ S.H
            assert np.abs(got[b].double().cpu().numpy() - want).max() <= 2.0 ** -10 * np.abs(want).max()


def test_pool_beyond_32_bit_offsets():
    """The same calls on a pool of more than 4 GiB, with the sequences in its last pages."""
    import torch
    import bit_paged_kv_diag_b200 as kvq
    hkv, group, page, block = 2, 4, 64, 64
    lens = [400, 130]
    rng = np.random.default_rng(2)
    pages = (1 << 32) // (hkv * page * 132) + 40
    need = [(n + page) // page + 1 for n in lens]
    k, v = (torch.from_numpy(rng.standard_normal((sum(lens), hkv, D)).astype(np.float16)).cuda() for _ in range(2))
    q = torch.from_numpy(rng.standard_normal((sum(lens), hkv * group, D)).astype(np.float16)).cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    cu, zero = torch.tensor([0, lens[0], sum(lens)], **i32), torch.zeros(2, **i32)
    after = torch.tensor(lens, **i32)
    last = torch.tensor([lens[0] - 1, sum(lens) - 1], device="cuda")
    rope = kvq.Rope(torch.ones(64, device="cuda") * 0.01)
    got = []
    for n in (sum(need), pages):
        d = kvq.Desc(1, hkv, hkv * group, D, block, page, n, 2, max(need), 0)
        pool = torch.empty(kvq.pool_bytes(d), dtype=torch.uint8, device="cuda")
        order = np.arange(n - 1, -1, -1, dtype=np.int32)
        cache, table = kvq.alloc_pages(d, np.array(lens, np.int32), order, pool=pool)
        pt, bd = torch.from_numpy(table).cuda(), kvq.BlockBounds.alloc(cache)
        qr = kvq.rope_quant_append(cache, 0, k, v, cu, zero, pt, rope, q=q)
        kvq.update_block_bounds(cache, 0, bd, cu, zero, pt, sum(lens))
        one = qr[last].contiguous()
        blocks = kvq.select_blocks(cache, 0, one, after, pt, bd, 3)
        got.append([qr, *kvq.gather_rows(cache, 0, cu, zero, pt, sum(lens)), blocks,
                    kvq.sparse_attention(cache, 0, one, after, pt, blocks), kvq.decode_attention(cache, 0, one, after, pt)])
        assert kvq.get_device_status(cache) == 0
        cache.close()
        del pool, bd
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_stream_argument():
    """Calls on a given stream, as an object and as an address, while the current one is another."""
    import torch
    s = Setup([100], [1], 2, 4, 64, 16, 0).fill()
    q = torch.randn(1, 8, D, device="cuda").half()
    bd, *_ = _filled_bounds(s, s.host())
    after = s.dev(s.after)
    want = s.kvq.select_blocks(s.cache, 0, q, after, s.pt, bd, 4)
    ref_out = s.kvq.sparse_attention(s.cache, 0, q, after, s.pt, want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for st in (side, side.cuda_stream):
        blocks = s.kvq.select_blocks(s.cache, 0, q, after, s.pt, bd, 4, stream=st)
        out = s.kvq.sparse_attention(s.cache, 0, q, after, s.pt, blocks, stream=st)
        side.synchronize()
        assert torch.equal(out, ref_out) and torch.equal(blocks, want)


# ------------------------------------------------------------------------------- refusals --
def test_refusals():
    import torch
    import bit_paged_kv_diag_b200 as kvq
    s = Setup([5, 9], [2, 1], 2, 4, 64, 16, 0)
    c, i32 = s.cache, dict(dtype=torch.int32, device="cuda")
    T = 3
    q = torch.zeros(T, 8, D, dtype=torch.float16, device="cuda")
    k, v = (torch.zeros(T, 2, D, dtype=torch.float16, device="cuda") for _ in range(2))
    cu, lens, aft = s.dev(s.cu), s.dev(s.before), s.dev(s.after)
    rope, bd = kvq.Rope(torch.ones(64, device="cuda")), kvq.BlockBounds.alloc(c)
    blocks = torch.zeros(T, 2, 4, **i32)

    def status(call):
        with pytest.raises(kvq.KVQError) as e:
            call()
        return e.value.status

    def append(**kw):
        a = dict(k=k, v=v, cu_new_tokens=cu, seq_lens=lens, page_table=s.pt, rope=rope, q=q)
        a.update(kw)
        return kvq.rope_quant_append(c, a.pop("layer", 0), **a)

    for bad in (dict(k=k.float()), dict(v=v.bfloat16()), dict(q=q.cpu()), dict(seq_lens=lens.long())):
        with pytest.raises(TypeError):
            append(**bad)
    for bad in (dict(k=k[:2]), dict(q=q[:, :7]), dict(v=v.transpose(0, 1).contiguous().transpose(0, 1)),
                dict(page_table=s.pt[:1]), dict(cu_new_tokens=cu[:2]), dict(positions=lens),
                dict(q=None, q_out=q)):
        with pytest.raises(ValueError):
            append(**bad)
    assert status(lambda: append(layer=1)) == kvq.KVQ_EINVAL
    assert status(lambda: append(rope=kvq.Rope(torch.ones(12, device="cuda")))) == kvq.KVQ_EUNSUPPORTED
    assert status(lambda: append(rope=kvq.Rope(torch.ones(72, device="cuda")))) == kvq.KVQ_EUNSUPPORTED
    assert status(lambda: append(rope=kvq.Rope(rope.inv_freq, factor=float("nan")))) == kvq.KVQ_EINVAL
    wide = torch.zeros(T, 2 * D + 4, dtype=torch.float16, device="cuda")
    assert status(lambda: append(k=wide[:, :2 * D].unflatten(1, (2, D)))) == kvq.KVQ_EINVAL   # stride
    odd = torch.zeros(T * 2 * D + 4, dtype=torch.float16, device="cuda")[4:].view(T, 2, D)
    assert status(lambda: append(v=odd)) == kvq.KVQ_EINVAL                                  # alignment
    assert status(lambda: append(k=k[:1].expand(T, 2, D))) == kvq.KVQ_EINVAL                # overlapping tokens

    with pytest.raises(TypeError):
        kvq.gather_rows(c, 0, cu, lens, s.pt, T, dtype=torch.float32)
    with pytest.raises(ValueError):
        kvq.gather_rows(c, 0, cu, lens, s.pt, T, k_out=k[:2])
    assert status(lambda: kvq.gather_rows(c, 0, cu, lens, s.pt, T, k_out=odd)) == kvq.KVQ_EINVAL
    with pytest.raises(ValueError):
        kvq.BlockBounds(bd.codes[:, :1].contiguous(), bd.scale)
    with pytest.raises(ValueError):
        kvq.update_block_bounds(c, 0, kvq.BlockBounds(bd.codes[:, :1].contiguous(), bd.scale[:, :1].contiguous()), cu,
                                lens, s.pt, T)
    assert status(lambda: kvq.update_block_bounds(c, 0, bd, cu, lens, s.pt, -1)) == kvq.KVQ_EINVAL

    def select(nb=4, qq=q, **kw):
        return kvq.select_blocks(c, 0, qq, aft, s.pt, bd, nb, **{**dict(cu_q=cu), **kw})

    for bad in (dict(nb=0), dict(sink=3, recent=2), dict(sink=-1), dict(recent=5), dict(cu_q=None)):
        assert status(lambda: select(**bad)) == kvq.KVQ_EINVAL, bad
    with pytest.raises(ValueError):
        select(blocks=torch.zeros(T, 2, 5, **i32))
    with pytest.raises(ValueError):
        kvq.sparse_attention(c, 0, q, aft, s.pt, blocks[:2], cu_q=cu)
    with pytest.raises(TypeError):
        kvq.sparse_attention(c, 0, q, aft, s.pt, blocks.long(), cu_q=cu)
    assert status(lambda: kvq.sparse_attention(c, 0, q, aft, s.pt, blocks)) == kvq.KVQ_EINVAL  # 3 queries, 2 sequences
    for scale in (-1.0, float("inf"), float("nan")):
        assert status(lambda: kvq.sparse_attention(c, 0, q, aft, s.pt, blocks, cu_q=cu, softmax_scale=scale)) == kvq.KVQ_EINVAL
    none = torch.zeros(T, 2, 0, **i32)
    assert status(lambda: kvq.sparse_attention(c, 0, q, aft, s.pt, none, cu_q=cu)) == kvq.KVQ_EINVAL
    long = kvq.Desc(1, 1, 1, D, 128, 16, 4, 1, 60000)
    cl, _ = kvq.alloc_pages(long)
    q1, l1 = torch.zeros(1, 1, D, dtype=torch.float16, device="cuda"), torch.ones(1, **i32)
    assert status(lambda: kvq.select_blocks(cl, 0, q1, l1, torch.zeros(1, 60000, **i32), kvq.BlockBounds.alloc(cl), 4)) == \
        kvq.KVQ_EUNSUPPORTED
    # Nothing to do: nothing is launched or refused.
    e = torch.zeros(0, 2, D, dtype=torch.float16, device="cuda")
    zero = torch.zeros(3, **i32)
    assert kvq.rope_quant_append(c, 0, e, e, zero, lens, s.pt, rope) is None
    assert kvq.gather_rows(c, 0, zero, lens, s.pt, 0)[0].shape == (0, 2, D)
    kvq.update_block_bounds(c, 0, bd, zero, lens, s.pt, 0)
    assert s.status() == 0


def test_bad_pages_and_positions_are_flagged_and_skipped():
    import torch
    import bit_paged_kv_diag_b200 as kvq
    s = Setup([20, 5, 40], [1, 1, 1], 2, 2, 64, 16, 0, extra=0, spare=0).fill()
    table = s.table.copy()
    table[0, 1] = 10 ** 6
    table[1, 0] = -3
    pt, cu = s.dev(table), s.dev(s.cu)
    lens = s.dev(np.array([20, 5, s.width * 16], np.int32))   # the third is at its page budget
    after = s.dev(np.array([21, 6, s.width * 16 + 1], np.int32))
    k, v, q = (torch.ones(3, n, D, dtype=torch.float16, device="cuda") for n in (2, 2, 4))
    pool = s.pool.clone()
    kvq.rope_quant_append(s.cache, 0, k, v, cu, lens, pt, kvq.Rope(torch.ones(64, device="cuda")), q=q)
    assert s.status() == kvq.KVQ_DEV_BAD_PAGE | kvq.KVQ_DEV_BAD_POS and torch.equal(pool, s.pool)
    ko, vo = kvq.gather_rows(s.cache, 0, cu, lens, pt, 3)
    assert s.status() == kvq.KVQ_DEV_BAD_PAGE | kvq.KVQ_DEV_BAD_POS and not ko.any() and not vo.any()
    bd = kvq.BlockBounds.alloc(s.cache)
    bd.scale.fill_(-1)
    kvq.update_block_bounds(s.cache, 0, bd, cu, lens, pt, 3)
    assert s.status() == kvq.KVQ_DEV_BAD_PAGE | kvq.KVQ_DEV_BAD_POS and (bd.scale == -1).all()
    bd.scale.fill_(1)
    o = kvq.select_blocks(s.cache, 0, q, after, pt, bd, 1, sink=0, recent=0)
    assert s.status() == kvq.KVQ_DEV_BAD_PAGE | kvq.KVQ_DEV_BAD_POS and (o[2] == -1).all() and (o[0] == 0).all()
    blocks = torch.tensor([0, 1], dtype=torch.int32, device="cuda").expand(3, 2, 2).contiguous()
    out = kvq.sparse_attention(s.cache, 0, q, after, pt, blocks)
    assert s.status() == kvq.KVQ_DEV_BAD_PAGE | kvq.KVQ_DEV_BAD_POS
    assert out[0].any() and not out[1].any() and not out[2].any()
    # A chunk longer than its sequence.
    cu2, short = torch.tensor([0, 1, 3, 3], dtype=torch.int32, device="cuda"), s.dev(np.array([6, 1, 0], np.int32))
    kvq.sparse_attention(s.cache, 0, q, short, s.pt, blocks, cu_q=cu2)
    assert s.status() == kvq.KVQ_DEV_BAD_POS
    o = kvq.select_blocks(s.cache, 0, q, short, s.pt, bd, 1, cu_q=cu2, sink=0)
    assert s.status() == kvq.KVQ_DEV_BAD_POS and (o[0] == 0).all() and (o[1:] == -1).all()
