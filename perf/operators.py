"""Cases and plain forms of the position-rotating append, the read-back of cached rows and
the block-sparse attention over the 4-bit paged cache.

Kinds of case (``op``):

* ``append``: position rotation of q and k, rotated 4-bit quantisation and paged append of
  k and v, then the appended rows read back in the model's basis (`rope_quant_append` and
  `gather_rows`); outputs: the rotated q, and K and V as the cache now holds them.
* ``rows``: cached rows of every sequence read back (`gather_rows`).
* ``bounds``: per-page key bounds of the pages that an append touched
  (`update_block_bounds`); output: the bounds as the values they stand for.
* ``select``: pages chosen per query and KV head by the bounds' score (`select_blocks`).
* ``sparse``: attention over chosen pages (`sparse_attention`).

Pool blocks are [K codes S x 64][V codes S x 64][K scales][V scales] per (page, KV head),
two 4-bit codes a byte; INT4 has one fp16 scale per row, NVFP4 one E4M3 per 16 channels.
"""
import math
import random

import numpy as np
import torch

own = False

D = 128


# ------------------------------------------------------------------------------ cases --
def listed():
    return [
        # one decode step's append of a 16-sequence batch, fp16 model, INT4 cache
        dict(name="append_decode", op="append", fmt=0, block=128, page=16, hkv=8, hq=32, batch=16, lo=4096, hi=4096,
             new_lo=1, new_hi=1, mix=0, dtype="float16", rd=128, inter=0, factor=1.0),
        # ragged prompt chunks behind cached prefixes: bf16 model, half of each head rotated, NVFP4 cache
        dict(name="append_ragged", op="append", fmt=1, block=64, page=64, hkv=4, hq=32, batch=7, lo=0, hi=32768,
             new_lo=1, new_hi=999, mix=1, dtype="bfloat16", rd=64, inter=1, factor=1.0),
        # prompts of 8 x 8192 tokens in one call
        dict(name="append_prefill", op="append", fmt=0, block=128, page=16, hkv=8, hq=32, batch=8, lo=0, hi=0,
             new_lo=8192, new_hi=8192, mix=0, dtype="float16", rd=128, inter=0, factor=1.0),
        # a short cached prefix read back for another request
        dict(name="rows_prefix", op="rows", fmt=0, block=32, page=16, hkv=2, hq=8, batch=1, lo=257, hi=257, mix=0,
             dtype="float16"),
        # long contexts read back whole
        dict(name="rows_long", op="rows", fmt=1, block=64, page=64, hkv=4, hq=32, batch=4, lo=16384, hi=65536, mix=2,
             dtype="bfloat16"),
        # one decode step of a wide ragged batch: each sequence's last page
        dict(name="bounds_decode", op="bounds", fmt=0, block=128, page=16, hkv=8, hq=32, batch=256, lo=0, hi=47,
             new_lo=1, new_hi=1, mix=3),
        # prompts of 8 x 8192 tokens: every page of them
        dict(name="bounds_prefill", op="bounds", fmt=0, block=128, page=64, hkv=8, hq=32, batch=8, lo=0, hi=0,
             new_lo=8192, new_hi=8192, mix=0),
        # one decode step over contexts of 32K to 128K tokens
        dict(name="select_decode", op="select", fmt=0, block=64, page=64, hkv=4, hq=32, batch=4, lo=32768, hi=131072,
             q_lo=1, q_hi=1, mix=4, blocks=64, sink=1, recent=2),
        # every query of a ragged prompt chunk
        dict(name="select_chunk", op="select", fmt=1, block=128, page=16, hkv=8, hq=32, batch=4, lo=8192, hi=16384,
             q_lo=100, q_hi=156, mix=5, blocks=64, sink=1, recent=4),
        # the smallest decode call
        dict(name="sparse_tiny", op="sparse", fmt=0, block=32, page=16, hkv=2, hq=8, batch=1, lo=257, hi=257,
             q_lo=1, q_hi=1, mix=0, blocks=8),
        # a decode step of 16 sequences, 4096 of their tokens attended
        dict(name="sparse_decode", op="sparse", fmt=0, block=128, page=64, hkv=8, hq=32, batch=16, lo=8192, hi=32768,
             q_lo=1, q_hi=1, mix=6, blocks=64),
        # a ragged prompt chunk, 1024 tokens attended per query
        dict(name="sparse_chunk", op="sparse", fmt=1, block=64, page=64, hkv=4, hq=32, batch=4, lo=8192, hi=32768,
             q_lo=200, q_hi=300, mix=7, blocks=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "rows", "bounds", "select", "sparse", "sparse"])
    hkv = rng.choice([1, 2, 4, 8])
    c = dict(op=op, fmt=rng.randrange(2), block=rng.choice([1, 32, 64, 128]), page=rng.choice([16, 32, 64, 128, 256]),
             hkv=hkv, hq=hkv * rng.choice([1, 2, 4, 8]), mix=rng.randrange(1 << 20))
    if op == "append":
        batch = _log(rng, 1, 64)
        new = _log(rng, 1, min(4096, 32768 // batch))
        c.update(batch=batch, lo=0, hi=_log(rng, 1, 4096), new_lo=max(1, new // 3), new_hi=new,
                 dtype=rng.choice(["float16", "bfloat16"]), rd=rng.choice([32, 64, 96, 128]), inter=rng.randrange(2),
                 factor=rng.choice([1.0, 1.25]))
    elif op == "rows":
        batch = _log(rng, 1, 64)
        n = _log(rng, 1, 65536 // batch)
        c.update(batch=batch, lo=max(1, n // 2), hi=n, dtype=rng.choice(["float16", "bfloat16"]))
    elif op == "bounds":
        batch = _log(rng, 1, 256)
        new = _log(rng, 1, 32768 // batch)
        c.update(batch=batch, lo=0, hi=rng.randrange(1, 600), new_lo=max(1, new // 2), new_hi=new)
    else:
        batch = _log(rng, 1, 16)
        queries = rng.choice([1, 1, 1, _log(rng, 2, 128 // batch)])
        n = _log(rng, 256, 98304 // batch if op == "sparse" else 196608 // batch // (1 if queries == 1 else 8))
        blocks = max(4, _log(rng, 64, 4096 if queries == 1 else 1024) // c["page"])
        c.update(batch=batch, lo=n // 2, hi=n, q_lo=max(1, queries // 2), q_hi=queries, blocks=blocks)
        if op == "select":
            c.update(sink=rng.randrange(0, 2), recent=rng.randrange(1, 3))
    return c


def _spread(case, lo, hi, salt):
    """One length per sequence in [lo, hi], fixed by the case; the first and last take the ends."""
    r = random.Random(case["mix"] * 8 + salt)
    n = [r.randint(lo, hi) for _ in range(case["batch"])]
    n[0] = hi
    n[-1] = lo if case["batch"] > 1 else hi
    return n


def _lengths(case):
    """(cached tokens before, tokens or query rows of the call, cached tokens after) per sequence."""
    if case["op"] in ("append", "bounds"):
        before, new = _spread(case, case["lo"], case["hi"], 1), _spread(case, case["new_lo"], case["new_hi"], 2)
        return before, new, [a + b for a, b in zip(before, new)]
    after = _spread(case, case["lo"], case["hi"], 1)
    if case["op"] == "rows":
        return [0] * len(after), after, after
    rows = _spread(case, case["q_lo"], case["q_hi"], 2)
    return [n - r for n, r in zip(after, rows)], rows, after


def _row_bytes(fmt):
    return 144 if fmt else 132


def work(case):
    hkv, hq, S, R = case["hkv"], case["hq"], case["page"], _row_bytes(case["fmt"])
    before, rows, after = _lengths(case)
    T = sum(rows)
    if case["op"] == "append":
        # q, k, v in; q, the cache rows and their read-back out
        return dict(bytes=T * ((hq + 2 * hkv) * 256 + hq * 256 + hkv * (R + 512)),
                    flops=T * ((hq + hkv) * 3 * D + 3 * hkv * 2 * 7 * D))
    if case["op"] == "rows":
        return dict(bytes=T * hkv * (R + 512), flops=T * hkv * 2 * 8 * D)
    if case["op"] == "bounds":
        first, last = [n // S for n in before], [(n - 1) // S for n in after]
        read = sum(n - f * S for n, f in zip(after, first))
        pages = sum(b - a + 1 for a, b in zip(first, last))
        return dict(bytes=hkv * (read * R // 2 + pages * (260 + 1024)), flops=hkv * read * 3 * D)
    if case["op"] == "select":
        pages = sum((n + S - 1) // S for n in after)
        per_query = sum(r * ((n + S - 1) // S) for r, n in zip(rows, after))
        return dict(bytes=hkv * pages * 260 + T * (hq * 256 + hkv * case["blocks"] * 4),
                    flops=per_query * hq * 4 * D)
    read = sum(min(n, r * case["blocks"] * S) for r, n in zip(rows, after))
    att = sum(r * min(n, case["blocks"] * S) for r, n in zip(rows, after))
    return dict(bytes=hkv * read * R + T * (hq * 512 + hkv * case["blocks"] * 4), flops=att * hq * 4 * D)


# ------------------------------------------------------------------------ plain pieces --
def _butterfly(x, b):
    """Block-diagonal orthonormal Hadamard transform of the last axis (128), fp32 stages
    h = 1, 2, ..., b/2 and one product with the fp32 value nearest 1/sqrt(b)."""
    if b == 1:
        return x
    shape, h = x.shape, 1
    while h < b:
        x = x.reshape(*shape[:-1], D // (2 * h), 2, h)
        x = torch.stack((x[..., 0, :] + x[..., 1, :], x[..., 0, :] - x[..., 1, :]), -2).reshape(shape)
        h *= 2
    return x * float(np.float32(1.0 / math.sqrt(b)))


def _pack(n):
    n = n & 15
    return (n[..., 0::2] | (n[..., 1::2] << 4)).to(torch.uint8)


def _quantise(y, fmt):
    """Rotated fp32 rows [..., 128] -> (codes [..., 64] uint8, scales [..., 2 or 8] uint8)."""
    if not fmt:
        s = (y.abs().amax(-1) / torch.full((), 7.0, device=y.device)).clamp(max=65504.0).to(torch.float16)
        f = s.float()[..., None]
        n = torch.where(f > 0, (y / f).round().clamp(-8, 7), torch.zeros_like(y)).to(torch.int16)
        return _pack(n), s[..., None].contiguous().view(torch.uint8)
    z = y.reshape(*y.shape[:-1], 8, 16)
    s = (z.abs().amax(-1) / torch.full((), 6.0, device=y.device)).clamp(max=448.0).to(torch.float8_e4m3fn)
    f = s.float()[..., None]
    t = torch.where(f > 0, z * (1.0 / f), torch.zeros_like(z)).reshape(y.shape)
    a = t.abs()
    n = ((a > 0.25).to(torch.int16) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return _pack(n + 8 * torch.signbit(t)), s.view(torch.uint8)


def _values(codes, scales, fmt):
    """The fp32 rows [..., 128] that codes and scales stand for."""
    n = torch.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], D)
    if not fmt:
        return ((n ^ 8).to(torch.float32) - 8.0) * scales.view(torch.float16).float()
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    f = scales.view(torch.float8_e4m3fn).float().repeat_interleave(16, -1)
    return table[n.to(torch.int64)] * f if n.numel() < (1 << 28) else table[n.to(torch.int32)] * f


def _views(pool, case):
    """K codes, V codes, K scales, V scales of a pool: uint8 [pages, hkv, page, ...]."""
    S, hkv, w = case["page"], case["hkv"], 8 if case["fmt"] else 2
    blk = pool.view(-1, hkv, S * (D + 2 * w))
    kc, vc, ks, vs = blk.split([S * 64, S * 64, S * w, S * w], -1)
    return [x.unflatten(-1, (S, -1)) for x in (kc, vc, ks, vs)]


def _rope(x, c, s, case):
    """Position rotation of x [T, heads, 128] fp32 by cos and sin [T, rd / 2] fp32."""
    rd = case["rd"]
    c, s = c[:, None], s[:, None]
    if case["inter"]:
        a, b = x[..., 0:rd:2], x[..., 1:rd:2]
        y = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = x[..., : rd // 2], x[..., rd // 2: rd]
        y = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((y, x[..., rd:]), -1)


def _bounds_of(k, filled):
    """Keys [..., S, 128] fp32 with `filled` [...] slots -> (codes [..., 2, 128] int8, scale [...] fp32)."""
    on = (torch.arange(k.shape[-2], device=k.device) < filled[..., None])[..., None]
    lo = torch.where(on, k, torch.inf).amin(-2)
    hi = torch.where(on, k, -torch.inf).amax(-2)
    m, e = torch.frexp(torch.maximum(lo.abs(), hi.abs()).amax(-1))
    power = ((e - 7 + (m > 0.9921875) + 127) << 23).to(torch.int32).view(torch.float32)
    scale = torch.where(m > 0, power, torch.zeros_like(m))
    step = torch.where(m > 0, scale, torch.ones_like(m))[..., None]
    return torch.stack((torch.floor(lo / step), torch.ceil(hi / step)), -2).to(torch.int8), scale


# ----------------------------------------------------------------------------- inputs --
def _rows(g, n, heads, device):
    """fp16-like K or V rows: N(0, 1), one channel per head large, row norms log-normal."""
    x = torch.randn(n, heads, D, generator=g, device=device)
    up = torch.exp(torch.rand(heads, generator=g, device=device) * math.log(5.0) + math.log(10.0))
    ch = torch.randint(0, D, (heads,), generator=g, device=device)
    x[:, torch.arange(heads, device=device), ch] *= up
    return x * torch.exp(0.5 * torch.randn(n, heads, 1, generator=g, device=device))


def _pool(g, case, pages, device):
    """A pool whose every slot holds a quantised row."""
    out = []
    for _ in range(2):
        y = _butterfly(_rows(g, pages * case["page"], case["hkv"], device).half().float(), case["block"])
        c, s = _quantise(y, case["fmt"])
        out.append([x.reshape(pages, case["page"], case["hkv"], -1).transpose(1, 2).reshape(pages, case["hkv"], -1)
                    for x in (c, s)])
    (kc, ks), (vc, vs) = out
    return torch.cat((kc, vc, ks, vs), -1).reshape(-1).contiguous()


def prepare(case, seed):
    device = "cuda"
    g = torch.Generator(device=device).manual_seed(seed)
    S, hkv, hq, op = case["page"], case["hkv"], case["hq"], case["op"]
    before, rows, after = _lengths(case)
    need = [(n + S - 1) // S for n in after]
    pages, width = sum(need), max(need)
    order = torch.randperm(pages, generator=g, device=device).to(torch.int32).cpu().numpy()
    table = np.full((case["batch"], width), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    st = dict(case=case, table=torch.from_numpy(table).to(device),
              before=torch.tensor(before, dtype=torch.int32, device=device),
              after=torch.tensor(after, dtype=torch.int32, device=device),
              cu=torch.tensor(np.concatenate(([0], np.cumsum(rows))), dtype=torch.int32, device=device), total=sum(rows))
    T = st["total"]
    if op == "append":
        dt = getattr(torch, case["dtype"])
        st["pool"] = torch.zeros(pages * hkv * S * _row_bytes(case["fmt"]), dtype=torch.uint8, device=device)
        qkv = torch.empty(T, (hq + 2 * hkv) * D, dtype=dt, device=device)  # the projection's output
        qkv[:, : hq * D].copy_(torch.randn(T, hq * D, generator=g, device=device))
        qkv[:, hq * D: (hq + hkv) * D].copy_(_rows(g, T, hkv, device).flatten(1))
        qkv[:, (hq + hkv) * D:].copy_(_rows(g, T, hkv, device).flatten(1))
        q, k, v = qkv.split([hq * D, hkv * D, hkv * D], -1)
        st.update(q=q.unflatten(-1, (hq, D)), k=k.unflatten(-1, (hkv, D)), v=v.unflatten(-1, (hkv, D)))
        st["inv"] = (1e6 ** -(torch.arange(0, case["rd"], 2, device=device, dtype=torch.float64) / case["rd"])).float()
    else:
        st["pool"] = _pool(g, case, pages, device)
    if op in ("bounds", "select"):
        st["codes"] = torch.zeros(1, pages, hkv, 2, D, dtype=torch.int8, device=device)
        st["scale"] = torch.zeros(1, pages, hkv, dtype=torch.float32, device=device)
    if op in ("select", "sparse"):
        st["q"] = torch.randn(T, hq, D, generator=g, device=device).half()
    if op == "select":
        kc, _, ks, _ = _views(st["pool"], case)
        filled = torch.full((pages,), S, dtype=torch.int32)
        for b, n in enumerate(need):
            filled[table[b, n - 1]] = after[b] - (n - 1) * S
        st["codes"][0], st["scale"][0] = _bounds_of(_values(kc, ks, case["fmt"]), filled.to(device)[:, None].expand(-1, hkv))
    if op == "sparse":
        # each query and head: the first and the last pages, and others at random, in order
        n = (_positions(st)[0] // S + 1)[:, None, None]
        key = torch.rand(T, hkv, width, generator=g, device=device)
        page = torch.arange(width, device=device)
        key = torch.where((page == 0) | (page == n - 1), 2.0, torch.where(page < n, key, -1.0))
        k = min(case["blocks"], width)
        top, idx = key.topk(k, -1)
        idx = torch.where(top < 0, width, idx).sort(-1).values
        blocks = torch.full((T, hkv, case["blocks"]), -1, dtype=torch.int32, device=device)
        blocks[..., :k] = torch.where(idx == width, -1, idx)
        st["blocks"] = blocks
    if own:
        import bit_paged_kv_diag_b200 as kvq
        d = kvq.Desc(1, hkv, hq, D, case["block"], S, pages, case["batch"], width, case["fmt"])
        st["cache"], _ = kvq.alloc_pages(d, pool=st["pool"])
        if op == "append":
            st["rope"] = kvq.Rope(st["inv"], interleaved=bool(case["inter"]), factor=case["factor"])
        if op in ("bounds", "select"):
            st["bounds"] = kvq.BlockBounds(st["codes"], st["scale"])
    return st


def _positions(st):
    """(cache position, sequence) of every row of the call."""
    t = torch.arange(st["total"], device=st["cu"].device, dtype=torch.int32)
    seq = torch.searchsorted(st["cu"][1:], t, right=True)
    return st["before"][seq] + t - st["cu"][seq], seq


# ------------------------------------------------------------------------------- run --
def _plain_append(st):
    case = st["case"]
    pos, seq = _positions(st)
    ang = pos.double()[:, None] * st["inv"].double()
    c, s = (ang.cos() * case["factor"]).float(), (ang.sin() * case["factor"]).float()
    q = _rope(st["q"].float(), c, s, case).half()
    kc, ks = _quantise(_butterfly(_rope(st["k"].float(), c, s, case), case["block"]), case["fmt"])
    vc, vs = _quantise(_butterfly(st["v"].float(), case["block"]), case["fmt"])
    page, slot = st["table"][seq, pos // case["page"]].long(), (pos % case["page"]).long()
    views = _views(st["pool"], case)
    for view, new in zip(views, (kc, vc, ks, vs)):
        view[page, :, slot] = new
    return [q, *_plain_rows(st, torch.float16)]


def _plain_rows(st, dtype):
    case = st["case"]
    pos, seq = _positions(st)
    page, slot = st["table"][seq, pos // case["page"]].long(), (pos % case["page"]).long()
    kc, vc, ks, vs = (view[page, :, slot] for view in _views(st["pool"], case))
    return [_butterfly(_values(c, s, case["fmt"]), case["block"]).to(dtype) for c, s in ((kc, ks), (vc, vs))]


def _plain_bounds(st):
    case = st["case"]
    S = case["page"]
    first, last = st["before"] // S, (st["after"] - 1) // S
    most = (case["new_hi"] + S - 2) // S + 1  # pages that a sequence's new tokens can touch
    lp = torch.minimum(first[:, None] + torch.arange(most, device=first.device), last[:, None])
    page = st["table"].gather(1, lp.long()).long()
    kc, _, ks, _ = _views(st["pool"], case)
    filled = torch.clamp(st["after"][:, None] - lp * S, max=S)
    codes, scale = _bounds_of(_values(kc[page], ks[page], case["fmt"]), filled[..., None].expand(-1, -1, case["hkv"]))
    st["codes"][0, page], st["scale"][0, page] = codes, scale
    return st["codes"] * st["scale"][..., None, None]


def _plain_select(st):
    case = st["case"]
    S, hkv, k = case["page"], case["hkv"], case["blocks"]
    pos, seq = _positions(st)
    y = _butterfly(st["q"].float(), case["block"])
    sq = y.abs().amax(-1, keepdim=True) / torch.full((), 127.0, device=y.device)
    c = torch.where(sq > 0, (y / sq).round().clamp(-127, 127), torch.zeros_like(y)).unflatten(1, (hkv, -1))
    c = torch.stack((c.clamp(max=0), c.clamp(min=0)), -2).flatten(-2)  # [T, hkv, G, 256]: with lo, with hi
    page = st["table"].clamp(min=0).long()  # [B, width]
    bound = st["codes"][0, page].float().flatten(-2).transpose(1, 2)[seq]  # [T, hkv, width, 256]
    score = (c @ bound.transpose(-1, -2)) * sq.unflatten(1, (hkv, -1))  # whole numbers below 2^24: exact
    score = score.amax(2) * st["scale"][0, page].transpose(1, 2)[seq]
    n = (pos // S + 1)[:, None, None]
    at = torch.arange(page.shape[1], device=y.device)
    forced = (at < case["sink"]) | (at >= n - case["recent"])
    score = torch.where(at < n, torch.where(forced, torch.inf, score), -torch.inf)
    idx = score.sort(dim=-1, descending=True, stable=True).indices[..., :k]
    idx = torch.where(idx < n, idx, 1 << 30).sort(-1).values
    out = torch.full((*idx.shape[:2], k), -1, dtype=torch.int32, device=y.device)
    out[..., : idx.shape[-1]] = torch.where(idx < (1 << 30), idx, -1)
    return out


def _plain_sparse(st):
    case = st["case"]
    S, hkv = case["page"], case["hkv"]
    pos, seq = _positions(st)
    q = _butterfly(st["q"].float(), case["block"]).unflatten(1, (hkv, -1))  # [T, hkv, G, 128]
    blocks = st["blocks"]
    page = st["table"][seq][:, None].expand(-1, hkv, -1).gather(2, blocks.clamp(min=0).long()).long()
    head = torch.arange(hkv, device=q.device)[:, None]
    kc, vc, ks, vs = (view[page, head].flatten(2, 3) for view in _views(st["pool"], case))  # [T, hkv, k S, ...]
    at = (blocks[..., None] * S + torch.arange(S, device=q.device, dtype=torch.int32)).flatten(2)
    on = ((blocks >= 0)[..., None].expand(-1, -1, -1, S).flatten(2) & (at <= pos[:, None, None]))[:, :, None]
    score = (q @ _values(kc, ks, case["fmt"]).transpose(-1, -2)) * (1.0 / math.sqrt(D))
    score = torch.where(on, score, -torch.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True))
    o = (p @ _values(vc, vs, case["fmt"])) / p.sum(-1, keepdim=True)
    return _butterfly(o, case["block"]).flatten(1, 2).half()


def run(st):
    case, op = st["case"], st["case"]["op"]
    if not own:
        if op == "append":
            return _plain_append(st)
        if op == "rows":
            return _plain_rows(st, getattr(torch, case["dtype"]))
        return {"bounds": _plain_bounds, "select": _plain_select, "sparse": _plain_sparse}[op](st)
    import bit_paged_kv_diag_b200 as kvq
    if op == "append":
        q = kvq.rope_quant_append(st["cache"], 0, st["k"], st["v"], st["cu"], st["before"], st["table"], st["rope"],
                                  q=st["q"])
        return [q, *kvq.gather_rows(st["cache"], 0, st["cu"], st["before"], st["table"], st["total"])]
    if op == "rows":
        return list(kvq.gather_rows(st["cache"], 0, st["cu"], st["before"], st["table"], st["total"],
                                    dtype=getattr(torch, case["dtype"])))
    if op == "bounds":
        kvq.update_block_bounds(st["cache"], 0, st["bounds"], st["cu"], st["before"], st["table"], st["total"])
        return st["codes"] * st["scale"][..., None, None]
    cu = None if case["q_hi"] == 1 else st["cu"]
    if op == "select":
        return kvq.select_blocks(st["cache"], 0, st["q"], st["after"], st["table"], st["bounds"], case["blocks"],
                                 cu_q=cu, sink=case["sink"], recent=case["recent"])
    return kvq.sparse_attention(st["cache"], 0, st["q"], st["after"], st["table"], st["blocks"], cu_q=cu)


# ----------------------------------------------------------------------------- exact --
def _hadamard(b):
    """Orthonormal block-diagonal Hadamard matrix in 64 bits: sign = parity of i & j inside a block."""
    i = np.arange(D)
    odd = np.vectorize(lambda v: bin(v).count("1") & 1)((i % b)[:, None] & (i % b)[None, :])
    same = (i[:, None] // b) == (i[None, :] // b)
    return torch.from_numpy(np.where(same, 1.0 - 2.0 * odd, 0.0) / math.sqrt(b)).cuda()


def _decode64(raw, case, S):
    """A pool's bytes [..., S * R] -> K, V [..., S, 128] in 64 bits, in the rotated basis."""
    w = 8 if case["fmt"] else 2
    got = []
    for kv in range(2):
        c = raw[..., kv * S * 64: (kv + 1) * S * 64].reshape(*raw.shape[:-1], S, 64)
        s = raw[..., S * (D + kv * w): S * (D + kv * w) + S * w].reshape(*raw.shape[:-1], S, w).contiguous()
        n = torch.empty(*c.shape[:-1], D, dtype=torch.float64, device=raw.device)
        for half, nib in ((0, c % 16), (1, c // 16)):
            if case["fmt"]:
                e, m = (nib // 2) % 4, (nib % 2).double()
                v = torch.where(e == 0, 0.5 * m, 0.5 * (1 << e.int()) * (1 + 0.5 * m)) * (1 - 2 * (nib // 8).double())
            else:
                v = nib.double() - 16.0 * (nib >= 8)
            n[..., half::2] = v
        f = s.view(torch.float8_e4m3fn if case["fmt"] else torch.float16).double()
        got.append((n.unflatten(-1, (w if case["fmt"] else 1, -1)) * f[..., None]).flatten(-2))
    return got


def _nearest64(y, case):
    """Rows in 64 bits -> the 4-bit values nearest to them, per the cache's format, in 64 bits."""
    if not case["fmt"]:
        s = (y.abs().amax(-1, keepdim=True) / 7.0).clamp(max=65504.0).half().double()
        return torch.where(s > 0, torch.round(y / s).clamp(-8, 7) * s, 0.0)
    z = y.unflatten(-1, (8, 16))
    s = (z.abs().amax(-1, keepdim=True) / 6.0).clamp(max=448.0).float().to(torch.float8_e4m3fn).double()
    t = torch.where(s > 0, z / s, 0.0)
    a = t.abs().clamp(max=6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return (torch.sign(t) * (torch.round(a / step) * step).clamp(max=6.0) * s).flatten(-2)


def exact(case, seed):
    st = prepare(case, seed)
    S, hkv, op = case["page"], case["hkv"], case["op"]
    before, rows, after = _lengths(case)
    H = _hadamard(case["block"])
    if op == "append":
        pos = torch.cat([torch.arange(a, a + r) for a, r in zip(before, rows)]).cuda().double()
        ang = pos[:, None] * st["inv"].double()
        c, s = (torch.cos(ang) * case["factor"])[:, None], (torch.sin(ang) * case["factor"])[:, None]

        def turn(x):
            y, h = x.clone(), case["rd"] // 2
            i, j = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if case["inter"] else (slice(0, h), slice(h, 2 * h))
            y[..., i] = x[..., i] * c - x[..., j] * s
            y[..., j] = x[..., j] * c + x[..., i] * s
            return y

        k = _nearest64(turn(st["k"].double()) @ H, case) @ H
        v = _nearest64(st["v"].double() @ H, case) @ H
        return [turn(st["q"].double()), k, v]
    raw = st["pool"].view(-1, hkv, S * _row_bytes(case["fmt"]))
    table = st["table"].long()
    if op == "rows":
        got = [[], []]
        for b, n in enumerate(after):
            for x, to in zip(_decode64(raw[table[b, : (n + S - 1) // S]], case, S), got):
                to.append(x.transpose(1, 2).flatten(0, 1)[:n] @ H)
        return [torch.cat(x) for x in got]
    if op == "bounds":
        out = torch.zeros(1, raw.shape[0], hkv, 2, D, dtype=torch.float64, device="cuda")
        for b in range(case["batch"]):
            f, n = before[b] // S, after[b]
            ids = table[b, f: (n - 1) // S + 1]
            k = _decode64(raw[ids], case, S)[0]
            gone = (torch.arange(len(ids) * S, device="cuda") + f * S >= n).view(-1, 1, S, 1)
            lo, hi = k.masked_fill(gone, math.inf).amin(2), k.masked_fill(gone, -math.inf).amax(2)
            a = torch.maximum(-lo, hi).amax(-1).clamp(min=0)
            a = torch.maximum(a, torch.maximum(lo, -hi).amax(-1))
            step = ((torch.floor(torch.log2(a / 127.0)).clamp(min=-1000).long() + 1022) << 52).view(torch.float64)
            step = step * (1 + (127.0 * step < a).double() + 2 * (127.0 * 2 * step < a).double())  # least power enough
            step = torch.where(a > 0, step, 1.0)[..., None]
            out[0, ids] = torch.stack((torch.floor(lo / step) * step, torch.ceil(hi / step) * step), -2)
        return out
    if op == "select":
        # the query's codes are defined by the 32-bit butterfly and two 32-bit divisions
        q = st["q"].float().cpu().numpy()
        h = 1
        while h < case["block"]:
            i = np.arange(D)
            a, b = q[..., i & ~h], q[..., i | h]
            q = np.where((i & h) == 0, a + b, a - b).astype(np.float32)
            h *= 2
        q = q * np.float32(1.0 / math.sqrt(case["block"]))
        sq = np.abs(q).max(-1) / np.float32(127.0)
        c = np.clip(np.rint(q / np.where(sq > 0, sq, np.float32(1))[..., None]), -127, 127)
        c = torch.from_numpy(c).cuda().double().unflatten(1, (hkv, -1))
        sq = torch.from_numpy(sq).cuda().unflatten(1, (hkv, -1))
        out, t = torch.full((st["total"], hkv, case["blocks"]), -1, dtype=torch.int32), 0
        for b, r in enumerate(rows):
            bd = st["codes"][0, table[b]].double()  # [width, hkv, 2, 128]
            sg = st["scale"][0, table[b]]
            whole = torch.einsum("rhgd,phd->rhgp", c[t:t + r].clamp(min=0), bd[:, :, 1]) + \
                torch.einsum("rhgd,phd->rhgp", c[t:t + r].clamp(max=0), bd[:, :, 0])
            score = (whole.float() * sq[t:t + r, :, :, None]).amax(2).double() * sg.T.double()
            score = score.cpu().numpy()
            for i in range(r):
                n = (before[b] + i) // S + 1
                for hd in range(hkv):
                    if n <= case["blocks"]:
                        pick = np.arange(n)
                    else:
                        mid = np.arange(case["sink"], n - case["recent"])
                        best = mid[np.argsort(-score[i, hd, mid], kind="stable")]
                        best = best[: case["blocks"] - case["sink"] - case["recent"]]
                        pick = np.sort(np.concatenate((np.arange(case["sink"]), best, np.arange(n - case["recent"], n))))
                    out[t + i, hd, : len(pick)] = torch.from_numpy(pick.astype(np.int32))
            t += r
        return out
    # sparse
    if sum(rows) * hkv * case["blocks"] * S > (1 << 24):
        return None
    q = (st["q"].double() @ H).unflatten(1, (hkv, -1))
    out, t = [], 0
    for b, r in enumerate(rows):
        for i in range(r):
            p = before[b] + i
            for hd in range(hkv):
                blk = st["blocks"][t, hd].long()
                blk = blk[blk >= 0]
                k, v = (x.flatten(0, 1) for x in _decode64(raw[table[b, blk], hd], case, S))
                at = (blk[:, None] * S + torch.arange(S, device="cuda")).flatten()
                z = (q[t, hd] @ k.T / math.sqrt(D)).masked_fill(at > p, -math.inf)
                out.append(torch.softmax(z, -1) @ v)
            t += 1
    return (torch.cat(out).view(t, case["hq"], D)) @ H
