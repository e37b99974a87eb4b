"""Plain numpy implementations of the calls around the cache, written from their definitions:
the position-rotating append, the read-back of rows, page bounds, page choice and attention over
chosen pages.  Rounded where the definitions round (fp32 in numpy is IEEE), 64 bits elsewhere."""
import math

import numpy as np

D = 128
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def hadamard(b):
    """Orthonormal block-diagonal Sylvester matrix [128][128] in 64 bits."""
    h = np.ones((1, 1))
    while h.shape[0] < b:
        h = np.block([[h, h], [h, -h]])
    return np.kron(np.eye(D // b), h) / math.sqrt(b)


def butterfly32(x, b):
    """The fixed-order fp32 butterfly and its final product."""
    x = np.asarray(x, np.float32)
    if b == 1:
        return x
    i, h = np.arange(D), 1
    while h < b:
        lo, hi = x[..., i & ~h], x[..., i | h]
        x = np.where(i & h, lo - hi, lo + hi).astype(np.float32)
        h *= 2
    return x * np.float32(1.0 / math.sqrt(b))


def e4m3(x):
    """Values rounded to E4M3 (nearest even, saturating): bytes and values."""
    import torch
    t = torch.from_numpy(np.minimum(np.asarray(x, np.float32), np.float32(448))).to(torch.float8_e4m3fn)
    return t.view(torch.uint8).numpy(), t.float().numpy()


def quantise(y, fmt):
    """Rotated fp32 rows [..., 128] -> codes [..., 128] (0..15), scale bytes [..., 2 | 8]."""
    if fmt == 0:
        s = np.minimum(np.abs(y).max(-1) / np.float32(7), np.float32(65504)).astype(np.float16)
        f = s.astype(np.float64)[..., None]
        n = np.where(f > 0, np.clip(np.rint(y / np.where(f > 0, f, 1)), -8, 7), 0).astype(np.int64)
        return n & 15, s[..., None].view(np.uint8)
    z = y.reshape(*y.shape[:-1], 8, 16)
    raw, f = e4m3(np.abs(z).max(-1) / np.float32(6))
    f = f[..., None]
    with np.errstate(divide="ignore"):
        r = np.where(f > 0, np.float32(1) / f, np.float32(0)).astype(np.float32)
    t = (z * r).reshape(y.shape)
    a = np.abs(t)
    n = ((a > 0.25).astype(np.int64) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    n = n + 8 * np.signbit(t)
    return np.where(np.repeat(f[..., 0] > 0, 16, -1), n, 0), raw


class Pool:
    """A pool of one layer on the host, by its documented layout."""

    def __init__(self, raw, hkv, page, fmt):
        w = 8 if fmt else 2
        blk = raw.reshape(-1, hkv, page * (D + 2 * w))
        cut = np.cumsum([page * 64, page * 64, page * w])
        self.fmt, self.page, self.hkv = fmt, page, hkv
        self.parts = [x.reshape(*x.shape[:-1], page, -1) for x in np.split(blk, cut, -1)]  # kc, vc, ks, vs

    def codes(self, kv):
        c = self.parts[kv]
        n = np.empty((*c.shape[:-1], D), np.int64)
        n[..., 0::2], n[..., 1::2] = c & 15, c >> 4
        return n

    def scales(self, kv):
        s = np.ascontiguousarray(self.parts[2 + kv])
        if self.fmt == 0:
            return s.view(np.float16).astype(np.float64)
        import torch
        return torch.from_numpy(s).view(torch.float8_e4m3fn).double().numpy()

    def values(self, kv):
        """[pages][hkv][page][128] in 64 bits, rotated basis."""
        n, s = self.codes(kv), self.scales(kv)
        if self.fmt == 0:
            return ((n ^ 8) - 8) * s
        v = E2M1[n & 7] * np.where(n & 8, -1.0, 1.0)
        return v * np.repeat(s, 16, -1)


def rope32(x, pos, inv, interleaved, factor):
    """The definition's fp32 rotation of x [T][heads][128]."""
    x = np.asarray(x, np.float32)
    ang = pos.astype(np.float64)[:, None] * inv.astype(np.float64)
    c = (np.cos(ang) * factor).astype(np.float32)[:, None]
    s = (np.sin(ang) * factor).astype(np.float32)[:, None]
    h = inv.shape[0]
    a, b = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if interleaved else (slice(0, h), slice(h, 2 * h))
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def rope64(x, pos, inv, interleaved, factor):
    x = np.asarray(x, np.float64)
    ang = pos.astype(np.float64)[:, None] * inv.astype(np.float64)
    c, s = (np.cos(ang) * factor)[:, None], (np.sin(ang) * factor)[:, None]
    h = inv.shape[0]
    a, b = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if interleaved else (slice(0, h), slice(h, 2 * h))
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def bounds(k, filled):
    """Keys [page][128] in 64 bits -> (lo, hi, sigma) over the first `filled` rows."""
    lo, hi = k[:filled].min(0), k[:filled].max(0)
    a = max(np.abs(lo).max(), np.abs(hi).max())
    if a == 0:
        return np.zeros(D, int), np.zeros(D, int), 0.0
    sigma = 2.0 ** math.floor(math.log2(a / 127))
    while 127 * sigma < a:
        sigma *= 2
    while 127 * (sigma / 2) >= a:
        sigma /= 2
    return np.floor(lo / sigma).astype(int), np.ceil(hi / sigma).astype(int), sigma


def choose(q, block, lo, hi, sigma, n, k, sink, recent):
    """Pages for one query and KV head: q [G][128] fp16; lo, hi [pages][128], sigma [pages]."""
    out = np.full(k, -1, np.int32)
    if n <= k:
        out[:max(n, 0)] = np.arange(max(n, 0))
        return out
    y = butterfly32(q.astype(np.float32), block)
    s = np.abs(y).max(-1) / np.float32(127)
    c = np.where(s[:, None] > 0, np.clip(np.rint(y / np.where(s > 0, s, 1)[:, None]), -127, 127), 0).astype(np.int64)
    whole = np.maximum(c, 0) @ hi[:n].T + np.minimum(c, 0) @ lo[:n].T
    score = ((whole.astype(np.float32) * s[:, None]).max(0) * sigma[:n].astype(np.float32)).astype(np.float64)
    mid = np.arange(sink, n - recent)
    best = mid[np.argsort(-score[mid], kind="stable")][:k - sink - recent]
    out[:] = np.sort(np.concatenate((np.arange(sink), best, np.arange(n - recent, n))))
    return out


def attend(q, H, k, v, scale):
    """q [G][128] -> (outputs [G][128], bound of the kernel's error [G][128]) over k, v [n][128]
    in the rotated basis, in 64 bits.

    The bound.  q' = q H scale log2(e) is carried to 2^-20 of M, the power of two above max |q'|
    (INT4: three int8 slices, 2^-21 M each side; NVFP4: two fp16 parts; both after fp32 butterfly
    roundings of 7 * 2^-24), so a score (log2 domain) is off by at most d = 2^-19 M max_t
    sum_d |k_td| with the fp32 sums; a weight by the factor 1 +- (2 d ln 2 + 2^-20) with exp2's
    2^-22, the split of p into two fp16 parts and the fp32 sums; numerator and denominator each
    by that: the vector by eps A with A = sum_t p_t |v_t|, eps = 4 d ln 2 + 2^-18.  The back
    rotation is orthonormal (|H e| <= |e|_2) and the store rounds by half a step of fp16."""
    qr = q.astype(np.float64) @ H
    z = qr @ k.T * scale
    p = np.exp(z - z.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    ref = (p @ v) @ H
    m = np.abs(qr).max(-1) * scale * 1.4427
    M = np.where(m > 0, 2.0 ** np.ceil(np.log2(np.maximum(m, 1e-300))), 1.0)
    d = 2.0 ** -19 * M * np.abs(k).sum(-1).max()
    eps = 4 * d * math.log(2) + 2.0 ** -18
    spread = np.linalg.norm(p @ np.abs(v), axis=-1)
    return ref, 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + (eps * spread)[:, None]
