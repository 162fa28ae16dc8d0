"""Plain forms of the head norm, the rotation, the 4-bit cache and attention, for
their tests: numpy, in the fp32 steps that the header names where results are
compared bit for bit, in 64 bits elsewhere."""
from __future__ import annotations

import numpy as np
import torch

DEV = torch.device("cuda:0")
BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
NAN_WORD = 0x7fc04300


def host(t):
    """A tensor's values as float64."""
    if t.dtype == torch.int16:
        t = t.view(BF16)
    return t.detach().double().cpu().numpy()


def host32(t):
    if t.dtype == torch.int16:
        t = t.view(BF16)
    return t.detach().float().cpu().numpy()


def table(rows, dim):
    """cos and sin [rows, dim/2], float32 on the GPU."""
    a = np.arange(rows)[:, None] * 10000.0 ** (-np.arange(0, dim, 2) / dim)
    return (torch.from_numpy(np.cos(a).astype(np.float32)).to(DEV),
            torch.from_numpy(np.sin(a).astype(np.float32)).to(DEV))


def turn(x, cos, sin, style):
    """x [...,D] with cos, sin broadcast against [...,dim/2]; x's own precision."""
    n = cos.shape[-1]
    i, j = ((slice(0, n), slice(n, 2 * n)) if style == "half" else
            (slice(0, 2 * n, 2), slice(1, 2 * n, 2)))
    y = x.copy()
    a, b = x[..., i], x[..., j]
    y[..., i] = a * cos - b * sin
    y[..., j] = b * cos + a * sin
    return y


def quantize(x):
    """Codes (uint8) [...,D], scale and z [...] (float32) and words (uint32) of fp32 rows."""
    x = np.asarray(x, dtype=np.float32)
    with np.errstate(all="ignore"):
        lo, hi = np.minimum(x.min(-1), np.float32(0)), np.maximum(x.max(-1), np.float32(0))
        rng = (hi - lo).astype(np.float32)
        bad = ~np.isfinite(x).all(-1) | ~np.isfinite(rng)
        s = (np.where(bad, 1, rng).astype(np.float32) / np.float32(15)).view(np.uint32)
        s = ((s.astype(np.uint64) + 0xffff) & 0xffff0000).astype(np.uint32)
        s = np.where(s < 0x00800000, np.uint32(0x3f800000), s).view(np.float32)
        z = np.minimum(np.rint(np.where(bad, 0, -lo).astype(np.float32) / s), 15)
        q = np.rint(np.where(bad[..., None], 0, x).astype(np.float32) / s[..., None])
        c = np.clip(q + z[..., None], 0, 15)
        c = np.where(bad[..., None], 0, c).astype(np.uint8)
        words = s.view(np.uint32) | ((z + 128).astype(np.float32).view(np.uint32) >> 16)
    words = np.where(bad, np.uint32(NAN_WORD), words).astype(np.uint32)
    return c, s, z, words


class Batch:
    """Sequences with `new` rows and `lengths` tokens in the cache, their pages in
    random order."""

    def __init__(self, new, lengths, page=32, seed=0, spare=2, before=0, behind=0, slack=0):
        g = np.random.default_rng(seed)
        self.new, self.lengths, self.page = list(new), list(lengths), page
        self.B = len(self.new)
        self.starts = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32) + before
        self.T = int(self.starts[-1]) + behind
        held = [-(-n // page) for n in self.lengths]
        self.max_pages = max(held + [1]) + slack
        self.pages = sum(held) + spare
        order = g.permutation(self.pages)
        self.table = np.full((self.B, self.max_pages), -1, np.int32)
        at = 0
        for b, n in enumerate(held):
            self.table[b, :n] = order[at:at + n]
            at += n

    def dev(self):
        return (torch.from_numpy(self.starts).to(DEV),
                torch.tensor(self.lengths, dtype=torch.int32, device=DEV),
                torch.from_numpy(self.table).to(DEV))

    def rows(self):
        """(row, sequence, place) of every row of a sequence."""
        for b in range(self.B):
            for i in range(self.new[b]):
                yield self.starts[b] + i, b, self.lengths[b] - self.new[b] + i

    def where(self, b, place):
        """(page, block, token) of a place, or None."""
        if place < 0 or place >= self.max_pages * self.page:
            return None
        p = int(self.table[b, place // self.page])
        if not 0 <= p < self.pages:
            return None
        return p, place % self.page // 32, place % 32


def block_bytes(D):
    return 32 * D + 256


def put(cache, at, shard, head, D, k=None, v=None):
    """Writes (codes, word) of a key and a value at `at` into a numpy cache."""
    page, block, t = at
    blk = cache[shard, page, head, block]
    if k is not None:
        blk[t * D // 2:(t + 1) * D // 2] = k[0][0::2] | k[0][1::2] << 4
        blk[32 * D + 4 * t:32 * D + 4 * t + 4] = np.frombuffer(np.uint32(k[1]).tobytes(), np.uint8)
    if v is not None:
        rows = blk[16 * D:32 * D].reshape(D, 16)
        old = rows[:, t // 2]
        rows[:, t // 2] = (old & 0x0f) | v[0] << 4 if t % 2 else (old & 0xf0) | v[0]
        o = 32 * D + 128 + 4 * t
        blk[o:o + 4] = np.frombuffer(np.uint32(v[1]).tobytes(), np.uint8)


def unpack(cache, D):
    """Keys and values [P,pages,Hk,blocks,32,D] in float64 of a numpy cache."""
    lead = cache.shape[:-1]
    k = cache[..., :16 * D].reshape(lead + (32, D // 2))
    k = np.stack((k & 15, k >> 4), -1).reshape(lead + (32, D))
    v = cache[..., 16 * D:32 * D].reshape(lead + (D, 16))
    v = np.swapaxes(np.stack((v & 15, v >> 4), -1).reshape(lead + (D, 32)), -1, -2)

    def value(c, raw):
        w = np.ascontiguousarray(raw).view(np.uint32)
        s = (w & 0xffff0000).view(np.float32).astype(np.float64)
        z = (w << np.uint32(16)).view(np.float32).astype(np.float64) - 128
        return (c.astype(np.float64) - z[..., None]) * s[..., None]
    with np.errstate(invalid="ignore"):
        return (value(k, cache[..., 32 * D:32 * D + 128]), value(v, cache[..., 32 * D + 128:]))


def random_cache(batch, P, Hk, D, seed=0, sigma=1.0):
    """A cache (numpy) whose every place holds the codes of random rows."""
    g = np.random.default_rng(seed + 17)
    cache = np.zeros((P, batch.pages, Hk, batch.page // 32, block_bytes(D)), np.uint8)
    lead = cache.shape[:-1]
    c, _, _, w = quantize(g.standard_normal(lead + (32, D)).astype(np.float32) * sigma)
    cache[..., :16 * D] = (c[..., 0::2] | c[..., 1::2] << 4).reshape(lead + (16 * D,))
    cache[..., 32 * D:32 * D + 128] = w.view(np.uint8).reshape(lead + (128,))
    c, _, _, w = quantize(g.standard_normal(lead + (32, D)).astype(np.float32))
    c = np.swapaxes(c, -1, -2)
    cache[..., 16 * D:32 * D] = (c[..., 0::2] | c[..., 1::2] << 4).reshape(lead + (16 * D,))
    cache[..., 32 * D + 128:] = w.view(np.uint8).reshape(lead + (128,))
    return cache


def attention(batch, cache, q, Hk, D, scale, causal=True, window=0):
    """(out, tolerance of its sums, lse, tolerance) [P,T,Hq,...] in float64; rows of
    no sequence are NaN.

    The kernel's first product adds D terms q*(128 + c), and the sum of q times 128
    + z goes off it: 143*sum|q| bounds every term and partial sum of both, each
    off by U a step of the D + 16, and the score is that times scale*s. (Keys as
    exact fp16 code - z make both smaller.) p is then off by that much of itself (and by 8U for exp2 and its argument, of up to
    |t|*log2(e)), and p*s' rounded to bf16 by 2^-8. The sum over keys adds at most
    U a step of at most L/128*32 + 64 more. Like the scores, the second product is
    the difference of sums of p*s'*(128 + code) and of p*s'*(128 + z), so those steps
    are off by U of up to 143*sum(p*s') in either of them, also where the values
    themselves are small: for weights that sum to 1, 2*143*(L/4 + 64)*U*sum(p*s').
    """
    P, T, Hq = q.shape[:3]
    G = Hq // Hk
    kk, vv = unpack(cache, D)
    steps, vsteps = (
        (np.ascontiguousarray(cache[..., at:at + 128]).view(np.uint32) & 0xffff0000)
        .view(np.float32).astype(np.float64) for at in (32 * D, 32 * D + 128))
    out = np.full((P, T, Hq, D), np.nan)
    tol, lse, ltol = out.copy(), np.full((P, T, Hq), np.nan), np.full((P, T, Hq), np.nan)
    for b in range(batch.B):
        n, length = batch.new[b], max(0, min(batch.lengths[b], batch.max_pages * batch.page))
        places = [(j, batch.where(b, j)) for j in range(length)]
        places = [(j, w) for j, w in places if w is not None]
        js = np.array([j for j, _ in places], dtype=np.int64)
        pg, bl, tk = (np.array([w[i] for _, w in places], dtype=np.int64) for i in range(3))
        for p in range(P):
            for h in range(Hq):
                k, v = kk[p, pg, h // G, bl, tk], vv[p, pg, h // G, bl, tk]
                st, vst = steps[p, pg, h // G, bl, tk], vsteps[p, pg, h // G, bl, tk]
                for i in range(n):
                    row, at = batch.starts[b] + i, length - n + i
                    seen = np.ones(len(js), bool)
                    if causal:
                        seen &= js <= at
                    if window:
                        seen &= js > at - window
                    if not seen.any():
                        out[p, row, h], tol[p, row, h], lse[p, row, h], ltol[p, row, h] = 0, 0, -np.inf, 0
                        continue
                    x = q[p, row, h]
                    t = (k[seen] @ x) * scale
                    m = t.max()
                    e = np.exp(t - m)
                    total = e.sum()
                    out[p, row, h] = e @ v[seen] / total
                    eps = (scale * st[seen].max() * 143 * np.abs(x).sum() * (D + 16) * U
                           + (8 + 2 * np.abs(t).max()) * U + (len(js) / 4 + 64) * U)
                    tol[p, row, h] = ((2.0 ** -8 + 2 * eps) * (e @ np.abs(v[seen]) / total)
                                      + 2 * 143 * (len(js) / 4 + 64) * U * (e @ vst[seen]) / total)
                    lse[p, row, h] = m + np.log(total)
                    ltol[p, row, h] = eps + 4 * U * (1 + abs(lse[p, row, h]))
    return out, tol, lse, ltol
