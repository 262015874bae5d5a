"""The paged int8 K/V cache and attention over it in 64 bits, from the definition, for the tests."""
import math

import numpy as np
import torch


def f32(x):
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        return np.asarray(x, np.float64).astype(np.float32).astype(np.float64)


class Batch:
    """Lengths, block table and (optionally filled) cache of a batch; everything on the CPU."""

    def __init__(self, new, lens, heads, D, block, seed=0, extra=3, width=None):
        g = np.random.default_rng(seed)
        self.new, self.lens, self.heads, self.D, self.block = list(new), list(lens), heads, D, block
        self.B = len(self.new)
        self.cu = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.T = int(self.cu[-1])
        self.width = width or max([1] + [(n + block - 1) // block for n in self.lens])
        self.num = self.B * self.width + extra
        self.table = g.permutation(self.num)[: self.B * self.width].astype(np.int32).reshape(self.B, self.width)
        self.k, self.v = (g.normal(0, 32, (self.num, heads, block, D)).round().clip(-127, 127).astype(np.int8)
                          for _ in range(2))
        self.kqs, self.vqs = (f32(127.0 / g.uniform(1.0, 6.0, (self.num, heads))) for _ in range(2))

    def gpu(self):
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        return dict(cu=t(self.cu), lens=t(np.array(self.lens, np.int32)), table=t(self.table), k=t(self.k), v=t(self.v),
                    kqs=t(self.kqs.astype(np.float32)), vqs=t(self.vqs.astype(np.float32)))


def append_one(x, codes, qs, b, length, batch):
    """Sequence b's new rows x (fp64 of 16-bit values, [n, heads, D]) into codes, qs in place."""
    n, bs = x.shape[0], batch.block
    at = length - n
    done = 0
    while done < n:
        pos = at + done
        j, kept = pos // bs, pos % bs
        take = min(n - done, bs - kept)
        blk = batch.table[b, j]
        part = x[done : done + take]
        for h in range(batch.heads):
            rows = part[:, h]
            now = f32(127.0 * f32(1.0 / np.maximum(np.abs(rows).max(), f32(1e-8)))) if np.isfinite(rows).all() else np.nan
            old = qs[blk, h]
            if kept:
                now = np.nan if np.isnan(old) else (now if np.isnan(now) else min(now, old))
                if now < old:
                    r = f32(now / old)
                    codes[blk, h, :kept] = np.rint(f32(codes[blk, h, :kept] * r)).clip(-127, 127).astype(np.int8)
            if np.isnan(now):
                codes[blk, h, kept : kept + take] = 0  # not compared
            else:
                codes[blk, h, kept : kept + take] = np.rint(f32(rows * now)).clip(-127, 127).astype(np.int8)
            qs[blk, h] = now
        done += take


def append(batch, k, v):
    """k, v: fp64 [T, heads, D] of 16-bit values."""
    for b in range(batch.B):
        lo, hi = batch.cu[b], batch.cu[b + 1]
        append_one(k[lo:hi], batch.k, batch.kqs, b, batch.lens[b], batch)
        append_one(v[lo:hi], batch.v, batch.vqs, b, batch.lens[b], batch)


def attention(batch, q, scale, causal=True):
    """q: fp64 torch [T, Hq, D] (any device) -> (output, sum of weight x |value|), both fp64."""
    dev = q.device
    T, hq, D = q.shape
    G, bs = hq // batch.heads, batch.block
    y, mass = torch.zeros_like(q), torch.zeros_like(q)
    for b in range(batch.B):
        lo, hi, n, length = batch.cu[b], batch.cu[b + 1], batch.new[b], batch.lens[b]
        if n == 0 or length == 0:
            continue
        rows = batch.table[b, : (length + bs - 1) // bs]
        kk = batch.k[rows].astype(np.float64) / batch.kqs[rows][..., None, None]
        vv = batch.v[rows].astype(np.float64) / batch.vqs[rows][..., None, None]
        kk, vv = (torch.from_numpy(a.transpose(1, 0, 2, 3).reshape(batch.heads, -1, D)[:, :length].copy()).to(dev)
                  for a in (kk, vv))
        qq = q[lo:hi].transpose(0, 1).reshape(batch.heads, G, n, D)
        s = torch.einsum("hgnd,hkd->hgnk", qq, kk) * scale
        if causal:
            late = torch.arange(length, device=dev) > (length - n + torch.arange(n, device=dev))[:, None]
            s = s.masked_fill(late, -math.inf)
        p = torch.softmax(s, -1)
        p = torch.where(torch.isneginf(s).all(-1, keepdim=True), 0.0, p)  # a row without keys is zero
        y[lo:hi] = torch.einsum("hgnk,hkd->hgnd", p, vv).reshape(hq, n, D).transpose(0, 1)
        mass[lo:hi] = torch.einsum("hgnk,hkd->hgnd", p, vv.abs()).reshape(hq, n, D).transpose(0, 1)
    return y, mass
