"""kv_attention on bf16 queries in 64 bits with the queries that the kernels
multiply, and bounds without the queries' rounding: tight enough that a tile of
32 keys left out of some thousands, or taken twice, shows.

The kernels rotate a query in binary32 (stages of stride 1, 2, 4, 8, one
rounding a sum), scale the row by the power of two that brings its largest
value into [2^12, 2^13) and round to fp16.  All of it is defined operation by
operation, so the model takes the very same fp16 numbers; products of them with
decoded values (11 and 6 significant bits) are exact."""
from __future__ import annotations

import numpy as np
import torch

import kv_model
import oracle
from test_kv_gpu import Scene


def rounded_queries(q, rotate):
    """The rows' fp16 numbers over their power of two, as float64."""
    x = q.float().numpy().astype(np.float32)
    shape = x.shape
    if rotate:
        z = x.reshape(-1, 16).copy()
        for h in (1, 2, 4, 8):
            p = z.reshape(-1, 8 // h, 2, h)
            z = np.stack((p[:, :, 0] + p[:, :, 1], p[:, :, 0] - p[:, :, 1]), 2).reshape(-1, 16)
        x = (z * np.float32(0.25)).reshape(shape)
    assert x.dtype == np.float32
    top = np.abs(x).max(-1, keepdims=True)
    e = np.where(top > 0, 13 - np.frexp(np.where(top > 0, top, 1))[1], 0)
    return np.ldexp(np.ldexp(x.astype(np.float64), e).astype(np.float16).astype(np.float64), -e)


class TiledScene(Scene):
    """A scene of bf16 queries whose V has, beside noise, a constant row for
    each 32 keys of a request, so that each tile of keys pulls the results its
    own way."""

    def __init__(self, seed, new, cached, q_heads, kv_heads, d, page, **kw):
        super().__init__(seed, new, cached, q_heads, kv_heads, d, page, **kw)
        gen = torch.Generator().manual_seed(seed + 1)
        total = int(self.lens.sum())
        k = torch.randn(total, kv_heads, d, generator=gen).bfloat16()
        v, at = torch.randn(total, kv_heads, d, generator=gen), 0
        for n in self.lens:
            own = 3.0 * torch.sign(torch.randn(-(-int(n) // 32), kv_heads, d, generator=gen))
            v[at:at + n] += own.repeat_interleave(32, 0)[:n]
            at += int(n)
        slots = [int(self.table[r, t // page]) * page + t % page for r, n in enumerate(self.lens) for t in range(n)]
        kv_model.append(k, v.bfloat16(), slots, self.cache, self.amax, page, self.rotate)


class Attention:
    """out and bound of each row, also with some keys counted other than once.

    Bounds, for weights p of sum 1, mass = sum p |v| of the V elements as
    stored, n keys, all relative to mass unless said otherwise:
      logits: binary32 sums of d exact products, (d + 8) 2^-23 of sum |q k|
        (a matrix instruction may truncate), and 2^-22 of the logit for its
        factor and the exponent's argument; a weight is off by exp of that - 1;
      weights: 2^-20 for the exponential, in numerator and denominator; 2^-11
        for rounding to fp16, in the numerator alone; below fp16's normal range
        2^-25 absolute, of weights whose largest is 2^12 or more: 2^-37 max|v|
        a key;
      sums: n 2^-24 each for numerator and denominator, and 16 2^-24 for the
        joining, the scale and the rotation back;
      the result's own rounding: half a step of it."""

    def __init__(self, s, r, causal=True, window=0, scale=None):
        """Request r of a scene of bf16 queries."""
        a, b = int(s.cu[r]), int(s.cu[r + 1])
        kv, n, d, page = int(s.lens[r]), b - a, s.q.shape[2], s.page
        kvh, group = s.cache.shape[1], s.q.shape[1] // s.cache.shape[1]
        self.rotate, self.rows, self.d = s.rotate, slice(a, b), d
        g = [float(oracle.global_scale(float(x))) for x in s.amax]
        ids = [int(i) for i in s.table[r][:-(-kv // page)]]
        x = rounded_queries(s.q[a:b], s.rotate)
        scale = np.float64(np.float32(d ** -0.5 if scale is None else scale))
        i, j = np.arange(n)[:, None], np.arange(kv)[None]
        pos = kv - n + i
        seen = (j <= pos) if causal else np.ones((n, kv), bool)
        if window:
            seen = seen & (j > pos - window)
        self.seen = seen
        self.p, self.v, self.dl = [], [], []
        for h in range(kvh):
            k, v = (np.concatenate([kv_model.decode(s.cache[c, h], page, d, g[w], w) for c in ids])[:kv]
                    for w in (0, 1))
            for qh in range(h * group, (h + 1) * group):
                logits = np.where(seen, scale * (x[:, qh] @ k.T), -np.inf)
                spread = scale * (np.abs(x[:, qh]) @ np.abs(k).T)
                dl = spread * (d + 8) * 2.0 ** -23 + np.where(seen, np.abs(logits), 0) * 2.0 ** -22
                self.dl.append(np.where(seen, dl, 0).max(1))
                top = logits.max(1, keepdims=True)
                self.p.append(np.exp(logits - np.where(np.isfinite(top), top, 0)))
                self.v.append(v)

    def result(self, times=None):
        """out and bound [n, heads, d]; times: how often each key counts."""
        h16 = kv_model.hadamard()
        outs, bounds = [], []
        for p, v, dl in zip(self.p, self.v, self.dl):
            w = p if times is None else p * times
            total = w.sum(1, keepdims=True)
            w = w / np.where(total > 0, total, 1)
            o, mass = w @ v, w @ np.abs(v)
            n = self.seen.sum(1, keepdims=True)
            rel = 2 * (np.expm1(dl)[:, None] + 2.0 ** -20 + n * 2.0 ** -24) + 2.0 ** -11 + 16 * 2.0 ** -24
            err = rel * mass + n * 2.0 ** -37 * np.abs(v).max()
            if self.rotate:
                o = (o.reshape(-1, 16) @ h16).reshape(o.shape)
                err = (err.reshape(-1, 16) @ np.abs(h16)).reshape(o.shape)
            outs.append(o)
            # half a step of bf16 (8 significant bits) at the largest value that is rounded
            bounds.append(err + np.exp2(np.floor(np.log2(np.abs(o) + err + 1e-300)) - 8))
        return np.stack(outs, 1), np.stack(bounds, 1)

    def worst_without(self, lo, hi, count=0):
        """How far off, in bounds, results are in which keys [lo, hi) count
        `count` times."""
        out, bound = self.result()
        times = np.ones(self.seen.shape[1])
        times[lo:hi] = count
        other, _ = self.result(times)
        live = self.seen.any(1)
        return float((np.abs(other - out)[live] / bound[live]).max())
