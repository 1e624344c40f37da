"""Paged caches in 4 bits for the tests, and the operators' definitions on them in 64 bits.

Everything that a call must not look at is filled with what would show: slots that no query sees are all
ones (their scales and biases NaN), page-table entries that no query needs hold numbers out of range.
"""
from __future__ import annotations

import math

import numpy as np
import torch

from compressed_kv_cache_dkv_gb300 import dkv
from tests import paged_ref as R

DT = R.DT


def quantise(x):
    """x [..., d] fp64 -> codes [..., d / 64, 64], scale and bias [..., d / 64], fp64, by the definition."""
    x = x.numpy().astype(np.float64)
    x = np.clip(np.where(np.isnan(x), 0.0, x), -61440.0, 61440.0).reshape(*x.shape[:-1], x.shape[-1] // 64, 64)
    top = np.abs(x).max(-1)
    _, e = np.frexp(top * (65.0 / 64.0))                      # top in [2^(e-1), 2^e)
    u = np.ldexp(1.0, np.maximum(np.where(top == 0.0, -99, e) - 1 - 10, -24))
    b = np.rint(x.min(-1) / u)
    s = np.ceil((np.rint(x.max(-1) / u) - b) / 15.0)
    c = np.clip(np.rint((x / u[..., None] - b[..., None]) / np.maximum(s, 1.0)[..., None]), 0, 15) * (s > 0)[..., None]
    return torch.from_numpy(c), torch.from_numpy(s * u), torch.from_numpy(b * u)


def values(c, s, b):
    return (c * s[..., None] + b[..., None]).flatten(-2)


def block_bytes(K, V):
    """Quantised K and V (code, scale, bias) of 16 tokens -> the bytes of a block."""
    parts = []
    for c, _, _ in (K, V):                                    # [16][g][64] -> [g][16][32]
        c = c.to(torch.uint8)
        parts.append((c[..., ::2] | (c[..., 1::2] << 4)).transpose(0, 1).reshape(-1))
    for _, s, b in (K, V):
        parts.append(torch.stack([s, b], -1).to(torch.float16).reshape(-1).view(torch.uint8))
    return torch.cat(parts)


class Cache:
    """Sequences of the given lengths in shuffled pages."""

    def __init__(self, lens, hkv, d, page, dtype="fp16", seed=0, spare=2, width=None, scale=1.0, pad_head=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.hkv, self.d, self.page, self.dt, self.device = list(lens), hkv, d, page, DT[dtype], device
        self.B = len(self.lens)
        self.width = width or max(1, max(-(-n // page) for n in self.lens))
        used = [-(-n // page) for n in self.lens]
        self.n_pages = sum(used) + spare
        perm = torch.randperm(self.n_pages, generator=g).int()
        self.table = torch.full((self.B, self.width), -7, dtype=torch.int32)
        at = 0
        for b, n in enumerate(used):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.free = perm[at:]
        self.bytes = page * 9 * d // 8
        store = torch.full((self.n_pages, hkv, self.bytes + pad_head), 0xFF, dtype=torch.uint8)
        self.q = []                                            # [sequence](K, V) quantised, [hkv][n]...
        for b, n in enumerate(self.lens):
            kv = []
            for _ in range(2):
                x = torch.randn(hkv, n, d, generator=g) * scale + 0.5 * torch.randn(hkv, 1, d, generator=g) * scale
                x = x * torch.exp(torch.randn(hkv, n, 1, generator=g))   # scales that differ from token to token
                kv.append(quantise(x.to(self.dt).double()))
            self.q.append(kv)
            for h in range(hkv):
                for t0 in range(0, n, 16):
                    m = min(16, n - t0)
                    rows = []
                    for c, s, bb in kv:
                        rows.append([torch.cat([y[h, t0:t0 + m], torch.full((16 - m, *y.shape[2:]), float("nan") if i else 15.0, dtype=y.dtype)])
                                     for i, y in enumerate((c, s, bb))])
                    store[self.table[b, t0 // page], h, t0 % page // 16 * 18 * d:][:18 * d] = block_bytes(*rows)
        self.store = store.to(device)
        self.cache = self.store[..., :self.bytes]
        self.K = [values(*kv[0]) for kv in self.q]
        self.V = [values(*kv[1]) for kv in self.q]

    def layout(self, hq, window=0, sinks=0):
        return dkv.dkv_qpaged_layout(self.cache, self.B, hq, self.d, self.width, dtype=self.dt, window=window, sinks=sinks)

    def dev(self, x):
        return torch.tensor(x, dtype=torch.int32, device=self.device)

    hidden_table = R.Cache.hidden_table


def attend(q, cache, b, h, pos, window, sinks):
    """q [Tq][d] fp64 against head h of sequence b -> (out, lse, weights, sums p |v| and p (s c + |b|), bounds of what a
    score's parts add up to: of q k, of the codes' and biases' products, and of what bf16 queries lose in fp16)."""
    kc, ks, kb = (x[h] for x in cache.q[b][0])
    vc, vs, vb = (x[h] for x in cache.q[b][1])
    K, V = cache.K[b][h], cache.V[b][h]
    ref = R.attend(q, K, V, pos, window, sinks)
    c = 1.0 / math.sqrt(q.shape[1])
    if K.shape[0]:
        size = values(kc, ks, kb.abs())
        m = R.seen(pos, K.shape[0], window, sinks)
        parts = float(torch.where(m, q.abs() @ size.T * c, 0.0).max())
        parts = max(parts, float((torch.where(m.any(0)[None], (q.abs().max(1).values[:, None] * (15 * ks.sum(1) * 64 + kb.abs().sum(1) * 64)[None]) * c, 0.0)).max()) * 2.0 ** -25)
        pv = ref[2] @ values(vc, vs, vb.abs())
    else:
        parts, pv = 0.0, ref[3]
    return ref, parts, pv
