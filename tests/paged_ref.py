"""Paged caches for the tests, and the operators' definitions on them in 64 bits.

Everything that a call must not look at is filled with what would show: slots that no query sees
hold NaN and infinities, page-table entries that no query needs hold numbers out of range.
"""
from __future__ import annotations

import math

import torch

from compressed_kv_cache_dkv_gb300 import dkv

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


class Cache:
    """Sequences of the given lengths in shuffled pages; K, V: their rows, fp64 on the CPU."""

    def __init__(self, lens, hkv, d, page, dtype="fp16", order="head", seed=0, spare=2, width=None, device="cuda"):
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
        self.K, self.V = ([torch.randn(hkv, n, d, generator=g).to(self.dt).double() for n in self.lens] for _ in range(2))
        shape = (self.n_pages, hkv, page, d) if order == "head" else (self.n_pages, page, hkv, d)
        pools = []
        for rows in (self.K, self.V):
            x = torch.full(shape, float("nan"), dtype=self.dt)
            x.view(-1)[::3] = float("inf")
            view = x if order == "head" else x.transpose(1, 2)
            for b, n in enumerate(self.lens):
                t = torch.arange(n)
                view[self.table[b].long()[t // page], :, t % page] = rows[b].transpose(0, 1).to(self.dt)
            y = x.to(device)
            pools.append(y if order == "head" else y.transpose(1, 2))
        self.k, self.v = pools

    def layout(self, hq, window=0, sinks=0):
        return dkv.dkv_paged_layout(self.k, self.B, hq, self.width, window=window, sinks=sinks)

    def dev(self, x):
        return torch.tensor(x, dtype=torch.int32, device=self.device)

    def hidden_table(self, first_pos, window, sinks):
        """The page table with rubbish in every entry that queries from position first_pos[b] on do not need."""
        t = self.table.clone()
        for b, n in enumerate(self.lens):
            for i in range(self.width):
                lo, hi = i * self.page, min(n, (i + 1) * self.page)
                need = lo < hi and (not window or hi > max(0, first_pos[b]) - window + 1 or lo < sinks)
                if not need:
                    t[b, i] = [-1, 1 << 30, -(1 << 31)][i % 3]
        return t.to(self.device)

    def row(self, pool, b, h, t):
        """Rows t of a sequence's head as the pool holds them now (fp64)."""
        x = pool.cpu()
        return x[self.table[b].long()[t // self.page], h, t % self.page].double()


def seen(pos, n, window, sinks):
    """[len(pos)][n] truth values: the query at pos sees token t."""
    t, p = torch.arange(n)[None], pos[:, None]
    m = t <= p
    if window:
        m &= (t > p - window) | (t < sinks)
    return m


def attend(q, K, V, pos, window, sinks):
    """q [Tq][d], K, V [n][d] fp64 -> out, lse, weights [Tq][n], the scale of the output's error terms
    (sum p |v|) and the largest sum of |q k| behind a score."""
    c = 1.0 / math.sqrt(q.shape[1])
    m = seen(pos, K.shape[0], window, sinks)
    s = torch.where(m, (q @ K.T) * c, torch.tensor(-math.inf, dtype=torch.float64))
    top = s.max(1, keepdim=True).values if K.shape[0] else torch.full((q.shape[0], 1), -math.inf, dtype=torch.float64)
    e = torch.where(m, (s - torch.where(top == -math.inf, 0.0, top)).exp(), torch.tensor(0.0, dtype=torch.float64))
    l = e.sum(1, keepdim=True)
    w = torch.where(l > 0, e / torch.where(l > 0, l, 1.0), 0.0)
    # 0 x NaN in a place that is not seen is nothing
    seen_v = torch.where(m.any(0)[:, None], V, 0.0)
    out = w @ seen_v
    lse = torch.where(l > 0, top + l.log(), -math.inf)[:, 0]
    big = float((torch.where(m, (q.abs() @ K.abs().T) * c, 0.0)).max()) if K.shape[0] else 0.0
    return out, lse, w, w @ seen_v.abs(), big


def score_error(d, big):
    """Bound of a score's error: products are exact in fp32, the tensor cores add d of them one by one or
    in groups, truncating, each addition off by at most 2^-23 of a partial sum that is at most `big`; the
    scaling to base 2, the subtraction of the maximum and ex2 add a few 2^-23 of values of that size."""
    return (d + 8) * 2.0 ** -23 * max(big, 1.0)


def check_rows(out, lse, ref, d, dt, p_eps, what=""):
    """out [Tq][d], lse [Tq] against attend()'s.  The errors: the output's rounding (half a step of its
    type), p's rounding p_eps, and the scores' errors, which move a weight and the sum they are divided by:
    twice score_error, relative, on sum p |v|."""
    o, l, _, scale, big = ref
    u, ds = torch.finfo(dt).eps / 2, score_error(d, big)
    tiny = torch.finfo(dt).smallest_normal * torch.finfo(dt).eps  # half a step of subnormals, and a spare half
    tol = u * o.abs() + (p_eps + 2 * ds) * (1 + u) * scale + tiny
    err = (out.double().cpu() - o).abs()
    assert bool((err <= tol).all()), f"{what}: out off by {float((err / tol.clamp(min=1e-300)).max()):.2f} of its bound"
    if lse is not None:
        got = lse.double().cpu()
        assert torch.equal(torch.isneginf(got), torch.isneginf(l)), f"{what}: empty rows"
        f = ~torch.isneginf(l)
        bound = ds + 2.0 ** -22 * l[f].abs().clamp(min=1.0)
        assert bool(((got[f] - l[f]).abs() <= bound).all()), f"{what}: lse off by {float((got[f] - l[f]).abs().max())}"


def evict(weights, n, budget, first, recent):
    """Positions kept of n tokens with these weights (a list of floats)."""
    if n <= budget:
        return list(range(n))
    w = [-math.inf if math.isnan(x) else x for x in weights]
    must = set(range(first)) | set(range(n - recent, n))
    rest = sorted((t for t in range(n) if t not in must), key=lambda t: (-w[t], t))
    return sorted(list(must) + rest[:budget - len(must)])
