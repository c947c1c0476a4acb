"""Paged-cache test cases: random batches on the CPU and the definitions in 64 bits.

Rows that nobody may read are NaN (pages of nobody, rows past a sequence's
end), so that a kernel that let one of them into a sum would show it.
"""
from __future__ import annotations

import math

import torch

import causal_sliding_window_rope_b200 as cs

BF = torch.bfloat16
NAN = float("nan")


class Case:
    """lens: rows before the call; news: new tokens of each sequence."""

    def __init__(self, lens, news, H, Hk, D, page, W=None, cap=None, pad=0, ve=False, seed=0, spare=3, max_new=None,
                 scale=0.0):
        g = torch.Generator().manual_seed(1000 + seed)
        self.g = g
        self.lens, self.news, self.H, self.Hk, self.D, self.page = list(lens), list(news), H, Hk, D, page
        self.B = len(lens)
        need = max(L + n for L, n in zip(lens, news))
        self.cap = cap or max(1, need)
        self.W = W or self.cap
        self.pps = -(-self.cap // page)
        self.n_pages = self.B * self.pps + spare
        self.table = torch.randperm(self.n_pages, generator=g)[: self.B * self.pps].view(self.B, self.pps).to(torch.int32)
        self.start = [0]
        for n in news:
            self.start.append(self.start[-1] + n)
        self.N = self.start[-1] + pad
        self.max_new = max_new or max(1, max(news))
        self.spec = cs.LayerSpec(self.B, self.cap, H, Hk, D, self.W, has_ve=ve, softmax_scale=scale)
        self.scale = scale or D ** -0.5
        self.k_pages = torch.full((self.n_pages, page, Hk, D), NAN, dtype=BF)
        self.v_pages = torch.full((self.n_pages, page, Hk, D), NAN, dtype=BF)

    def randn(self, *shape):
        return torch.randn(*shape, generator=self.g)

    def place(self, b, row):
        return int(self.table[b, row // self.page]), row % self.page

    def fill(self, upto_new=True):
        """Random rows for every sequence: k of root mean square 1, as the prologue leaves them."""
        for b in range(self.B):
            rows = torch.arange(self.lens[b] + (self.news[b] if upto_new else 0))
            p, o = self.table[b].long()[rows // self.page], rows % self.page
            k = self.randn(len(rows), self.Hk, self.D)
            self.k_pages[p, o] = (k / k.square().mean(-1, keepdim=True).sqrt()).to(BF)
            self.v_pages[p, o] = self.randn(len(rows), self.Hk, self.D).to(BF)
        return self

    def queries(self):
        q = self.randn(self.N, self.H, self.D)
        return (q / q.square().mean(-1, keepdim=True).sqrt()).to(BF)

    def batch(self, device="cuda"):
        return cs.PagedBatch(self.table.to(device), torch.tensor(self.lens, dtype=torch.int32, device=device),
                             torch.tensor(self.start, dtype=torch.int32, device=device), self.N, self.max_new)

    def rows_of(self, b, pool):
        rows = torch.arange(self.lens[b] + self.news[b])
        return pool[self.table[b].long()[rows // self.page], rows % self.page]


def attention(c: Case, q):
    """Per sequence, in 64 bits: probabilities' outputs and their bounds.

    Returns O, lse and elementwise bounds for a kernel that rounds each
    probability to bf16 (half a step, 2^-8 of it), the output to bf16, and
    sums products in float32 (D terms, each sum off by at most 2^-23 of the
    partial sum, so the score by D 2^-23 of the sum of magnitudes)."""
    O = torch.full((c.N, c.H, c.D), NAN, dtype=torch.float64)
    lse = torch.full((c.N, c.H), NAN, dtype=torch.float64)
    tol_O, tol_l = torch.zeros_like(O), torch.zeros_like(lse)
    grp = c.H // c.Hk
    for b in range(c.B):
        L, n = c.lens[b], c.news[b]
        if n == 0:
            continue
        t = slice(c.start[b], c.start[b] + n)
        k, v = c.rows_of(b, c.k_pages).double(), c.rows_of(b, c.v_pages).double()
        row = L + torch.arange(n)[:, None]
        key = torch.arange(L + n)[None, :]
        seen = (key <= row) & (key > row - c.W)
        for h in range(c.H):
            qh, kh, vh = q[t, h].double(), k[:, h // grp], v[:, h // grp]
            s = (qh @ kh.T) * c.scale
            mag = ((qh.abs() @ kh.abs().T) * c.scale).masked_fill(~seen, 0.0).amax(-1)
            s = s.masked_fill(~seen, -math.inf)
            z = torch.logsumexp(s, -1)
            p = torch.exp(s - z[:, None])
            O[t, h], lse[t, h] = p @ vh, z
            ds = c.D * 2.0 ** -23 * mag + 2.0 ** -20 * (1 + z.abs())  # error of a score, and of log2/exp2
            spread = p @ vh.abs()
            tol_O[t, h] = (2.0 ** -8 + 2 * ds[:, None]) * spread + 2.0 ** -8 * O[t, h].abs() + 1e-30
            tol_l[t, h] = 2 * ds
    return O, lse, tol_O, tol_l


def weights(c: Case, q, lse, weight):
    """weight + the sums, and the bound of a float32 kernel's error."""
    out, tol = weight.double().clone(), torch.zeros(weight.shape, dtype=torch.float64)
    grp = c.H // c.Hk
    for b in range(c.B):
        L, n = c.lens[b], c.news[b]
        if n == 0:
            continue
        t = slice(c.start[b], c.start[b] + n)
        k = c.rows_of(b, c.k_pages).double()
        rows = torch.arange(L + n)
        p, o = c.table[b].long()[rows // c.page], rows % c.page
        row = L + torch.arange(n)[:, None]
        seen = (rows[None, :] <= row) & (rows[None, :] > row - c.W)
        for h in range(c.H):
            s = (q[t, h].double() @ k[:, h // grp].T) * c.scale
            mag = (q[t, h].double().abs() @ k[:, h // grp].abs().T) * c.scale
            x = torch.exp(s - lse[t, h].double()[:, None]).masked_fill(~seen, 0.0)
            ds = c.D * 2.0 ** -23 * mag + 2.0 ** -20 * (1 + lse[t, h].double().abs()[:, None])
            out[p, h // grp, o] += x.sum(0)
            tol[p, h // grp, o] += (x * 2 * ds).sum(0) + x.sum(0) * n * grp * 2.0 ** -24
    return out, tol + 2.0 ** -23 * out.abs()


def rope(x, pos, freq, factor, interleaved):
    """RMSNorm (eps 1e-6) and rotation in 64 bits; x (tokens, heads, D)."""
    x = x.double()
    x = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt()
    R = 2 * len(freq)
    a = torch.as_tensor(pos, dtype=torch.float64)[:, None, None] * torch.tensor(freq, dtype=torch.float64)
    cos, sin = a.cos() * factor, a.sin() * factor
    y = x.clone()
    i = torch.arange(R // 2)
    lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
    y[..., lo] = x[..., lo] * cos - x[..., hi] * sin
    y[..., hi] = x[..., lo] * sin + x[..., hi] * cos
    return y


def rope_tol(x, pos_freq_factor):
    """Half a bf16 step of the result, and float32 arithmetic on terms as large as a row's largest."""
    return 2.0 ** -8, 2.0 ** -19 * pos_freq_factor


def select(weight, position, next_pos, L, n_keep, n_recent):
    """(src, dst) of one head by plain sorting of Python tuples; weight, position: its L rows in order."""
    if L <= n_keep:
        return [], []

    def order(r):
        w = float(weight[r])
        if position[r] >= next_pos - n_recent:
            return (0, 0, 0.0, r)
        return (1, 1 if math.isnan(w) else 0, 0.0 if math.isnan(w) else -w, r)
    kept = set(sorted(range(L), key=order)[:n_keep])
    return sorted(r for r in kept if r >= n_keep), [r for r in range(n_keep) if r not in kept]
