"""The paged attention and row weights where every CTA has long runs of blocks:
rings that turn many times, maxima that grow late, tiles of different ranges
over the same blocks. Compared with the definitions in 64 bits, computed on
the GPU by plain products.
"""
import math

import pytest
import torch

import causal_sliding_window_rope_b200 as cs
from _paged import BF, NAN, Case

pytestmark = pytest.mark.gpu


def fill(c, q):
    """Pools on the GPU: random rows for every sequence, NaN where no row is. Some late rows are copies of queries, so
    that the maximum of a query's row grows by far in its last blocks."""
    g = torch.Generator(device="cuda").manual_seed(c.N + c.B)
    k = torch.randn(c.n_pages, c.page, c.Hk, c.D, generator=g, device="cuda")
    k = (k * torch.rsqrt(k.square().mean(-1, keepdim=True))).to(BF)
    v = torch.randn(c.n_pages, c.page, c.Hk, c.D, generator=g, device="cuda").to(BF)
    grp, used = c.H // c.Hk, torch.zeros(c.n_pages, c.page, dtype=torch.bool, device="cuda")
    for b in range(c.B):
        end = c.lens[b] + c.news[b]
        rows = torch.arange(end)
        p, o = c.table[b].long()[rows // c.page].cuda(), (rows % c.page).cuda()
        used[p, o] = True
        if c.news[b] and end > 8:
            for r in torch.randint(3 * end // 4, end, (6,), generator=c.g).tolist():
                token = c.start[b] + int(torch.randint(0, c.news[b], (1,), generator=c.g))
                head = int(torch.randint(0, grp, (1,), generator=c.g))
                k[p[r], o[r]] = q[token, head::grp]
    k[~used], v[~used] = NAN, NAN
    return k, v


def definition(c, q, k, v, lse_in=None, weight=None):
    """O, lse and their bounds; or, with lse_in, weight + the sums and their bound. The bounds are those of
    tests/_paged.py (half a bf16 step for each probability and output; a score off by D 2^-23 of its terms' magnitudes)
    and for the long sums float32's 2^-24 a term."""
    f64 = dict(dtype=torch.float64, device="cuda")
    O, lse = torch.full((c.N, c.H, c.D), NAN, **f64), torch.full((c.N, c.H), NAN, **f64)
    tO, tl = torch.zeros_like(O), torch.zeros_like(lse)
    out = tw = None
    if weight is not None:
        out, tw = weight.double(), torch.zeros(weight.shape, **f64)
    grp = c.H // c.Hk
    for b in range(c.B):
        L, n = c.lens[b], c.news[b]
        rows = torch.arange(L + n, device="cuda")
        p, o = c.table[b].long().cuda()[rows // c.page], rows % c.page
        for i0 in range(0, n, 512):
            i1 = min(n, i0 + 512)
            t = slice(c.start[b] + i0, c.start[b] + i1)
            row = L + torch.arange(i0, i1, device="cuda")[:, None]
            seen = (rows <= row) & (rows > row - c.W)
            for h in range(c.H):
                qh, kh = q[t, h].double(), k[p, o, h // grp].double()
                s = (qh @ kh.T) * c.scale
                mag = (qh.abs() @ kh.abs().T) * c.scale
                if weight is None:
                    vh = v[p, o, h // grp].double()
                    z = torch.logsumexp(s.masked_fill(~seen, -math.inf), -1)
                    prob = torch.exp(s - z[:, None]).masked_fill(~seen, 0.0)
                    O[t, h], lse[t, h] = prob @ vh, z
                    ds = c.D * 2.0 ** -23 * mag.masked_fill(~seen, 0.0).amax(-1) + 2.0 ** -20 * (1 + z.abs())
                    ds = 2 * ds + seen.sum(-1) * 2.0 ** -24
                    tO[t, h] = (2.0 ** -8 + ds[:, None]) * (prob @ vh.abs()) + 2.0 ** -8 * O[t, h].abs() + 1e-30
                    tl[t, h] = ds
                else:
                    z = lse_in[t, h].double()[:, None]
                    x = torch.exp(s - z).masked_fill(~seen, 0.0)
                    ds = c.D * 2.0 ** -23 * mag + 2.0 ** -20 * (1 + z.abs())
                    out[p, h // grp, o] += x.sum(0)
                    tw[p, h // grp, o] += (x * 2 * ds).sum(0) + x.sum(0) * n * grp * 2.0 ** -24
    return (O, lse, tO, tl) if weight is None else (out, tw + 2.0 ** -23 * out.abs())


def within(got, want, tol, what):
    ok = torch.isfinite(want)
    assert torch.isfinite(got[ok]).all(), what
    over = (got.double()[ok] - want[ok]).abs() - tol[ok]
    assert over.max() <= 0, f"{what}: {int((over > 0).sum())} of {over.numel()} values past the bound by up to {float(over.max()):.3g}"


def check(c):
    q = c.queries().cuda()
    k, v = fill(c, q)
    batch = c.batch()
    w0 = torch.rand(c.n_pages, c.Hk, c.page, device="cuda")
    cache = cs.PagedCache(c.spec, k=k, v=v, weight=w0.clone())
    ws = torch.empty(cs.attn_paged_workspace_bytes(c.spec, batch, cache), dtype=torch.uint8, device="cuda")
    wO, wl, tO, tl = definition(c, q, k, v)
    lse_in = wl.float()
    ww, tw = definition(c, q, k, v, lse_in, w0)
    seen = ww != w0.double()
    first = None
    for _ in range(3):
        O, lse = torch.full((c.N, c.H, c.D), 5.0, dtype=BF, device="cuda"), torch.full((c.N, c.H), 5.0, device="cuda")
        cs.attn_paged(c.spec, batch, cache, q, O, lse, ws)
        cache.weight.copy_(w0)
        cs.attn_paged_weigh(c.spec, batch, cache, q, lse_in)
        cs.cswattn_sync_status()
        within(O, wO, tO, "O")
        within(lse, wl, tl, "lse")
        within(cache.weight, ww, tw, "weight")
        assert torch.equal(cache.weight[~seen], w0[~seen])
        n = c.start[-1]
        assert (O[n:] == 5.0).all() and (lse[n:] == 5.0).all()
        now = (O, lse, cache.weight.clone())
        assert first is None or all(torch.equal(a, b) for a, b in zip(first, now))
        first = now


def lengths(B, lo, hi, seed):
    return torch.randint(lo, hi + 1, (B,), generator=torch.Generator().manual_seed(seed)).tolist()


FEW = [
    # B, lens, most new tokens, H, Hk, D, page, W, scale
    (32, (1500, 4500), 1, 12, 4, 128, 64, None, 0.0),    # 3 query rows: 40 blocks a CTA, 5 turns of 8 slots
    (32, (1500, 4500), 4, 12, 4, 128, 48, None, 0.0),    # 12
    (32, (1500, 4500), 8, 12, 4, 128, 16, None, 0.4),    # 24
    (32, (2500, 5500), 1, 12, 4, 64, 128, None, 0.0),    # 54 blocks a CTA, 3 turns of 16 slots
    (32, (2500, 5500), 5, 12, 4, 64, 32, None, 0.5),
    (32, (2500, 5500), 6, 16, 4, 64, 16, 3500, 0.0),
    (1, (300000, 300000), 1, 8, 2, 128, 256, None, 0.0),  # one sequence over every SM
    (9, (20000, 40000), 2, 6, 1, 128, 64, 25000, 0.0),
]


@pytest.mark.parametrize("B,lens,new,H,Hk,D,page,W,scale", FEW)
def test_few_query_rows(B, lens, new, H, Hk, D, page, W, scale):
    lens = lengths(B, *lens, seed=B + new)
    news = [new] + lengths(B - 1, 1, new, seed=7)
    c = Case(lens, news, H, Hk, D, page, W=W, seed=H + new, pad=3, scale=scale)
    check(c)


MANY = [
    ([4096, 4096], [1024, 1024], 16, 4, 128, 128, None, 0.0),   # over 30 blocks a CTA
    ([4000, 1500, 77], [700, 1300, 1], 16, 4, 128, 48, 900, 0.4),
    ([6000, 0, 333], [900, 1500, 40], 10, 2, 64, 64, None, 0.0),  # 25 tokens a tile
    ([5000, 3000], [800, 1100], 8, 4, 64, 16, 2000, 0.5),
    ([100] * 64, [300] * 64, 16, 4, 128, 32, None, 0.0),         # many units of few blocks a CTA
    ([60000], [200], 8, 2, 128, 256, None, 0.0),
    ([40, 2000] * 20, [150, 1] * 20, 6, 2, 64, 32, 500, 0.0),
]


@pytest.mark.parametrize("lens,news,H,Hk,D,page,W,scale", MANY, ids=[f"{len(m[0])}seq-{max(m[0])}+{max(m[1])}-D{m[4]}" for m in MANY])
def test_many_query_rows(lens, news, H, Hk, D, page, W, scale):
    check(Case(lens, news, H, Hk, D, page, W=W, seed=H + max(news), pad=1, scale=scale))
