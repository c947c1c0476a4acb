"""The paged cache as a serving program meets it: batches that hold a sequence
which does not fit, the documented loop, captured loops, what is left after an
eviction."""
import os
import re
import types

import pytest
import torch

import causal_sliding_window_rope_b200 as cs
from _paged import BF, Case

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device="cuda")


def pools(c, weight=7.0):
    return cs.PagedCache(c.spec, k=c.k_pages.cuda(), v=c.v_pages.cuda(),
                         weight=torch.full((c.n_pages, c.Hk, c.page), weight, device="cuda"),
                         position=torch.full((c.n_pages, c.Hk, c.page), -5, **I32))


@pytest.mark.parametrize("start,max_new", [
    ([0, 1000, 5, 8], 5),                  # the first has more tokens than there are
    ([0, 7, 5, 8], 5),                     # ... than a sequence may have
    ([-2, 6, 5, 8], 8),                    # ... a start before the first token
    ([-(2 ** 31), 2 ** 31 - 1, 5, 8], 8),
    ([5, 8, -(2 ** 31), 2 ** 31 - 1], 8),  # the one that fits comes first
])
def test_tokens_of_a_sequence_beside_one_that_does_not_fit(start, max_new):
    """Tokens 5 to 7 are a sequence's that fits, and lie in the range of one that does not: their rows are written as
    without it, and its own are left alone."""
    c = Case([20, 9, 33], [5, 0, 3], 4, 2, 64, 16, seed=70).fill(upto_new=False)
    q, k, v = (c.randn(c.N, h, 64).to(BF).cuda() for h in (4, 2, 2))
    good = start.index(5) if start[0] == 5 else 2
    lens = [20, 9, 33]
    lens[good], lens[2] = 33, lens[good]
    table = c.table.clone()
    table[good], table[2] = c.table[2], c.table[good]
    outs = []
    for s in ([5] * (good + 1) + [8] * (3 - good), start):  # the sequence that fits alone, then beside the others
        cache, q_out = pools(c), torch.full((8, 4, 64), 3.0, dtype=BF, device="cuda")
        batch = cs.PagedBatch(table.cuda(), torch.tensor(lens, **I32), torch.tensor(s, **I32), 8, max_new)
        cs.attn_paged_append(c.spec, batch, cache, q, k, v, None, None, q_out)
        if s is start:
            with pytest.raises(cs.CswattnError) as err:
                cs.cswattn_sync_status()
            assert err.value.status == cs.ERR_INVALID_ARG
        else:
            cs.cswattn_sync_status()
        outs.append([q_out, cache.k, cache.v, cache.weight, cache.position])
    p, o = c.place(2, 33 + 2)
    assert torch.equal(outs[0][2][p, o], v[7]) and int(outs[0][4][p, 0, o]) == 35
    for alone, beside in zip(*outs):
        assert torch.equal(alone.view(torch.int16 if alone.dtype == BF else torch.int32),
                           beside.view(torch.int16 if beside.dtype == BF else torch.int32))


def test_the_documented_loop():
    """README's serving loop, word for word: prompts' chunks beside single tokens, then generation until rows go."""
    readme = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")).read()
    code = re.search(r"A serving loop over a paged cache.*?```python\n(.*?)```", readme, re.S).group(1)
    g = torch.Generator(device="cuda").manual_seed(71)
    B, H, Hk, D, K = 32, 16, 4, 128, 4096
    length, next_pos = torch.zeros(B, **I32), torch.zeros(B, **I32)
    page_table = torch.randperm(4096, generator=g, device="cuda").to(torch.int32).view(B, 128)
    total = [0] * B
    for news in ([2500, 1, 7] + [0] * 29, [2500] + [60] * 31, [1] * B, [0, 1] * 16):
        start = torch.tensor([sum(news[:b]) for b in range(B + 1)], **I32)
        N, most = sum(news), max(news)
        r = lambda h: torch.randn(N, h, D, generator=g, device="cuda").to(BF)  # noqa: E731
        q, k, v = r(H), r(Hk), r(Hk)
        token = torch.arange(N, device="cuda")
        b = torch.searchsorted(start[1:].long(), token, right=True)
        positions = (next_pos[b] + token - start[b]).to(torch.int32)
        next_pos += start[1:] - start[:-1]
        q_out, O = torch.empty_like(q), torch.full_like(q, float("nan"))
        lse = torch.full((N, H), float("nan"), device="cuda")
        n_moves, new_len = torch.empty(B, Hk, **I32), torch.empty(B, **I32)
        src, dst = torch.empty(B, Hk, K, **I32), torch.empty(B, Hk, K, **I32)
        space = dict(locals(), torch=torch, cs=cs)
        if total[0]:
            space["cs"] = types.SimpleNamespace(**{**vars(cs), "PagedCache": lambda *a, **kw: cache})  # the one there is
        exec(code, space)
        cache = space["cache"]
        cs.cswattn_sync_status()
        total = [min(K, t + n) for t, n in zip(total, news)]
        assert length.tolist() == total and torch.isfinite(O.float()).all() and torch.isfinite(lse).all()
        assert (n_moves[1:] == 0).all() and bool((n_moves[0] > 0).all()) == (news[0] > 0 and total[0] == K)
