"""The paged cache as a serving program meets it: batches that hold a sequence
which does not fit, the documented loop, captured loops, what is left after an
eviction."""
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
