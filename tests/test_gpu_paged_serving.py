"""The paged cache as a serving program meets it: batches that hold a sequence
which does not fit, the documented loop, captured loops, what is left after an
eviction."""
import os
import re
import types

import pytest
import torch

import _paged as ref
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
    """The documented serving loop, word for word: prompts' chunks beside single tokens, then generation until rows go."""
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


# ------------------------------------------------------------------ captured

@pytest.mark.parametrize("lens,news,Hk,keep", [
    ([40, 90], [1, 1], 2, 30),
    ([5000, 70], [1, 1], 2, 600),     # a head's rows over a cluster of CTAs
    ([300, 90, 0], [40, 1, 9], 1, 50),  # a chunk
])
def test_a_captured_loop_with_eviction(lens, news, Hk, keep):
    """Append, attend, weigh, select and move in one CUDA graph; two graphs share the workspaces. Replayed on new inputs
    from the same rows, they leave what the calls themselves leave, bit for bit."""
    c = Case(lens, news, 4, Hk, 64, 16, cap=max(lens) + 60, seed=72).fill()
    batch = c.batch()
    after = cs.PagedBatch(batch.page_table, batch.cache_len + torch.tensor(news, **I32))
    next_pos = after.cache_len.clone()
    cache = pools(c)
    q, k, v = (torch.empty(c.N, h, 64, dtype=BF, device="cuda") for h in (4, Hk, Hk))
    scratch = lambda n: torch.empty(max(1, n), dtype=torch.uint8, device="cuda")  # noqa: E731
    ws = scratch(cs.attn_paged_workspace_bytes(c.spec, batch, cache))
    wws = scratch(cs.attn_paged_weigh_workspace_bytes(c.spec, batch, cache))
    begin = [c.k_pages.cuda(), c.v_pages.cuda(), c.randn(c.n_pages, Hk, 16).abs().cuda(),
             torch.randint(0, min(lens) + 1, (c.n_pages, Hk, 16), generator=c.g, dtype=torch.int32).cuda()]

    def buffers():
        return [torch.zeros(c.N, 4, 64, dtype=BF, device="cuda"), torch.zeros(c.N, 4, 64, dtype=BF, device="cuda"),
                torch.zeros(c.N, 4, device="cuda"), torch.zeros(c.B, Hk, **I32), torch.zeros(c.B, Hk, keep, **I32),
                torch.zeros(c.B, Hk, keep, **I32), torch.zeros(c.B, **I32)]

    def step(q_out, O, lse, n_moves, src, dst, new_len):
        cs.attn_paged_append(c.spec, batch, cache, q, k, v, None, None, q_out)
        cs.attn_paged(c.spec, batch, cache, q_out, O, lse, ws)
        cs.attn_paged_weigh(c.spec, batch, cache, q_out, lse, workspace=wws)
        cs.attn_paged_select(c.spec, after, cache, next_pos, keep, 9, n_moves, src, dst, new_len)
        cs.attn_paged_move(c.spec, after, cache, n_moves, src, dst)

    def everything(run, bufs):
        held = [cache.k, cache.v, cache.weight, cache.position]
        for t, was in zip(held, begin):
            t.copy_(was)
        run()
        torch.cuda.synchronize()
        return [t.clone() for t in bufs + held]
    warm = buffers()
    for t in (q, k, v):
        t.normal_()
    step(*warm)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        bufs, gr = buffers(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            step(*bufs)
        graphs.append((gr, bufs))
    last = None
    for _ in range(3):
        for t in (q, k, v):
            t.normal_()
        want = everything(lambda: step(*warm), warm)
        assert (want[3] > 0).any() and want[6].tolist() == [min(keep, a + n) for a, n in zip(lens, news)]
        bits = lambda t: t.view(torch.int16 if t.dtype == BF else torch.int32)  # noqa: E731
        assert last is None or not torch.equal(bits(last[1]), bits(want[1]))
        last = want
        for gr, bufs in graphs:
            got = everything(gr.replay, bufs)
            assert all(torch.equal(bits(a), bits(b)) for a, b in zip(got, want))
    cs.cswattn_sync_status()


# ------------------------------------------------------------------ after an eviction

@pytest.mark.parametrize("rope", [None, cs.RopeSpec(64, interleaved=True, scaling="yarn", factor=4.0, original_length=64)])
@pytest.mark.parametrize("H,Hk,D,page,keep,recent", [(4, 2, 64, 16, 50, 12), (6, 2, 128, 32, 77, 0), (8, 1, 64, 48, 40, 40)])
def test_attention_over_what_is_left(H, Hk, D, page, keep, recent, rope):
    """A model of the cache on the CPU, a list of rows for each head, goes through the same steps: the attention and the
    weights of every call are those of the model's rows in 64 bits, and after each eviction the cache holds the model's
    rows, bit for bit and in its order. (The model takes new rows and weights as the calls wrote them, once checked.)"""
    B, T, grp = 3, 160, H // Hk
    g = torch.Generator().manual_seed(73)
    spec = cs.LayerSpec(B, T, H, Hk, D, T, has_ve=False)
    pps = -(-T // page)
    table = torch.randperm(B * pps + 2, generator=g)[: B * pps].view(B, pps).to(torch.int32)
    cache = cs.PagedCache(spec, n_pages=B * pps + 2, page_size=page, track_weights=True)
    cache.k.fill_(float("nan")), cache.v.fill_(float("nan"))
    length, next_pos = torch.zeros(B, **I32), torch.zeros(B, **I32)
    model = [[dict(k=torch.empty(0, D, dtype=BF), v=torch.empty(0, D, dtype=BF), w=torch.empty(0),
                   p=torch.empty(0, dtype=torch.int32)) for _ in range(Hk)] for _ in range(B)]
    moved = evicted = 0

    def held(b, h, lo, hi):
        r = torch.arange(lo, hi)
        p, o = table[b].long()[r // page], r % page
        return dict(k=cache.k.cpu()[p, o, h], v=cache.v.cpu()[p, o, h], w=cache.weight.cpu()[p, h, o],
                    p=cache.position.cpu()[p, h, o])
    for news in ([60, 3, 0], [1, 1, 90], [1, 1, 1], [40, 60, 1], [1, 0, 1], [1, 1, 1], [1, 1, 1], [30, 2, 5]):
        N, lens = sum(news), length.tolist()
        start = [sum(news[:b]) for b in range(B + 1)]
        q, k, v = (torch.randn(N, h, D, generator=g).to(BF).cuda() for h in (H, Hk, Hk))
        positions = torch.cat([next_pos[b] + torch.arange(news[b], **I32) for b in range(B)])
        batch = cs.PagedBatch(table.cuda(), length, torch.tensor(start, **I32), N, max(news))
        q_out, O, lse = torch.empty_like(q), torch.empty_like(q), torch.empty(N, H, device="cuda")
        ws = torch.empty(cs.attn_paged_workspace_bytes(spec, batch, cache), dtype=torch.uint8, device="cuda")
        cs.attn_paged_append(spec, batch, cache, q, k, v, None, None, q_out, positions=positions, rope=rope)
        cs.attn_paged(spec, batch, cache, q_out, O, lse, ws)
        cs.attn_paged_weigh(spec, batch, cache, q_out, lse)
        cs.cswattn_sync_status()
        qd, Od, ld = q_out.double().cpu(), O.double().cpu(), lse.double().cpu()
        for b in range(B):
            L, n = lens[b], news[b]
            seen = torch.arange(L + n) <= L + torch.arange(n)[:, None]
            for h in range(Hk):
                m, new = model[b][h], held(b, h, L, L + n)
                assert new["p"].tolist() == list(range(int(next_pos[b]), int(next_pos[b]) + n))
                new["w"] = torch.zeros(n)
                m = {x: torch.cat([m[x], new[x]]) for x in m}
                weight, tol_w = m["w"].double(), torch.zeros(L + n, dtype=torch.float64)
                for e in range(h * grp, (h + 1) * grp):
                    t = slice(start[b], start[b] + n)
                    s = (qd[t, e] @ m["k"].double().T) * D ** -0.5
                    mag = (qd[t, e].abs() @ m["k"].double().abs().T) * D ** -0.5
                    s = s.masked_fill(~seen, -float("inf"))
                    z = torch.logsumexp(s, -1)
                    prob = torch.exp(s - z[:, None])
                    # the bounds of tests/_paged.py: a score off by ds, half a bf16 step of each probability and output
                    ds = D * 2.0 ** -23 * mag.masked_fill(~seen, 0.0) + 2.0 ** -20 * (1 + z.abs()[:, None])
                    top = ds.amax(-1) if n else z
                    want = prob @ m["v"].double()
                    tol = (2.0 ** -8 + 2 * top[:, None]) * (prob @ m["v"].double().abs()) + 2.0 ** -8 * want.abs()
                    assert ((Od[t, e] - want).abs() <= tol + 1e-30).all() and ((ld[t, e] - z).abs() <= 2 * top).all()
                    x = torch.exp(s - ld[t, e][:, None])
                    weight += x.sum(0)
                    tol_w += (x * 2 * ds).sum(0) + x.sum(0) * n * grp * 2.0 ** -24
                now = held(b, h, 0, L + n)
                assert ((now["w"].double() - weight).abs() <= tol_w + 2.0 ** -23 * weight).all()
                m["w"] = now["w"]
                model[b][h] = m
        length += torch.tensor(news, **I32)
        next_pos += torch.tensor(news, **I32)
        n_moves, new_len = torch.empty(B, Hk, **I32), torch.empty(B, **I32)
        src, dst = torch.empty(B, Hk, keep, **I32), torch.empty(B, Hk, keep, **I32)
        after = cs.PagedBatch(table.cuda(), length)
        cs.attn_paged_select(spec, after, cache, next_pos, keep, recent, n_moves, src, dst, new_len)
        cs.attn_paged_move(spec, after, cache, n_moves, src, dst)
        cs.cswattn_sync_status()
        for b in range(B):
            for h in range(Hk):
                m = model[b][h]
                s, d = ref.select(m["w"].tolist(), m["p"].tolist(), int(next_pos[b]), int(length[b]), keep, recent)
                moved += len(s)
                evicted += max(0, int(length[b]) - keep)
                for x in m:
                    m[x][d] = m[x][s]
                    m[x] = m[x][:keep].clone()
                now = held(b, h, 0, int(new_len[b]))
                for x in m:
                    assert torch.equal(now[x].view(torch.int16) if now[x].dtype == BF else now[x],
                                       m[x].view(torch.int16) if m[x].dtype == BF else m[x]), x
        length = new_len
    assert evicted > 20 and moved > 0  # the steps above do both


# ------------------------------------------------------------------ rotations

@pytest.mark.parametrize("base,kw", [(5e5, {}), (1e4, {}), (3e6, dict(scaling="linear", factor=4.0)),
                                     (5e5, dict(scaling="yarn", factor=4.0, original_length=65536, interleaved=True))])
def test_append_turns_by_the_layers_base(base, kw):
    """A rotation that names no base is the layer's: without scaling the bits of rope=None, else the definition."""
    H, Hk, D = 3, 1, 128
    c = Case([5], [40], H, Hk, D, 16, cap=64, seed=74)
    c.spec.rope_base = base
    q, k = c.randn(c.N, H, D).to(BF), c.randn(c.N, Hk, D).to(BF)
    pos = torch.arange(c.N) * 1571
    outs = []
    rope = cs.RopeSpec(D, **kw)
    for r in (rope, None if not kw else cs.RopeSpec(D, base=base, **kw)):
        cache, q_out = pools(c), torch.empty_like(q).cuda()
        cs.attn_paged_append(c.spec, c.batch(), cache, q.cuda(), k.cuda(), k.cuda(), None, None, q_out,
                             positions=pos.to(torch.int32).cuda(), rope=r)
        cs.cswattn_sync_status()
        outs.append([q_out, cache.k])
    assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(*outs))
    w = [base ** (-2 * i / D) for i in range(D // 2)]
    if kw.get("scaling") == "linear":
        w = [x / 4 for x in w]
    elif kw:
        w = cs.RopeSpec(D, base=base, **kw).frequencies  # (tested against the definition on the CPU)
    factor = rope.attention_factor
    want = ref.rope(q, pos, w, factor, kw.get("interleaved", False))
    relative, absolute = ref.rope_tol(q, 12 * factor)  # a normalised element is at most sqrt(128)
    assert ((outs[0][0].double().cpu() - want).abs() <= relative * want.abs() + absolute).all()
