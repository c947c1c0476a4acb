"""The paged cache on the GPU against the definitions in 64 bits (tests/_paged.py),
each operator alone and all of them as a serving loop uses them.

Bounds are elementwise and derived there: half a bf16 step for each rounding
(of the probabilities, of the output), float32 arithmetic for the rest.
"""
import numpy as np
import pytest
import torch

import causal_sliding_window_rope_b200 as cs
import _paged as ref
from _paged import BF, NAN, Case

pytestmark = pytest.mark.gpu


def within(got, want, tol, what):
    got = got.double().cpu()
    ok = torch.isfinite(want)
    assert torch.isfinite(got[ok]).all(), what
    over = ((got[ok] - want[ok]).abs() - tol[ok])
    assert over.numel() == 0 or over.max() <= 0, f"{what}: {int((over > 0).sum())} of {over.numel()} values past the bound by up to {over.max():.3g}"


# ------------------------------------------------------------------ append

APPEND = [
    # lens, news, H, Hk, D, page, rotary, interleaved, ve, positions, pad
    ([0], [1], 2, 1, 128, 16, 128, False, True, False, 0),
    ([5, 0, 31], [3, 0, 17], 6, 2, 128, 16, 128, False, True, False, 4),
    ([100, 7], [9, 30], 4, 4, 64, 48, 64, True, False, True, 1),
    ([0, 63, 64], [65, 1, 2], 3, 1, 64, 64, 16, False, True, True, 0),
    ([1, 2, 3, 4], [1, 1, 1, 1], 12, 4, 128, 32, 64, True, True, True, 9),
    ([17], [40], 5, 5, 128, 16, 48, False, False, True, 0),
    ([11] * 300, [1, 0, 2] * 100, 2, 2, 64, 16, 64, False, False, False, 7),
    ([3], [20], 16, 1, 128, 256, 112, True, True, True, 0),
]


@pytest.mark.parametrize("lens,news,H,Hk,D,page,rotary,inter,ve,given,pad", APPEND)
def test_append(lens, news, H, Hk, D, page, rotary, inter, ve, given, pad):
    c = Case(lens, news, H, Hk, D, page, ve=ve, pad=pad, seed=H + D + rotary).fill(upto_new=False)
    q, k, v = (c.randn(c.N, h, D).to(BF) for h in (H, Hk, Hk))
    e = c.randn(c.N, Hk, D).to(BF) if ve else None
    gate = c.randn(c.N, Hk).to(BF) if ve else None
    row = torch.cat([L + torch.arange(n) for L, n in zip(lens, news)] + [torch.zeros(pad, dtype=torch.int64)])
    pos = (row * 997 + 1_000_003 * (row % 2)) if given else row  # far positions
    spec = cs.RopeSpec(rotary, interleaved=inter, scaling="yarn", factor=4.0, original_length=2048)
    cache = cs.PagedCache(c.spec, k=c.k_pages.cuda(), v=c.v_pages.cuda(),
                          weight=torch.full((c.n_pages, Hk, page), 7.0, device="cuda"),
                          position=torch.full((c.n_pages, Hk, page), -5, dtype=torch.int32, device="cuda"))
    q_out = torch.full_like(q, 3.0).cuda()
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    cs.attn_paged_append(c.spec, c.batch(), cache, cu(q), cu(k), cu(v), cu(e), cu(gate), q_out,
                         positions=pos.to(torch.int32).cuda() if given else None, rope=spec)
    cs.cswattn_sync_status()
    n = c.start[-1]
    args = (pos[:n], spec.frequencies, spec.attention_factor, inter)
    big = 2.0 ** -19 * 12 * spec.attention_factor  # a normalised element is at most sqrt(128)

    def check(got, want, what):
        within(got, want, 2.0 ** -8 * want.abs() + big, what)
    check(q_out[:n], ref.rope(q[:n], *args), "q_out")
    assert (q_out[n:] == 3.0).all()  # tokens of nobody
    kw, vw = c.k_pages.double().clone(), c.v_pages.double().clone()
    ww, pw = torch.full((c.n_pages, Hk, page), 7.0), torch.full((c.n_pages, Hk, page), -5)
    kn = ref.rope(k[:n], *args)
    vn = v[:n].double() + (3 * torch.sigmoid(gate[:n].double())[..., None] * e[:n].double() if ve else 0)
    touched = torch.zeros(c.n_pages, page, dtype=torch.bool)
    for b in range(c.B):
        for i in range(news[b]):
            t, (p, o) = c.start[b] + i, c.place(b, lens[b] + i)
            kw[p, o], vw[p, o], ww[p, :, o], pw[p, :, o], touched[p, o] = kn[t], vn[t], 0.0, int(pos[t]), True
    check(cache.k[touched.cuda()], kw[touched], "k")
    check(cache.v[touched.cuda()], vw[touched], "v")
    for got, was in ((cache.k, c.k_pages), (cache.v, c.v_pages)):  # every other row bit for bit
        assert torch.equal(got.cpu()[~touched].view(torch.int16), was[~touched].view(torch.int16))
    assert torch.equal(cache.weight.cpu(), ww) and torch.equal(cache.position.cpu(), pw.to(torch.int32))


def test_append_matches_the_dense_prologue():
    """With the layer's plain RoPE the rows are attn_prologue's (angles there are float32 products: near
    positions agree to a bf16 step)."""
    B, T, H, Hk, D = 2, 70, 6, 2, 128
    c = Case([0] * B, [T] * B, H, Hk, D, 16, ve=True, seed=3)
    x = [c.randn(B, T, h, D).to(BF).cuda() for h in (H, Hk, Hk, Hk)]
    gate = c.randn(B, T, Hk).to(BF).cuda()
    buf = cs.LayerBuffers(c.spec)
    cs.attn_prologue(c.spec, *x, gate, buf.q_out, buf.k_out, buf.v_out, buf.rstd_q, buf.rstd_k)
    cache = cs.PagedCache(c.spec, n_pages=c.n_pages, page_size=16)
    q_out = torch.empty(B * T, H, D, dtype=BF, device="cuda")
    cs.attn_paged_append(c.spec, c.batch(), cache, *(t.flatten(0, 1) for t in x), gate.flatten(0, 1), q_out)
    cs.cswattn_sync_status()
    rows = torch.arange(T)
    for b in range(B):
        p, o = c.table[b].long()[rows // 16].cuda(), (rows % 16).cuda()
        for got, want in ((q_out[b * T:(b + 1) * T], buf.q_out[b]), (cache.k[p, o], buf.k_out[b]), (cache.v[p, o], buf.v_out[b])):
            d = (got.double() - want.double()).abs()
            assert (d <= 2.0 ** -7 * want.double().abs() + 1e-4).all()


# ------------------------------------------------------------------ attend and weigh

ATTEND = [
    # lens, news, H, Hk, D, page, W (None: all), cap (None: as needed), pad
    ([0], [1], 1, 1, 128, 16, None, None, 0),
    ([0], [1], 2, 1, 64, 16, None, None, 3),
    ([15, 16, 17, 0], [1, 1, 1, 1], 6, 6, 128, 16, None, None, 0),
    ([63, 64, 65, 127], [1, 1, 0, 1], 12, 4, 128, 64, 64, None, 2),
    ([300, 5, 129], [1, 2, 3], 8, 2, 64, 48, 100, None, 0),
    ([1000], [1], 16, 1, 128, 32, 1, None, 0),
    ([2500], [1], 6, 2, 128, 128, None, 4000, 0),          # split over many blocks
    ([900, 0, 33, 500], [5, 16, 1, 0], 16, 1, 128, 256, None, None, 0),
    ([70, 3], [21, 16], 3, 1, 64, 16, 17, None, 5),
    ([0], [128], 2, 2, 128, 16, None, None, 0),
    ([0, 100], [200, 131], 4, 2, 128, 64, None, None, 1),
    ([64, 0, 127], [129, 300, 1], 6, 2, 64, 48, 77, None, 0),
    ([333, 1], [150, 260], 5, 1, 128, 16, 130, None, 0),   # 5 heads: 25 tokens a tile
    ([10], [90], 128, 1, 64, 16, None, None, 0),           # one token a tile
    ([40], [3], 33, 1, 128, 32, None, None, 0),
    ([1111, 0], [257, 64], 8, 8, 64, 96, None, None, 0),
    ([50] * 70, [1, 2, 0, 3, 1] * 14, 4, 2, 64, 16, None, None, 0),
    ([3000], [260], 8, 2, 128, 128, None, None, 0),        # few tiles over a long cache
]
IDS = [f"{len(a[0])}seq-{max(a[0])}+{max(a[1])}-H{a[2]}.{a[3]}-D{a[4]}-p{a[5]}-W{a[6]}" for a in ATTEND]


def run_attend(c, q, k=None, v=None, ws_fill=0xFF):
    cache = cs.PagedCache(c.spec, k=c.k_pages.cuda() if k is None else k, v=c.v_pages.cuda() if v is None else v)
    batch = c.batch()
    O = torch.full((c.N, c.H, c.D), 5.0, dtype=BF, device="cuda")
    lse = torch.full((c.N, c.H), 5.0, device="cuda")
    ws = torch.full((cs.attn_paged_workspace_bytes(c.spec, batch, cache),), ws_fill, dtype=torch.uint8, device="cuda")
    cs.attn_paged(c.spec, batch, cache, q.cuda(), O, lse, ws)
    return O, lse


@pytest.mark.parametrize("lens,news,H,Hk,D,page,W,cap,pad", ATTEND, ids=IDS)
def test_attend(lens, news, H, Hk, D, page, W, cap, pad):
    c = Case(lens, news, H, Hk, D, page, W=W, cap=cap, pad=pad, seed=sum(lens) + H).fill()
    q = c.queries()
    O, lse = run_attend(c, q)
    cs.cswattn_sync_status()
    wO, wl, tO, tl = ref.attention(c, q)
    within(O, wO, tO, "O")
    within(lse, wl, tl, "lse")
    n = c.start[-1]
    assert (O[n:] == 5.0).all() and (lse[n:] == 5.0).all()
    O2, lse2 = run_attend(c, q, ws_fill=0x3C)  # what the workspace holds does not matter; the bits repeat
    assert torch.equal(O, O2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("lens,news,H,Hk,D,page,W,cap,pad", ATTEND, ids=IDS)
def test_weigh(lens, news, H, Hk, D, page, W, cap, pad):
    c = Case(lens, news, H, Hk, D, page, W=W, cap=cap, pad=pad, seed=sum(lens) + 2 * H).fill()
    q = c.queries()
    _, lse, _, _ = ref.attention(c, q)
    lse = lse.float()  # NaN at the tokens of nobody
    w0 = c.randn(c.n_pages, Hk, page).abs()
    cache = cs.PagedCache(c.spec, k=c.k_pages.cuda(), weight=w0.cuda())
    cs.attn_paged_weigh(c.spec, c.batch(), cache, q.cuda(), lse.cuda())
    cs.cswattn_sync_status()
    want, tol = ref.weights(c, q, lse, w0)
    within(cache.weight, want, tol, "weight")
    seen = want != w0.double()
    assert torch.equal(cache.weight.cpu()[~seen], w0[~seen])  # rows that nobody sees, bit for bit
    again = cs.PagedCache(c.spec, k=c.k_pages.cuda(), weight=w0.cuda())
    cs.attn_paged_weigh(c.spec, c.batch(), again, q.cuda(), lse.cuda())
    assert torch.equal(again.weight, cache.weight)


@pytest.mark.parametrize("lens,news,H,Hk,D", [
    ([12000], [40], 4, 1, 128),    # a unit of 160 rows over 94 blocks: 47 shares
    ([9000, 0], [9, 3], 8, 1, 64),
    ([5000], [30], 8, 4, 128),     # 20 shares a head
    ([12000], [2], 12, 4, 128),    # few rows: pairs cut in 37
    ([16000], [1], 6, 1, 64),      # ... one in 125
    ([0], [100], 128, 1, 64),      # one tile of cached rows under 100 tiles of query rows
    ([28], [100], 128, 1, 128),
])
def test_work_cut_in_many_shares(lens, news, H, Hk, D):
    test_attend(lens, news, H, Hk, D, 64, None, None, 1)
    test_weigh(lens, news, H, Hk, D, 64, None, None, 1)


@pytest.mark.parametrize("news", [[1, 1], [40, 1], [1, 300]])
def test_other_scale_and_large_scores(news):
    """Scores up to hundreds: only the largest key counts, nothing overflows."""
    c = Case([200, 77], news, 4, 2, 128, 32, seed=5, scale=3.0).fill()
    q = c.queries()
    O, lse = run_attend(c, q)
    cs.cswattn_sync_status()
    wO, wl, tO, tl = ref.attention(c, q)
    within(O, wO, tO, "O")
    within(lse, wl, tl, "lse")


@pytest.mark.parametrize("news", [[1, 1, 1], [3, 64, 1], [1, 200, 0]])
def test_attend_matches_the_dense_decode_and_forward(news):
    """One sequence's chunk equals the dense forward of the whole sequence at those rows, to bf16 rounding."""
    lens, H, Hk, D, W = [37, 130, 300], 6, 2, 128, 120
    c = Case(lens, news, H, Hk, D, 16, W=W, seed=11).fill()
    q = c.queries()
    O, lse = run_attend(c, q)
    for b in range(c.B):
        n, T = news[b], lens[b] + news[b]
        if n == 0:
            continue
        spec = cs.LayerSpec(1, T, H, Hk, D, W, has_ve=False)
        full = torch.zeros(1, T, H, D, dtype=BF, device="cuda")
        full[0, lens[b]:] = q[c.start[b]: c.start[b] + n].cuda()
        k, v = (c.rows_of(b, p)[None].contiguous().cuda() for p in (c.k_pages, c.v_pages))
        O1, lse1 = torch.empty_like(full), torch.empty(1, H, T, device="cuda")
        cs.attn_fwd(spec, full, k, v, O1, lse1)
        cs.cswattn_sync_status()
        d = (O[c.start[b]: c.start[b] + n].double() - O1[0, lens[b]:].double()).abs()
        assert (d <= 0.03).all()
        assert (lse[c.start[b]: c.start[b] + n] - lse1[0, :, lens[b]:].T).abs().max() <= 1e-3


def test_pages_before_the_window_are_not_read():
    """Table entries of rows that no token sees may be anything."""
    c = Case([1000, 200], [1, 30], 4, 2, 128, 16, W=40, seed=6).fill()
    q = c.queries()
    want = run_attend(c, q)
    for b in range(c.B):
        c.table[b, : (c.lens[b] - c.W + 1) // 16] = -7
        c.table[b, -(-(c.lens[b] + c.news[b]) // 16):] = 1 << 30
    got = run_attend(c, q)
    cs.cswattn_sync_status()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    w = torch.zeros(c.n_pages, c.Hk, c.page, device="cuda")
    cs.attn_paged_weigh(c.spec, c.batch(), cs.PagedCache(c.spec, k=c.k_pages.cuda(), weight=w), q.cuda(), got[1])
    cs.cswattn_sync_status()
    assert torch.isfinite(w).all()
    # every token's weights sum to 1 for each head
    assert abs(w.double().sum().item() - c.H * sum(c.news)) <= 1e-4 * c.H * sum(c.news)


def test_many_sequences():
    """More sequences than threads of a CTA, most of them without a row or a token."""
    r = np.random.RandomState(4)
    B = 1500
    news = [int(x) for x in r.choice([0, 0, 0, 1, 1, 2, 40], B)]
    lens = [int(x) for x in r.choice([0, 1, 15, 16, 30], B)]
    c = Case(lens, news, 4, 2, 64, 16, seed=41, pad=2).fill()
    q = c.queries()
    O, lse = run_attend(c, q)
    cs.cswattn_sync_status()
    wO, wl, tO, tl = ref.attention(c, q)
    within(O, wO, tO, "O")
    within(lse, wl, tl, "lse")
    w0 = c.randn(c.n_pages, 2, 16).abs()
    cache = cs.PagedCache(c.spec, k=c.k_pages.cuda(), weight=w0.cuda())
    cs.attn_paged_weigh(c.spec, c.batch(), cache, q.cuda(), wl.float().cuda())
    cs.cswattn_sync_status()
    want, tol = ref.weights(c, q, wl.float(), w0)
    within(cache.weight, want, tol, "weight")


def test_the_largest_number_of_sequences():
    """4096 sequences of one row and one token: each attends to its two rows."""
    B, H, Hk, D = 4096, 2, 1, 64
    c = Case([1] * B, [1] * B, H, Hk, D, 16, seed=42, spare=0)
    k, v = torch.randn(B, 16, Hk, D, generator=c.g).to(BF), torch.randn(B, 16, Hk, D, generator=c.g).to(BF)
    k[:, 2:], v[:, 2:] = NAN, NAN
    c.k_pages[c.table[:, 0].long()], c.v_pages[c.table[:, 0].long()] = k, v
    q = c.queries()
    O, lse = run_attend(c, q)
    cs.cswattn_sync_status()
    s = torch.einsum("bhd,bjd->bhj", q.double(), k[:, :2, 0].double()) * D ** -0.5
    want = torch.softmax(s, -1) @ v[:, :2, 0].double()
    mag = torch.softmax(s, -1) @ v[:, :2, 0].double().abs()
    within(O, want, 2.0 ** -8 * (mag + want.abs()) + 1e-3 * mag, "O")
    within(lse, torch.logsumexp(s, -1), torch.full((B, H), 1e-4, dtype=torch.float64), "lse")


def test_a_stream_by_handle_and_a_workspace_of_the_callers():
    c = Case([300, 20], [70, 1], 4, 2, 128, 32, seed=43).fill()
    q = c.queries().cuda()
    lse = ref.attention(c, q.cpu())[1].float().cuda()
    batch, got = c.batch(), []
    side = torch.cuda.Stream()
    for kind in ("own", "default", "handle", "stream"):
        cache = cs.PagedCache(c.spec, k=c.k_pages.cuda(), weight=torch.zeros(c.n_pages, 2, 32, device="cuda"))
        torch.cuda.synchronize()
        if kind == "own":
            ws = torch.empty(cs.attn_paged_weigh_workspace_bytes(c.spec, batch, cache), dtype=torch.uint8, device="cuda")
            cs.attn_paged_weigh(c.spec, batch, cache, q, lse, workspace=ws)
        elif kind == "default":
            cs.attn_paged_weigh(c.spec, batch, cache, q, lse)
        else:
            cs.attn_paged_weigh(c.spec, batch, cache, q, lse, stream=side.cuda_stream if kind == "handle" else side)
        torch.cuda.synchronize()
        got.append(cache.weight)
    assert got[0].sum() > 0 and all(torch.equal(got[0], w) for w in got[1:])


def test_tensors_that_do_not_fit_are_refused():
    """Types, shapes, strides, hosts and missing pools: before anything is enqueued."""
    c = Case([30, 20], [3, 1], 4, 2, 128, 16, seed=44).fill()
    q, batch = c.queries().cuda(), c.batch()
    cache = cs.PagedCache(c.spec, k=c.k_pages.cuda(), v=c.v_pages.cuda())
    O, lse = torch.zeros_like(q), torch.zeros(c.N, 4, device="cuda")
    ws = torch.empty(cs.attn_paged_workspace_bytes(c.spec, batch, cache), dtype=torch.uint8, device="cuda")
    wide = torch.zeros(c.N, 4, 256, dtype=BF, device="cuda")[..., ::2]
    for change in (dict(q_out=q.float()), dict(q_out=q[:2]), dict(q_out=wide), dict(q_out=q.cpu()), dict(O=None),
                   dict(lse=lse.double()), dict(lse=lse[:, :3]), dict(workspace=ws.cpu()), dict(workspace=ws[::2])):
        args = {**dict(q_out=q, O=O, lse=lse, workspace=ws), **change}
        with pytest.raises(ValueError):
            cs.attn_paged(c.spec, batch, cache, **args)
    with pytest.raises(TypeError):
        cs.attn_paged(c.spec, batch, cache, q.tolist(), O, lse, ws)
    with pytest.raises(cs.CswattnError) as err:  # less than the call needs, said by the caller or by the tensor
        cs.attn_paged(c.spec, batch, cache, q, O, lse, ws, workspace_bytes=ws.numel() - 1)
    assert err.value.status == cs.ERR_INVALID_ARG
    with pytest.raises(cs.CswattnError):
        cs.attn_paged(c.spec, batch, cache, q, O, lse, ws[:256], workspace_bytes=1 << 40)
    with pytest.raises(ValueError, match="weight"):  # no pool to add to
        cs.attn_paged_weigh(c.spec, batch, cache, q, lse)
    other = cs.LayerSpec(2, c.cap, 4, 4, 128, c.cap, has_ve=False)
    with pytest.raises(ValueError):  # a cache of another layer
        cs.attn_paged(other, batch, cache, q, O, lse, ws)
    with pytest.raises(ValueError, match="sequences"):
        cs.attn_paged(cs.LayerSpec(3, c.cap, 4, 2, 128, c.cap, has_ve=False), batch, cache, q, O, lse, ws)
    i64 = lambda t: t.to(torch.int64)  # noqa: E731
    for a in ((i64(batch.page_table), batch.cache_len, batch.new_start), (batch.page_table, i64(batch.cache_len), None),
              (batch.page_table, batch.cache_len[:1], None), (batch.page_table, batch.cache_len, batch.cache_len),
              (batch.page_table.cpu(), batch.cache_len, None), (batch.page_table.T, batch.cache_len, None)):
        with pytest.raises(ValueError):
            cs.PagedBatch(*a)
    with pytest.raises(ValueError):
        cs.PagedCache(c.spec, k=c.k_pages.cuda(), v=c.v_pages[:-1].cuda())
    with pytest.raises(ValueError):
        cs.attn_paged_append(c.spec, cs.PagedBatch(batch.page_table, batch.cache_len, None, c.N, 3), cache, q, q, q, None, None, O)
    assert (O == 0).all() and (lse == 0).all()
    cs.cswattn_sync_status()


# ------------------------------------------------------------------ select and move

SELECT = [
    # lens, Hk, D, page, n_keep, n_recent, cap, ties
    ([1], 1, 128, 16, 1, 0, None, False),
    ([2], 2, 64, 16, 1, 1, None, False),
    ([5, 0, 40, 41], 2, 128, 16, 40, 7, None, True),
    ([100, 33], 3, 64, 48, 32, 32, None, True),
    ([1025] * 3, 4, 128, 64, 1024, 100, None, True),
    ([2049, 3000, 17], 1, 64, 128, 2048, 0, None, False),
    ([700], 2, 64, 16, 3, 2, None, True),
    ([5000, 4999], 2, 128, 256, 1300, 500, 6000, True),
    ([33000], 1, 64, 128, 20000, 5, None, True),
    ([60001], 1, 64, 128, 700, 20, None, True),
]


def evict_case(lens, Hk, D, page, cap, ties, seed):
    c = Case(lens, [0] * len(lens), Hk, Hk, D, page, cap=cap, seed=seed)
    w = torch.exp(2 * c.randn(c.n_pages, Hk, page))
    if ties:
        w = torch.round(w)  # many zeros
    pos = torch.randint(0, 2 * max(lens) + 1, (c.n_pages, Hk, page), generator=c.g, dtype=torch.int32)
    return c, w, pos


def run_select(c, w, pos, next_pos, n_keep, n_recent):
    cache = cs.PagedCache(c.spec, weight=w.cuda(), position=pos.cuda())
    i32 = dict(dtype=torch.int32, device="cuda")
    n, new_len = torch.full((c.B, c.Hk), 99, **i32), torch.full((c.B,), 99, **i32)
    src, dst = torch.full((c.B, c.Hk, n_keep), 99, **i32), torch.full((c.B, c.Hk, n_keep), 99, **i32)
    cs.attn_paged_select(c.spec, c.batch(), cache, next_pos.to(torch.int32).cuda(), n_keep, n_recent, n, src, dst, new_len)
    return n, src, dst, new_len


def head_rows(c, b, h, pool):
    rows = torch.arange(c.lens[b])
    return pool[c.table[b].long()[rows // c.page], h, rows % c.page]


def check_select(c, w, pos, next_pos, n_keep, n_recent, got):
    n, src, dst, new_len = (t.cpu() for t in got)
    for b in range(c.B):
        assert int(new_len[b]) == min(c.lens[b], n_keep)
        for h in range(c.Hk):
            s, d = ref.select(head_rows(c, b, h, w).tolist(), head_rows(c, b, h, pos).tolist(), int(next_pos[b]),
                              c.lens[b], n_keep, n_recent)
            m = len(s)
            assert int(n[b, h]) == m
            assert src[b, h].tolist() == s + [-1] * (n_keep - m)
            assert dst[b, h].tolist() == d + [-1] * (n_keep - m)


@pytest.mark.parametrize("lens,Hk,D,page,n_keep,n_recent,cap,ties", SELECT)
def test_select(lens, Hk, D, page, n_keep, n_recent, cap, ties):
    c, w, pos = evict_case(lens, Hk, D, page, cap, ties, seed=n_keep)
    next_pos = torch.tensor([2 * L for L in lens])
    got = run_select(c, w, pos, next_pos, n_keep, n_recent)
    cs.cswattn_sync_status()
    check_select(c, w, pos, next_pos, n_keep, n_recent, got)


def test_select_beyond_shared_memory():
    """A head of more rows than its CTA holds in shared memory (so many heads that none has a second CTA): the rows
    past them are read again in every pass."""
    B, L, K = 75, 60000, 20000
    c = Case([L] + [3] * (B - 1), [0] * B, 1, 1, 64, 128, cap=L, seed=50)
    w = torch.round(torch.exp(2 * c.randn(c.n_pages, 1, 128)))
    pos = torch.randint(0, 2 * L, (c.n_pages, 1, 128), generator=c.g, dtype=torch.int32)
    next_pos = torch.tensor([2 * L] + [6] * (B - 1))
    n, src, dst, new_len = (t.cpu() for t in run_select(c, w, pos, next_pos, K, 900))
    cs.cswattn_sync_status()
    wt, ps = head_rows(c, 0, 0, w).double().numpy(), head_rows(c, 0, 0, pos).numpy()
    key = np.where(ps >= 2 * L - 900, np.inf, wt)
    kept = np.zeros(L, bool)
    kept[np.argsort(-key, kind="stable")[:K]] = True
    rows = np.arange(L)
    s, d = rows[kept & (rows >= K)], rows[~kept & (rows < K)]
    m = int(n[0, 0])
    assert m == len(s) == len(d) and int(new_len[0]) == K
    assert (src[0, 0, :m].numpy() == s).all() and (dst[0, 0, :m].numpy() == d).all() and (src[0, 0, m:] == -1).all()
    assert (n[1:] == 0).all() and (new_len[1:] == 3).all() and (src[1:] == -1).all() and (dst[1:] == -1).all()


@pytest.mark.parametrize("kind", ["equal", "nan", "infinite", "signed", "all recent", "denormal"])
def test_select_values(kind):
    """Every order of values the definition names: equal ones by row, a NaN after all numbers, both zeros equal."""
    c, w, pos = evict_case([900, 512, 511], 2, 64, 32, None, False, seed=21)
    next_pos, n_recent = torch.tensor([1800, 1024, 1022]), 30
    if kind == "equal":
        w[:] = 0.25
    elif kind == "nan":
        w[c.randn(*w.shape) > 0.3] = NAN
    elif kind == "infinite":
        w[c.randn(*w.shape) > 0.8] = float("inf")
        w[c.randn(*w.shape) > 0.8] = float("-inf")
    elif kind == "signed":
        w = torch.round(c.randn(*w.shape)) * 0.5
        w[w == 0] = torch.where(c.randn(int((w == 0).sum())) > 0, 0.0, -0.0)
    elif kind == "all recent":
        next_pos, n_recent = torch.tensor([-(2 ** 31)] * 3), 512
    else:
        w = w * 2.0 ** -149 * 4
    got = run_select(c, w, pos, next_pos, 512, n_recent)
    cs.cswattn_sync_status()
    check_select(c, w, pos, next_pos, 512, n_recent, got)


@pytest.mark.parametrize("lens,Hk,D,page,n_keep,n_recent,cap,ties", SELECT[1:8])
def test_move(lens, Hk, D, page, n_keep, n_recent, cap, ties):
    c, w, pos = evict_case(lens, Hk, D, page, cap, ties, seed=n_keep + 1)
    c.fill()
    got = run_select(c, w, pos, torch.tensor([2 * L for L in lens]), n_keep, n_recent)
    cache = cs.PagedCache(c.spec, k=c.k_pages.cuda(), v=c.v_pages.cuda(), weight=w.cuda(), position=pos.cuda())
    kw, vw, ww, pw = c.k_pages.clone(), c.v_pages.clone(), w.clone(), pos.clone()
    for b in range(c.B):
        for h in range(Hk):
            for s, d in zip(got[1][b, h].tolist(), got[2][b, h].tolist()):
                if s >= 0:
                    (p, o), (z, y) = c.place(b, s), c.place(b, d)
                    kw[z, y, h], vw[z, y, h] = c.k_pages[p, o, h], c.v_pages[p, o, h]
                    ww[z, h, y], pw[z, h, y] = w[p, h, o], pos[p, h, o]
    for _ in range(2):  # a second run changes nothing
        cs.attn_paged_move(c.spec, c.batch(), cache, *got[:3])
        cs.cswattn_sync_status()
        for g, want in ((cache.k, kw), (cache.v, vw)):
            assert torch.equal(g.cpu().view(torch.int16), want.view(torch.int16))
        assert torch.equal(cache.weight.cpu(), ww) and torch.equal(cache.position.cpu(), pw)


# ------------------------------------------------------------------ what does not fit

def expect_range_error():
    with pytest.raises(cs.CswattnError) as err:
        cs.cswattn_sync_status()
    assert err.value.status == cs.ERR_INVALID_ARG
    cs.cswattn_sync_status()  # cleared


@pytest.mark.parametrize("bad", ["negative", "past T", "too many", "decreasing", "past n_tokens"])
@pytest.mark.parametrize("news", [[2, 3, 1], [2, 150, 90]])
def test_lengths_that_do_not_fit_leave_the_sequence_alone(bad, news):
    c = Case([20, 60, 33], news, 4, 2, 64, 16, seed=8, max_new=max(news)).fill()
    q = c.queries()
    good = run_attend(c, q)
    cs.cswattn_sync_status()
    batch = c.batch()
    hit = [1]
    if bad == "negative":
        batch.cache_len[1] = -3
    elif bad == "past T":
        batch.cache_len[1] = c.cap - c.news[1] + 1
    elif bad == "too many":
        batch.max_new = 1
        hit = [b for b in range(3) if c.news[b] > 1]
    elif bad == "decreasing":
        batch.new_start[2] = c.start[1] - 1
        hit = [1, 2]  # sequence 2 has a token more than its own
        batch.cache_len[2] = c.cap
    else:
        batch.new_start[3] = c.N + 1
        hit = [2]
    cache = cs.PagedCache(c.spec, k=c.k_pages.cuda(), v=c.v_pages.cuda(),
                          weight=torch.zeros(c.n_pages, c.Hk, 16, device="cuda"),
                          position=torch.zeros(c.n_pages, c.Hk, 16, dtype=torch.int32, device="cuda"))
    O = torch.full((c.N, c.H, c.D), 5.0, dtype=BF, device="cuda")
    lse = torch.full((c.N, c.H), 5.0, device="cuda")
    ws = torch.empty(cs.attn_paged_workspace_bytes(c.spec, batch, cache), dtype=torch.uint8, device="cuda")
    cs.attn_paged(c.spec, batch, cache, q.cuda(), O, lse, ws)
    expect_range_error()
    cs.attn_paged_weigh(c.spec, batch, cache, q.cuda(), good[1])
    expect_range_error()
    for b in range(3):
        t = slice(c.start[b], c.start[b] + c.news[b])
        if b in hit:
            assert (O[t] == 5.0).all() and (lse[t] == 5.0).all()
        else:  # the others as they are without it (another split of the work may round otherwise)
            assert (O[t].double() - good[0][t].double()).abs().max() <= 0.03
        pages = c.table[b].long().cuda()
        total = cache.weight[pages].double().sum().item()
        assert total == 0.0 if b in hit else abs(total - c.H * c.news[b]) <= 1e-3 * c.H * c.news[b]
    x = torch.zeros(c.N, c.Hk, c.D, dtype=BF, device="cuda")
    q_out = torch.full((c.N, c.H, c.D), 5.0, dtype=BF, device="cuda")
    k0 = cache.k.clone()
    cs.attn_paged_append(c.spec, batch, cache, q.cuda(), x, x, None, None, q_out)
    expect_range_error()
    for b in hit:
        t = slice(c.start[b], c.start[b] + c.news[b])
        assert (q_out[t] == 5.0).all()
        pages = c.table[b].long().cuda()
        assert torch.equal(cache.k[pages].view(torch.int16), k0[pages].view(torch.int16))


@pytest.mark.parametrize("entry", [-1, 1 << 30])
def test_pages_outside_the_pool_are_reported(entry):
    for news in ([1, 1], [100, 90]):
        c = Case([100, 50], news, 4, 2, 128, 16, seed=9).fill()
        c.table[0, 3] = entry
        q = c.queries()
        O, lse = run_attend(c, q)
        expect_range_error()
        assert torch.isfinite(O[c.start[1]:].float()).all() and torch.isfinite(O[: c.start[1]].float()).all()
        w = torch.zeros(c.n_pages, 2, 16, device="cuda")
        cs.attn_paged_weigh(c.spec, c.batch(), cs.PagedCache(c.spec, k=c.k_pages.cuda(), weight=w), q.cuda(), lse)
        expect_range_error()
        assert torch.isfinite(w).all()
    c, w, pos = evict_case([100, 50], 2, 64, 16, None, False, seed=1)
    c.table[0, 3] = entry
    n, src, dst, _ = run_select(c, w, pos, torch.tensor([200, 100]), 30, 3)
    expect_range_error()
    k = torch.zeros(c.n_pages, 16, 2, 64, dtype=BF, device="cuda")
    cache = cs.PagedCache(c.spec, k=k, v=k.clone(), weight=w.cuda(), position=pos.cuda())
    src[0, 0, 0], dst[0, 0, 0] = 50, 2  # row 50 lies in the page that is none
    n[0, 0] = 1
    cs.attn_paged_move(c.spec, c.batch(), cache, n, src, dst)
    expect_range_error()
    n[0, 0] = 31  # more moves than entries
    cs.attn_paged_move(c.spec, c.batch(), cache, n, src, dst)
    expect_range_error()
    n[0, 0], src[0, 0, 0] = 1, 100000
    cs.attn_paged_move(c.spec, c.batch(), cache, n, src, dst)
    expect_range_error()


def test_select_length_that_does_not_fit():
    c, w, pos = evict_case([100, 50], 2, 64, 16, None, False, seed=2)
    batch = c.batch()
    batch.cache_len[0] = 101
    cache = cs.PagedCache(c.spec, weight=w.cuda(), position=pos.cuda())
    i32 = dict(dtype=torch.int32, device="cuda")
    n, new_len = torch.full((2, 2), 99, **i32), torch.full((2,), 99, **i32)
    src, dst = torch.full((2, 2, 30), 99, **i32), torch.full((2, 2, 30), 99, **i32)
    cs.attn_paged_select(c.spec, batch, cache, torch.tensor([200, 100], **i32), 30, 3, n, src, dst, new_len)
    expect_range_error()
    assert (n[0] == 99).all() and (src[0] == 99).all() and int(new_len[0]) == 99
    assert int(new_len[1]) == 30 and (n[1] != 99).all()


@pytest.mark.parametrize("length", [-1, 101])
def test_moves_of_a_length_that_does_not_fit(length):
    # What select has left as it was may hold moves of an earlier call: they are not made.
    c, w, pos = evict_case([100, 50], 2, 64, 16, None, False, seed=3)
    batch = c.batch()
    batch.cache_len[0] = length
    g = torch.Generator().manual_seed(4)
    k = torch.randn(c.n_pages, 16, 2, 64, generator=g).to(BF).cuda()
    cache = cs.PagedCache(c.spec, k=k, v=k.clone(), weight=w.cuda(), position=pos.cuda())
    i32 = dict(dtype=torch.int32, device="cuda")
    n, new_len = torch.full((2, 2), 1, **i32), torch.full((2,), 99, **i32)
    src, dst = torch.full((2, 2, 30), 40, **i32), torch.full((2, 2, 30), 7, **i32)
    cs.attn_paged_select(c.spec, batch, cache, torch.tensor([200, 100], **i32), 30, 3, n, src, dst, new_len)
    expect_range_error()
    k0, w0, p0 = k.clone(), cache.weight.clone(), cache.position.clone()
    cs.attn_paged_move(c.spec, batch, cache, n, src, dst)
    expect_range_error()
    mine = c.table[0].long().cuda()
    for now, then in ((cache.k, k0), (cache.v, k0), (cache.weight, w0), (cache.position, p0)):
        assert torch.equal(now[mine], then[mine])
    assert (n[1] > 0).all() and not torch.equal(cache.k, k0)  # the other sequence's rows did move


# ------------------------------------------------------------------ together

class Server:
    """A serving loop over one layer, in the cache's own terms: what a user writes."""

    def __init__(self, lens_max, H, Hk, D, page, B, W=None, budget=None, recent=0, split_rope=None):
        g = torch.Generator().manual_seed(77)
        self.g, self.H, self.Hk, self.D, self.page, self.B = g, H, Hk, D, page, B
        self.pps = -(-lens_max // page)
        self.spec = cs.LayerSpec(B, lens_max, H, Hk, D, W or lens_max, has_ve=True)
        self.cache = cs.PagedCache(self.spec, n_pages=B * self.pps + 2, page_size=page, track_weights=True)
        self.cache.k.fill_(NAN), self.cache.v.fill_(NAN)
        self.table = torch.randperm(B * self.pps + 2, generator=g)[: B * self.pps].view(B, self.pps).to(torch.int32).cuda()
        self.len = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.pos = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.budget, self.recent, self.rope = budget, recent, split_rope
        # the model of it in 64 bits: per sequence the (position, k, v, weight) of every head's rows
        self.rows = [[[] for _ in range(Hk)] for _ in range(B)]

    def inputs(self, news):
        N, r = sum(news), lambda *s: torch.randn(*s, generator=self.g).to(BF)
        return [r(N, h, self.D) for h in (self.H, self.Hk, self.Hk, self.Hk)] + [r(N, self.Hk)]

    def call(self, news, x):
        i32 = dict(dtype=torch.int32, device="cuda")
        start = torch.tensor([0] + np.cumsum(news).tolist(), **i32)
        N = sum(news)
        batch = cs.PagedBatch(self.table, self.len, start, N, max(1, max(news)))
        positions = torch.cat([p + torch.arange(n, **i32) for p, n in zip(self.pos, news)]) if N else None
        q_out = torch.empty(N, self.H, self.D, dtype=BF, device="cuda")
        O, lse = torch.empty_like(q_out), torch.empty(N, self.H, device="cuda")
        ws = torch.empty(cs.attn_paged_workspace_bytes(self.spec, batch, self.cache), dtype=torch.uint8, device="cuda")
        cs.attn_paged_append(self.spec, batch, self.cache, *(t.cuda() for t in x), q_out, positions=positions, rope=self.rope)
        cs.attn_paged(self.spec, batch, self.cache, q_out, O, lse, ws)
        cs.attn_paged_weigh(self.spec, batch, self.cache, q_out, lse)
        self.len += torch.tensor(news, **i32)
        self.pos += torch.tensor(news, **i32)
        if self.budget:
            n, new = torch.empty(self.B, self.Hk, **i32), torch.empty(self.B, **i32)
            src, dst = torch.empty(self.B, self.Hk, self.budget, **i32), torch.empty(self.B, self.Hk, self.budget, **i32)
            after = cs.PagedBatch(self.table, self.len)
            cs.attn_paged_select(self.spec, after, self.cache, self.pos, self.budget, self.recent, n, src, dst, new)
            cs.attn_paged_move(self.spec, after, self.cache, n, src, dst)
            self.len = new
        cs.cswattn_sync_status()
        return O, lse


def test_serving_loop_without_eviction_is_the_dense_layer():
    """Prompts in chunks, then single tokens, two sequences out of step: the outputs are the dense layer's."""
    H, Hk, D, T, W = 6, 2, 128, 200, 90
    s = Server(T, H, Hk, D, 16, 2, W=W)
    steps = [(130, 7), (20, 60), (1, 1), (1, 0), (0, 33), (1, 1), (30, 1)]
    xs, outs = [], []
    for news in steps:
        x = s.inputs(news)
        xs.append(x)
        outs.append(s.call(list(news), x)[0].cpu())
    for b in range(2):
        n = sum(t[b] for t in steps)
        cut = lambda ts: torch.cat([t[(0, st[0])[b]: st[0] + st[1] if b else st[0]] for t, st in zip(ts, steps)])[None]  # noqa: E731
        q, k, v, e, gate = (cut([x[i] for x in xs]).contiguous().cuda() for i in range(5))
        spec = cs.LayerSpec(1, n, H, Hk, D, W)
        buf = cs.LayerBuffers(spec)
        cs.layer_forward(spec, buf, q, k, v, e, gate)
        cs.cswattn_sync_status()
        d = (cut(outs).double() - buf.O.cpu().double()).abs()
        assert d.max() <= 0.05  # two roundings of P, k~, q~ each way apart, outputs of size 1


@pytest.mark.parametrize("rope", [None, cs.RopeSpec(64, interleaved=True, scaling="yarn", factor=4.0, original_length=64)])
def test_serving_loop_with_eviction(rope):
    """A budget of rows: the cache's own weights, positions and rows decide; at every step the attention over
    what is left is right, and each sequence keeps the newest rows."""
    H, Hk, D, B = 4, 2, 64, 3
    s = Server(150, H, Hk, D, 16, B, budget=50, recent=12, split_rope=rope)
    for news in ([60, 3, 0], [1, 1, 90], [1, 1, 1], [40, 60, 1], [1, 0, 1], [1, 1, 1]):
        before, lens = [s.cache.k.cpu(), s.cache.v.cpu(), s.cache.position.cpu()], s.len.tolist()
        O, lse = s.call(news, s.inputs(news))
        assert torch.isfinite(O.float()).all()
        assert s.len.tolist() == [min(50, L + n) for L, n in zip(lens, news)]
        for b in range(B):
            L, P = int(s.len[b]), int(s.pos[b])
            rows = torch.arange(L)
            p, o = s.table[b].long().cpu()[rows // 16], rows % 16
            pos = s.cache.position.cpu()[p, :, o]  # (L, Hk)
            for h in range(Hk):
                have = set(pos[:, h].tolist())
                assert len(have) == L and set(range(max(0, P - 12), P)) <= have
            if L:
                assert torch.isfinite(s.cache.k.cpu()[p, o].float()).all()
        # weights of the whole cache: what each token spread over the rows, less what left with the evicted
        assert torch.isfinite(s.cache.weight).all() and (s.cache.weight >= 0).all()


@pytest.mark.parametrize("B,T,H,Hk,W", [(1, 128, 2, 2, 128), (2, 300, 4, 2, 300)])
def test_dense_backward_after_scores_of_nan(B, T, H, Hk, W):
    """What a kernel leaves in tensor memory is nobody's input: the dense layer's gradients are as before after an
    attention over NaN rows (a backward part that has no step once multiplied what it found there by zero)."""
    from _helpers import make_inputs
    spec = cs.LayerSpec(B, T, H, Hk, 128, W, has_ve=True)
    dev = {n: t.cuda() for n, t in make_inputs(B, T, H, Hk, 128, True, "bf16", config=98).items()}
    c = Case([2000], [1500], 16, 4, 128, 128, seed=61)  # its pages are NaN; work for every SM
    q, outs = c.queries(), []
    for dirty in (False, True):
        if dirty:
            O, _ = run_attend(c, q)
            cs.cswattn_sync_status()
            assert torch.isnan(O.float()).all()
        buf = cs.LayerBuffers(spec)
        cs.layer_forward(spec, buf, dev["q"], dev["k"], dev["v"], dev["ve"], dev["gate"])
        cs.layer_backward(spec, buf, dev["q"], dev["k"], dev["ve"], dev["gate"], dev["dO"])
        cs.cswattn_sync_status()
        outs.append([t.float() for t in (buf.O, buf.lse, buf.dQ, buf.dK, buf.dV, buf.dve, buf.dgate)])
    for clean, after in zip(*outs):
        assert torch.isfinite(after).all()
        assert (clean - after).abs().max() <= 1e-2 * clean.abs().max()  # dQ adds its parts in any order


def test_a_captured_loop_replays():
    """Append, attend, weigh, select and move in one CUDA graph, replayed on new inputs; two graphs share a workspace."""
    c = Case([40, 90], [1, 1], 4, 2, 64, 16, cap=120, ve=False, seed=31).fill()
    batch = c.batch()
    cache = cs.PagedCache(c.spec, k=c.k_pages.cuda(), v=c.v_pages.cuda(),
                          weight=torch.zeros(c.n_pages, 2, 16, device="cuda"),
                          position=torch.zeros(c.n_pages, 2, 16, dtype=torch.int32, device="cuda"))
    q, k, v = (c.randn(2, h, 64).to(BF).cuda() for h in (4, 2, 2))
    ws = torch.empty(cs.attn_paged_workspace_bytes(c.spec, batch, cache), dtype=torch.uint8, device="cuda")

    def buffers():
        return [torch.empty(2, 4, 64, dtype=BF, device="cuda"), torch.empty(2, 4, 64, dtype=BF, device="cuda"),
                torch.empty(2, 4, device="cuda")]

    def step(q_out, O, lse):
        cs.attn_paged_append(c.spec, batch, cache, q, k, v, None, None, q_out)
        cs.attn_paged(c.spec, batch, cache, q_out, O, lse, ws)
        cs.attn_paged_weigh(c.spec, batch, cache, q_out, lse)
    warm = buffers()
    step(*warm)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        bufs, gr = buffers(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            step(*bufs)
        graphs.append((gr, bufs))
    for seed in range(3):
        q.copy_(torch.randn(2, 4, 64, generator=c.g).to(BF))
        k.copy_(torch.randn(2, 2, 64, generator=c.g).to(BF))
        step(*warm)
        want = [t.clone() for t in warm]
        w0 = cache.weight.clone()
        for gr, bufs in graphs:
            gr.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(bufs, want))
        assert (cache.weight >= w0 * 0).all()
    cs.cswattn_sync_status()


def test_on_another_stream():
    c = Case([400, 90], [1, 130], 4, 2, 128, 16, seed=32).fill()
    q = c.queries()
    want = run_attend(c, q)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = run_attend(c, q)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes and 2^31 elements: the last pages are as good as the first."""
    H, Hk, D, page = 4, 4, 128, 256
    n_pages = (1 << 31) // (page * Hk * D) + 64
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("not enough free memory")
    c = Case([700, 300], [1, 140], H, Hk, D, page, seed=33).fill()
    q = c.queries()
    want = run_attend(c, q)
    k = torch.empty(n_pages, page, Hk, D, dtype=BF, device="cuda")
    v = torch.empty_like(k)
    used = c.table.flatten().long()
    moved = n_pages - 1 - used
    k[moved.cuda()], v[moved.cuda()] = c.k_pages[used].cuda(), c.v_pages[used].cuda()
    c.table = moved.view_as(c.table).to(torch.int32)
    got = run_attend(c, q, k, v)
    cs.cswattn_sync_status()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    w = torch.zeros(n_pages, Hk, page, device="cuda")
    cache = cs.PagedCache(c.spec, k=k, v=v, weight=w, position=torch.zeros_like(w, dtype=torch.int32))
    cs.attn_paged_weigh(c.spec, c.batch(), cache, q.cuda(), got[1])
    cs.cswattn_sync_status()
    assert abs(w.double().sum().item() - c.H * 141) <= 1e-3 * c.H * 141
    x = c.randn(c.N, Hk, D).to(BF).cuda()
    q_out = torch.empty(c.N, H, D, dtype=BF, device="cuda")
    cs.attn_paged_append(c.spec, c.batch(), cache, q.cuda(), x, x, None, None, q_out)
    cs.cswattn_sync_status()
    p, o = c.place(1, 300 + 139)
    assert torch.equal(cache.v[p, o], x[-1]) and int(cache.position[p, 0, o]) == 300 + 139
