"""The paged-cache operators as measured workloads: cases, inputs, plain forms and 64-bit values.

Five operators serve a batch of sequences whose key/value rows lie in pages:

    append   new tokens: RMSNorm, rotary positions, value residual, rows into the pages
    attend   attention of each sequence's new tokens over its pages
    weigh    attention weight of every cached row, accumulated over the new tokens
    select   which rows a sequence keeps under a budget of rows
    move     the kept rows into the places of the evicted ones

A batch is ragged: sequence b has ``cache_len[b]`` rows before the call and the new tokens
``new_start[b] .. new_start[b + 1]``; token i of it is row ``cache_len[b] + i``. Rows of q past
``new_start[B]`` belong to nobody and are left as they were.
"""
import math
import random

import torch

own = False

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
EPS = 1e-6
BASE = 10000.0

# ------------------------------------------------------------------ cases


def listed():
    d24 = dict(H=12, Hk=4, D=128)
    long = dict(H=16, Hk=4, D=128)
    d12 = dict(H=6, Hk=6, D=128)
    half = dict(layout="half", rotary=1.0, scaling="none", factor=1.0)
    return [
        # One generation step of 32 sequences of the d24 layer: launch latency.
        dict(name="append step", op="append", B=32, cap=2048, page=64, new=1, ragged=1, pad=0, ve=True, **d24, **half),
        # Prompts of a long-context layer whose positions are stretched by 4.
        dict(name="append prompts", op="append", B=6, cap=8192, page=128, new=2500, ragged=2, pad=37, ve=True,
             layout="interleaved", rotary=0.5, scaling="yarn", factor=4.0, **long),
        # One chat, one token: the smallest call of the attention.
        dict(name="attend one chat", op="attend", B=1, cap=1000, page=16, window=1000, new=1, ragged=3, pad=0, **d12),
        # The decode step of the benchmark, 32 sequences, over pages.
        dict(name="attend step", op="attend", B=32, cap=2048, page=64, window=2048, new=1, ragged=0, pad=0, **d24),
        # Chunked prefill beside generation: ragged chunks over ragged caches, short window, narrow heads.
        dict(name="attend mixed", op="attend", B=13, cap=4100, page=48, window=1024, new=203, ragged=4, pad=5,
             H=8, Hk=2, D=64),
        # A long prompt's chunk over what is cached of it already.
        dict(name="attend prompt", op="attend", B=2, cap=8192, page=128, window=8192, new=2048, ragged=0, pad=0, **long),
        # The weights of a generation step and of a prompt's chunk.
        dict(name="weigh step", op="weigh", B=32, cap=2048, page=64, window=2048, new=1, ragged=5, pad=0, **d24),
        dict(name="weigh chunk", op="weigh", B=3, cap=4500, page=128, window=4500, new=1024, ragged=6, pad=11, **long),
        # A cache one row over its budget, and a long one that loses most of its rows.
        dict(name="select one over", op="select", B=32, cap=1025, page=16, keep=1024, recent=256, ragged=0, **d24),
        dict(name="select long", op="select", B=4, cap=40000, page=128, keep=4096, recent=1000, ragged=7, **long),
        dict(name="move few", op="move", B=3, cap=700, page=16, keep=600, recent=64, ragged=8, H=8, Hk=2, D=64),
        dict(name="move long", op="move", B=16, cap=16384, page=128, keep=8192, recent=2048, ragged=9, **long),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "weigh", "select", "move"])
    Hk = rng.choice([1, 2, 4, 4, 6, 8])
    g = rng.choice([1, 2, 3, 4, 4, 5, 8, 16]) if Hk <= 2 else rng.choice([1, 2, 3, 4])
    c = dict(op=op, H=Hk * g, Hk=Hk, D=rng.choice([64, 128, 128]), page=rng.choice([16, 32, 48, 64, 128, 256]),
             ragged=rng.randrange(1, 1 << 30))
    if op == "append":
        c.update(B=_log(rng, 1, 64), new=_log(rng, 1, 2500), pad=rng.choice([0, 0, 1, 40]), ve=rng.random() < 0.5)
        c["new"] = max(1, min(c["new"], 15000 // c["B"], 200000 // (c["B"] * c["H"])))
        c["cap"] = c["new"] + _log(rng, 1, 6000)
        c.update(layout=rng.choice(["half", "interleaved"]), rotary=rng.choice([1.0, 1.0, 0.5, 0.25]),
                 scaling=rng.choice(["none", "linear", "ntk", "yarn"]), factor=1.0)
        if c["scaling"] != "none":
            c["factor"] = rng.choice([2.0, 4.0, 8.0])
    elif op in ("attend", "weigh"):
        c["B"] = _log(rng, 1, 48)
        c["new"] = 1 if rng.random() < 0.4 else _log(rng, 2, 2048)
        c["cap"] = _log(rng, max(16, c["new"]), 8192)
        # no more scores than the largest listed case computes, no more rows than fit its states
        while c["B"] * c["H"] * c["new"] * c["cap"] > 2 * 16 * 2048 * 8192 or c["B"] * c["Hk"] * c["cap"] > 600000:
            c["B"] = max(1, c["B"] // 2)
            if c["B"] == 1:
                c["new"] = max(1, c["new"] // 2)
                c["cap"] = max(c["new"], c["cap"] * 3 // 4)
        c["window"] = rng.choice([c["cap"], c["cap"], _log(rng, 1, c["cap"])])
        c["pad"] = rng.choice([0, 0, 3, 130])
    else:
        c["B"] = _log(rng, 1, 32)
        c["cap"] = _log(rng, 40, 40000)
        while c["B"] * c["Hk"] * c["cap"] * (c["D"] if op == "move" else 8) > 16 * 4 * 16384 * 128:
            c["B"] = max(1, c["B"] // 2)
            if c["B"] == 1:
                c["cap"] = max(40, c["cap"] // 2)
        c["keep"] = rng.choice([max(1, c["cap"] - 1), _log(rng, 1, c["cap"])])
        c["recent"] = rng.randrange(0, c["keep"] + 1)
    return c


def _lengths(case):
    """(rows before the call, new tokens) of each sequence: the case alone says them, so that its work is known."""
    r = random.Random(case["ragged"])
    B, cap, new = case["B"], case["cap"], case.get("new", 0)
    lens, news = [], []
    for b in range(B):
        if case["ragged"] == 0:  # every sequence full
            n = new
            L = cap - n
        else:
            n = new if b == 0 else r.choice([new, r.randrange(0, new + 1), min(new, 1)])
            L = cap - n if b == B - 1 else r.randrange(0, cap - n + 1)
        lens.append(L)
        news.append(n)
    return lens, news


# ------------------------------------------------------------------ inputs


def _rotary_dim(case):
    return int(case["D"] * case["rotary"])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev = "cuda"

    def normal(*shape, dtype=BF):
        return torch.randn(*shape, generator=g, device=dev, dtype=F32).to(dtype)

    B, Hk, D, page = case["B"], case["Hk"], case["D"], case["page"]
    lens, news = _lengths(case)
    pps = -(-case["cap"] // page)
    n_pages = B * pps + 3  # a few pages nobody has
    order = torch.randperm(n_pages, generator=g, device=dev)
    s = dict(case=case, lens=lens, news=news, n_pages=n_pages, pages_per_seq=pps)
    s["page_table"] = order[: B * pps].to(I32).view(B, pps).contiguous()
    s["cache_len"] = torch.tensor(lens, dtype=I32, device=dev)
    start = [0]
    for n in news:
        start.append(start[-1] + n)
    s["new_start"] = torch.tensor(start, dtype=I32, device=dev)
    op = case["op"]
    if op in ("append", "attend", "weigh"):
        N = start[-1] + case["pad"]
        s["N"], s["max_new"] = N, case["new"]
        s["q"] = normal(N, case["H"], D)
    if op == "append":
        s["k"], s["v"] = normal(N, Hk, D), normal(N, Hk, D)
        s["ve"] = normal(N, Hk, D) if case["ve"] else None
        s["gate"] = normal(N, Hk) if case["ve"] else None
        s["q_out"] = torch.zeros_like(s["q"])
        # a stretched context holds positions past the trained ones
        far = 1 if case["scaling"] == "none" else int(case["factor"])
        tok = torch.arange(N, device=dev)
        b = torch.searchsorted(s["new_start"].long(), tok, right=True).clamp(max=B) - 1
        s["positions"] = ((s["cache_len"].long()[b] + tok - s["new_start"].long()[b]) * far).to(I32)
    if op in ("attend", "weigh"):
        # queries and keys as the prologue leaves them: rows of root mean square 1
        x = s["q"].float()
        s["q"] = (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)).to(BF)
        s["O"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros(N, case["H"], dtype=F32, device=dev)
    if op == "weigh":  # the log-sum-exp of each row is of this size where the keys are random
        see = torch.arange(1, N + 1, device=dev, dtype=F32).clamp(max=float(case["window"]))
        s["lse"] += torch.log(see.clamp(min=float(max(1, case["cap"] // 2)))).unsqueeze(1) + 0.5
    # the pools
    if op != "select":
        k = normal(n_pages, page, Hk, D, dtype=F32)
        s["k_pages"] = (k * torch.rsqrt(k.square().mean(-1, keepdim=True) + EPS)).to(BF)
        del k
        if op != "weigh":
            s["v_pages"] = normal(n_pages, page, Hk, D)
    if op != "attend":
        w = torch.exp(2 * torch.randn(n_pages, Hk, page, generator=g, device=dev))
        s["weight"] = torch.round(w * 64) / 64  # equal weights are met: ties
        if op == "weigh":
            s["weight"] /= 1024  # rows seen a few times: the call's own sums are not lost beside them
        s["position"] = torch.zeros(n_pages, Hk, page, dtype=I32, device=dev)
    if op in ("select", "move"):
        # rows of earlier evictions lie in no order: each head's positions are a permutation of its own
        s["next_pos"] = (s["cache_len"] * 2).to(I32)
        row = torch.arange(pps * page, device=dev).expand(B, Hk, -1)
        r = torch.rand(B, Hk, pps * page, generator=g, device=dev)
        r = torch.where(row < s["cache_len"].view(B, 1, 1), r, 2.0)
        pos = (2 * r.argsort(-1).argsort(-1) + (r > 0.5)).to(I32)
        pages = s["page_table"].long()
        s["position"][pages.reshape(-1)] = (
            pos.view(B, Hk, pps, page).permute(0, 2, 1, 3).reshape(-1, Hk, page))
        K = case["keep"]
        s["src"] = torch.full((B, Hk, K), -1, dtype=I32, device=dev)
        s["dst"] = torch.full((B, Hk, K), -1, dtype=I32, device=dev)
        s["n_moves"] = torch.zeros(B, Hk, dtype=I32, device=dev)
        s["new_len"] = torch.zeros(B, dtype=I32, device=dev)
    if op == "move":
        s["n_moves"], s["src"], s["dst"], s["new_len"] = _plain_select(s)
    return s


# ------------------------------------------------------------------ plain forms


def _frequencies(case):
    """Angle of one position for each pair of the rotary part, in 64 bits, and the factor on cos and sin."""
    R, f = _rotary_dim(case), case["factor"]
    i = torch.arange(R // 2, dtype=torch.float64, device="cuda")
    w = BASE ** (-2 * i / R)
    if case["scaling"] == "linear":
        return w / f, 1.0
    if case["scaling"] == "ntk":
        return (BASE * f ** (R / (R - 2))) ** (-2 * i / R), 1.0
    if case["scaling"] == "yarn":
        def pair_of(turns):
            return R * math.log(2048 / (turns * 2 * math.pi)) / (2 * math.log(BASE))
        lo, hi = max(math.floor(pair_of(32.0)), 0), min(math.ceil(pair_of(1.0)), R // 2 - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return w * (1 - ramp) + w / f * ramp, 0.1 * math.log(f) + 1.0
    return w, 1.0


def _tokens(s):
    """Sequence and row of each token that has one."""
    start = s["new_start"].long()
    n = start[-1]
    tok = torch.arange(s["N"], device="cuda")
    b = (torch.searchsorted(start, tok, right=True) - 1).clamp(max=s["case"]["B"] - 1)
    return tok < n, b, s["cache_len"].long()[b] + tok - start[b]


def _rope(x, positions, case):
    w, factor = _frequencies(case)
    R = _rotary_dim(case)
    angle = positions.double().unsqueeze(1) * w
    cos = (torch.cos(angle) * factor).float().unsqueeze(1)
    sin = (torch.sin(angle) * factor).float().unsqueeze(1)
    x = x.float()
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    y = x.clone()
    if case["layout"] == "half":
        a, b = x[..., : R // 2], x[..., R // 2: R]
        y[..., : R // 2] = a * cos - b * sin
        y[..., R // 2: R] = a * sin + b * cos
    else:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y[..., 0:R:2] = a * cos - b * sin
        y[..., 1:R:2] = a * sin + b * cos
    return y.to(BF)


def _plain_append(s):
    case, page = s["case"], s["case"]["page"]
    has, b, row = _tokens(s)
    s["q_out"][has] = _rope(s["q"], s["positions"], case)[has]
    v = s["v"].float()
    if s["ve"] is not None:
        v = v + (3 * torch.sigmoid(s["gate"].float())).unsqueeze(-1) * s["ve"].float()
    b, row = b[has], row[has]
    at = s["page_table"].long()[b, row // page]
    s["k_pages"][at, row % page] = _rope(s["k"], s["positions"], case)[has]
    s["v_pages"][at, row % page] = v.to(BF)[has]
    s["weight"][at, :, row % page] = 0.0
    s["position"][at, :, row % page] = s["positions"][has].unsqueeze(1)
    return dict(q_out=s["q_out"], k=s["k_pages"], v=s["v_pages"], weight=s["weight"], position=s["position"])


def _rows(pool, s):
    """(B, rows, Hk, D) of each sequence's pages in order."""
    x = pool[s["page_table"].long()]
    return x.reshape(x.shape[0], -1, *x.shape[3:])


def _scores(s):
    """Scaled scores (B, Hk, g, n, rows), which of them are seen, and the padded tokens' places."""
    case = s["case"]
    B, Hk, n = case["B"], case["Hk"], s["max_new"]
    g = case["H"] // Hk
    start, lens = s["new_start"].long(), s["cache_len"].long()
    i = torch.arange(n, device="cuda")
    tok = start[:-1].unsqueeze(1) + i
    has = tok < start[1:].unsqueeze(1)
    q = s["q"].float()[torch.where(has, tok, 0)].view(B, n, Hk, g, case["D"])
    k = _rows(s["k_pages"], s).float()
    score = torch.einsum("bnkgd,bskd->bkgns", q, k) * (case["D"] ** -0.5)
    row = lens.unsqueeze(1) + i  # of each token
    key = torch.arange(k.shape[1], device="cuda")
    seen = (key <= row.unsqueeze(2)) & (key > row.unsqueeze(2) - case["window"]) & has.unsqueeze(2)
    return score, seen.view(B, 1, 1, n, -1), tok, has


def _plain_attend(s):
    score, seen, tok, has = _scores(s)
    score = score.masked_fill_(~seen, -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    p = (score - top).exp_()
    total = p.sum(-1, keepdim=True)
    v = _rows(s["v_pages"], s).float()
    o = torch.einsum("bkgns,bskd->bnkgd", p / total.clamp(min=1e-30), v)
    lse = (top + total.log()).squeeze(-1).permute(0, 3, 1, 2)
    s["O"][tok[has]] = o.flatten(2, 3)[has].to(BF)
    s["lse"][tok[has]] = lse.flatten(2, 3)[has]
    return dict(O=s["O"], lse=s["lse"])


def _plain_weigh(s):
    case, page = s["case"], s["case"]["page"]
    score, seen, tok, has = _scores(s)
    B, Hk, n = case["B"], case["Hk"], s["max_new"]
    lse = s["lse"][torch.where(has, tok, 0)].view(B, n, Hk, -1).permute(0, 2, 3, 1).unsqueeze(-1)
    p = (score - lse).exp_().masked_fill_(~seen, 0.0).sum((2, 3))  # (B, Hk, rows)
    p = p.view(B, Hk, -1, page).transpose(1, 2)
    at = s["page_table"].long()
    s["weight"][at] = s["weight"][at] + p
    return dict(weight=s["weight"])


def _plain_select(s):
    case = s["case"]
    B, Hk, K = case["B"], case["Hk"], case["keep"]
    at = s["page_table"].long()
    w = s["weight"][at].transpose(1, 2).reshape(B, Hk, -1)
    pos = s["position"][at].transpose(1, 2).reshape(B, Hk, -1)
    row = torch.arange(w.shape[-1], device="cuda")
    L = s["cache_len"].long().view(B, 1, 1)
    w = torch.where(pos >= s["next_pos"].view(B, 1, 1) - case["recent"], math.inf, w)
    w = torch.where(row < L, w, -math.inf)
    rank = torch.sort(w, dim=-1, descending=True, stable=True).indices.argsort(-1)
    kept = (rank < K) & (row < L)
    hole = ~kept & (row < K) & (row < L)
    mover = kept & (row >= K)
    n = mover.sum(-1, dtype=I32)

    def places(mask):  # the rows of a mask in order, then -1
        x = torch.where(mask, row, 1 << 30).sort(-1).values
        x = torch.nn.functional.pad(x, (0, max(0, K - x.shape[-1])), value=1 << 30)[..., :K]
        return torch.where(torch.arange(K, device="cuda") < n.unsqueeze(-1), x, -1).to(I32)

    return n, places(mover), places(hole), s["cache_len"].clamp(max=K)


def _plain_move(s):
    case, page = s["case"], s["case"]["page"]
    B, Hk, K = case["B"], case["Hk"], case["keep"]
    has = (torch.arange(K, device="cuda") < s["n_moves"].unsqueeze(-1)).reshape(-1)
    b = torch.arange(B, device="cuda").view(B, 1, 1).expand(B, Hk, K).reshape(-1)[has]
    h = torch.arange(Hk, device="cuda").view(1, Hk, 1).expand(B, Hk, K).reshape(-1)[has]
    src, dst = s["src"].long().reshape(-1)[has], s["dst"].long().reshape(-1)[has]
    table = s["page_table"].long()
    ps, pd = table[b, src // page], table[b, dst // page]
    for name in ("k_pages", "v_pages"):
        s[name][pd, dst % page, h] = s[name][ps, src % page, h]
    for name in ("weight", "position"):
        s[name][pd, h, dst % page] = s[name][ps, h, src % page]
    return dict(k=s["k_pages"], v=s["v_pages"], weight=s["weight"], position=s["position"])


# ------------------------------------------------------------------ one pass


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if not own:
        if op == "append":
            return _plain_append(s)
        if op == "attend":
            return _plain_attend(s)
        if op == "weigh":
            return _plain_weigh(s)
        if op == "select":
            n, src, dst, new_len = _plain_select(s)
            return dict(n_moves=n, src=src, dst=dst, new_len=new_len)
        return _plain_move(s)

    import causal_sliding_window_rope_b200 as cs
    spec = cs.LayerSpec(case["B"], case["cap"], case["H"], case["Hk"], case["D"], case.get("window", case["cap"]),
                        has_ve=case.get("ve", False), rope_base=BASE, eps=EPS)
    cache = cs.PagedCache(spec, k=s.get("k_pages"), v=s.get("v_pages"), weight=s.get("weight"),
                          position=s.get("position"))
    batch = cs.PagedBatch(s["page_table"], s["cache_len"], s["new_start"], n_tokens=s.get("N", 0),
                          max_new=s.get("max_new", 0))
    if op == "append":
        rope = cs.RopeSpec(_rotary_dim(case), interleaved=case["layout"] == "interleaved", scaling=case["scaling"],
                           factor=case["factor"], original_length=2048)
        cs.attn_paged_append(spec, batch, cache, s["q"], s["k"], s["v"], s["ve"], s["gate"], s["q_out"],
                             positions=s["positions"], rope=rope)
        return dict(q_out=s["q_out"], k=s["k_pages"], v=s["v_pages"], weight=s["weight"], position=s["position"])
    if op == "attend":
        if "workspace" not in s:  # kept by the program, as the layer's buffers are
            s["workspace"] = torch.empty(max(1, cs.attn_paged_workspace_bytes(spec, batch, cache)),
                                         dtype=torch.uint8, device="cuda")
        cs.attn_paged(spec, batch, cache, s["q"], s["O"], s["lse"], s["workspace"])
        return dict(O=s["O"], lse=s["lse"])
    if op == "weigh":
        cs.attn_paged_weigh(spec, batch, cache, s["q"], s["lse"])
        return dict(weight=s["weight"])
    if op == "select":
        cs.attn_paged_select(spec, batch, cache, s["next_pos"], case["keep"], case["recent"], s["n_moves"], s["src"],
                             s["dst"], s["new_len"])
        return dict(n_moves=s["n_moves"], src=s["src"], dst=s["dst"], new_len=s["new_len"])
    cs.attn_paged_move(spec, batch, cache, s["n_moves"], s["src"], s["dst"])
    return dict(k=s["k_pages"], v=s["v_pages"], weight=s["weight"], position=s["position"])


# ------------------------------------------------------------------ work


def work(case):
    """Bytes and operations that one pass cannot do without."""
    B, Hk, D, H = case["B"], case["Hk"], case["D"], case["H"]
    lens, news = _lengths(case)
    n = sum(news)
    op = case["op"]
    if op == "append":
        ve = Hk * D * 2 + Hk * 2 if case["ve"] else 0
        return {"bytes": n * (2 * H * D * 2 + 4 * Hk * D * 2 + ve + 4 + 8 * Hk), "flops": n * (H + Hk) * D * 8}
    if op in ("attend", "weigh"):
        W = case["window"]
        rows = pairs = 0
        for L, m in zip(lens, news):
            if m:
                rows += L + m - max(0, L - W + 1)
                full = max(0, min(m, W - 1 - L))  # tokens that see every row before them
                pairs += full * L + full * (full + 1) // 2 + (m - full) * W
        if op == "attend":
            return {"bytes": rows * Hk * D * 4 + n * H * (D * 4 + 4), "flops": 4 * D * H * pairs}
        return {"bytes": rows * Hk * (D * 2 + 8) + n * H * (D * 2 + 4), "flops": 2 * D * H * pairs}
    K, R = case["keep"], case["recent"]
    moved = 0.0
    for L in lens:
        if L > K:  # a row's weight and age say nothing of its place
            moved += Hk * (L - K) * K / L
    if op == "select":
        return {"bytes": sum(lens) * Hk * 8 + B * Hk * (K * 8 + 4), "flops": sum(lens) * Hk}
    return {"bytes": moved * (8 + 2 * (4 * D + 8)) + B * Hk * 4, "flops": 0}


# ------------------------------------------------------------------ 64 bits


def _exact_rope(x, pos, case):
    """One token's heads (heads, D) in 64 bits, rotated as complex numbers."""
    R, f = _rotary_dim(case), case["factor"]
    x = x.double()
    x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS)
    j = torch.arange(0, R, 2, dtype=torch.float64, device=x.device)
    theta = torch.exp(-j / R * math.log(BASE))
    factor = 1.0
    if case["scaling"] == "linear":
        theta = theta / f
    elif case["scaling"] == "ntk":
        theta = torch.exp(-j / R * (math.log(BASE) + R / (R - 2) * math.log(f)))
    elif case["scaling"] == "yarn":
        first = max(0, math.floor(R * math.log(2048 / (64 * math.pi)) / (2 * math.log(BASE))))
        last = min(R // 2 - 1, math.ceil(R * math.log(2048 / (2 * math.pi)) / (2 * math.log(BASE))))
        slow = torch.clamp((j / 2 - first) / max(last - first, 0.001), 0, 1)
        theta = theta * (1 - slow + slow / f)
        factor = 1.0 + math.log(f) / 10
    turn = torch.polar(torch.full_like(theta, factor).expand(pos.shape[0], -1), pos.double()[:, None] * theta)[:, None]
    out = x.clone()
    if case["layout"] == "half":
        z = torch.complex(x[..., : R // 2], x[..., R // 2: R]) * turn
        out[..., :R] = torch.cat([z.real, z.imag], -1)
    else:
        z = torch.view_as_complex(x[..., :R].reshape(*x.shape[:-1], R // 2, 2).contiguous()) * turn
        out[..., :R] = torch.view_as_real(z).flatten(-2)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op, page, B, Hk, D = case["op"], case["page"], case["B"], case["Hk"], case["D"]
    table = s["page_table"].long()
    if op == "select":
        return None  # whole numbers only
    if op == "append":
        out = dict(q_out=s["q_out"].double(), k=s["k_pages"].double(), v=s["v_pages"].double(),
                   weight=s["weight"].double(), position=None)
        at = 0
        for b, (L, n) in enumerate(zip(s["lens"], s["news"])):
            t = slice(at, at + n)
            r = torch.arange(L, L + n, device="cuda")
            p, o = table[b, r // page], r % page
            out["q_out"][t] = _exact_rope(s["q"][t], s["positions"][t], case)
            out["k"][p, o] = _exact_rope(s["k"][t], s["positions"][t], case)
            v = s["v"][t].double()
            if case["ve"]:
                v = v + 3 / (1 + torch.exp(-s["gate"][t].double()))[..., None] * s["ve"][t].double()
            out["v"][p, o] = v
            out["weight"][p, :, o] = 0
            at += n
        return out
    if op == "move":
        out = dict(k=s["k_pages"].double(), v=s["v_pages"].double(), weight=s["weight"].double(), position=None)
        for b in range(B):
            for h in range(Hk):
                m = int(s["n_moves"][b, h])
                a, z = s["src"][b, h, :m].long(), s["dst"][b, h, :m].long()
                for name in ("k", "v"):
                    out[name][table[b, z // page], z % page, h] = out[name][table[b, a // page], a % page, h]
                out["weight"][table[b, z // page], h, z % page] = out["weight"][table[b, a // page], h, a % page]
        return out
    # attend, weigh: one sequence and KV head at a time, in blocks of tokens
    g = case["H"] // Hk
    O, lse_out = s["O"].double(), s["lse"].double()
    weight = s["weight"].double() if op == "weigh" else None
    at = 0
    for b, (L, n) in enumerate(zip(s["lens"], s["news"])):
        if n == 0:
            continue
        r = torch.arange(L + n, device="cuda")
        p, o = table[b, r // page], r % page
        for h in range(Hk):
            k = s["k_pages"][p, o, h].double()
            v = s["v_pages"][p, o, h].double() if op == "attend" else None
            total = torch.zeros(L + n, dtype=torch.float64, device="cuda")
            for i0 in range(0, n, 512):
                i1 = min(n, i0 + 512)
                q = s["q"][at + i0: at + i1, h * g: (h + 1) * g].double()
                x = (q @ k.T) / math.sqrt(D)  # (tokens, g, rows)
                row = torch.arange(L + i0, L + i1, device="cuda")[:, None, None]
                out_of_sight = (r > row) | (r <= row - case["window"])
                x = x.masked_fill(out_of_sight, -math.inf)
                if op == "attend":
                    z = torch.logsumexp(x, -1)
                    lse_out[at + i0: at + i1, h * g: (h + 1) * g] = z
                    O[at + i0: at + i1, h * g: (h + 1) * g] = torch.exp(x - z[..., None]) @ v
                else:
                    z = s["lse"][at + i0: at + i1, h * g: (h + 1) * g].double()
                    total += torch.exp(x - z[..., None]).sum((0, 1))
            if op == "weigh":
                weight[p, h, o] += total
        at += n
    return dict(O=O, lse=lse_out) if op == "attend" else dict(weight=weight)
