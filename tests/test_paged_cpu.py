"""Paged cache, on the host: what the entry points refuse, before anything is
enqueued, and the frequencies of stretched contexts."""
import ctypes
import math

import pytest

import causal_sliding_window_rope_b200 as cs
from causal_sliding_window_rope_b200 import build as cs_build


@pytest.fixture(scope="module")
def lib():
    cs_build.build()
    return cs.lib()


LAYER = dict(B=3, T=100, n_head=8, n_kv_head=2, head_dim=128, window=50, has_ve=True)
PAGED = dict(page_size=16, n_pages=30, pages_per_seq=7, n_tokens=10, max_new=5, page_table=256, cache_len=256,
             new_start=256)


def structs(layer=(), paged=()):
    return cs.LayerSpec(**{**LAYER, **dict(layer)}).c(), cs.CswattnPaged(**{**PAGED, **dict(paged)})


P = 1024  # a pointer that is never followed: every call here is refused


def call(lib, name, layer, paged, **change):
    a = dict(attn_paged_append=dict(rope=None, q=P, k=2 * P, v=3 * P, ve=4 * P, gate=5 * P, positions=6 * P, q_out=7 * P,
                                    k_pages=8 * P, v_pages=9 * P, weight=10 * P, position=11 * P),
             attn_paged=dict(q_out=P, k_pages=2 * P, v_pages=3 * P, O=4 * P, lse=5 * P, workspace=6 * P, size=0),
             attn_paged_weigh=dict(q_out=P, k_pages=2 * P, lse=3 * P, weight=4 * P, workspace=5 * P, size=1 << 40),
             attn_paged_select=dict(weight=P, position=2 * P, next_pos=3 * P, n_keep=40, n_recent=4, n_moves=4 * P,
                                    src=5 * P, dst=6 * P, new_len=7 * P),
             attn_paged_move=dict(n_moves=P, src=2 * P, dst=3 * P, n_keep=40, k_pages=4 * P, v_pages=5 * P, weight=6 * P,
                                  position=7 * P))[name]
    assert set(change) <= set(a)
    a.update(change)
    return getattr(lib, name)(None if layer is None else ctypes.byref(layer), None if paged is None else ctypes.byref(paged),
                              *a.values(), None)


ALL = ("attn_paged_append", "attn_paged", "attn_paged_weigh", "attn_paged_select", "attn_paged_move")


@pytest.mark.parametrize("name", ALL)
@pytest.mark.parametrize("layer,paged,code", [
    (dict(B=0), {}, cs.ERR_INVALID_ARG),
    (dict(T=0), {}, cs.ERR_INVALID_ARG),
    (dict(window=0), {}, cs.ERR_INVALID_ARG),
    (dict(n_kv_head=3), {}, cs.ERR_INVALID_ARG),
    (dict(head_dim=96), {}, cs.ERR_UNSUPPORTED),
    (dict(dtype="f32"), {}, cs.ERR_UNSUPPORTED),
    (dict(n_head=258, n_kv_head=2), {}, cs.ERR_UNSUPPORTED),
    (dict(B=4097), {}, cs.ERR_UNSUPPORTED),
    (dict(T=(1 << 20) + 1), dict(pages_per_seq=1 << 20), cs.ERR_UNSUPPORTED),
    (dict(T=113), {}, cs.ERR_INVALID_ARG),            # does not fit 7 pages of 16
    ({}, dict(page_size=0), cs.ERR_INVALID_ARG),
    ({}, dict(page_size=24, pages_per_seq=9), cs.ERR_UNSUPPORTED),
    ({}, dict(n_pages=0), cs.ERR_INVALID_ARG),
    ({}, dict(pages_per_seq=-1), cs.ERR_INVALID_ARG),
    ({}, dict(page_table=None), cs.ERR_INVALID_ARG),
    ({}, dict(cache_len=None), cs.ERR_INVALID_ARG),
    ({}, dict(cache_len=258), cs.ERR_INVALID_ARG),
])
def test_layer_and_batch_refused(lib, name, layer, paged, code):
    assert call(lib, name, *structs(layer, paged)) == code
    assert lib.cswattn_last_error() != b""
    assert lib.attn_paged_workspace_bytes(*map(ctypes.byref, structs(layer, paged))) == 0


@pytest.mark.parametrize("name", ALL)
def test_null_structs(lib, name):
    layer, paged = structs()
    assert call(lib, name, None, paged) == cs.ERR_INVALID_ARG
    assert call(lib, name, layer, None) == cs.ERR_INVALID_ARG


@pytest.mark.parametrize("name", ALL[:3])
@pytest.mark.parametrize("paged", [dict(n_tokens=-1), dict(max_new=0), dict(max_new=101), dict(new_start=None)])
def test_token_counts_refused(lib, name, paged):
    assert call(lib, name, *structs((), paged)) == cs.ERR_INVALID_ARG


@pytest.mark.parametrize("name", ALL[:3])
def test_no_tokens_enqueue_nothing(lib, name):
    layer, paged = structs((), dict(n_tokens=0))
    assert call(lib, name, layer, paged) == cs.OK  # no device here: a launch would have failed


def test_a_budget_of_every_row_moves_nothing(lib):
    layer, paged = structs()
    assert call(lib, "attn_paged_move", layer, paged, n_keep=100) == cs.OK


@pytest.mark.parametrize("name,args", [
    ("attn_paged_append", ("q", "k", "v", "ve", "gate", "q_out", "k_pages", "v_pages")),
    ("attn_paged", ("q_out", "k_pages", "v_pages", "O", "lse", "workspace")),
    ("attn_paged_weigh", ("q_out", "k_pages", "lse", "weight")),
    ("attn_paged_select", ("weight", "position", "next_pos", "n_moves", "src", "dst", "new_len")),
    ("attn_paged_move", ("n_moves", "src", "dst", "k_pages", "v_pages", "weight", "position")),
])
def test_pointers_refused(lib, name, args):
    layer, paged = structs()
    size = dict(size=1 << 40) if name == "attn_paged" else {}
    for a in args:
        assert call(lib, name, layer, paged, **{a: None}, **size) == cs.ERR_INVALID_ARG, a
        assert call(lib, name, layer, paged, **{a: P + 1}, **size) == cs.ERR_INVALID_ARG, a


def test_append_refusals(lib):
    layer, paged = structs()
    bad = lambda **kw: call(lib, "attn_paged_append", layer, paged, **kw)  # noqa: E731
    assert bad(q_out=P) == cs.ERR_INVALID_ARG and b"alias" in lib.cswattn_last_error()
    assert bad(v_pages=8 * P) == cs.ERR_INVALID_ARG
    assert bad(weight=None) == cs.ERR_INVALID_ARG
    assert bad(position=None) == cs.ERR_INVALID_ARG
    assert bad(positions=P + 2) == cs.ERR_INVALID_ARG
    freq = (ctypes.c_double * 64)(*[1.0] * 64)
    for rope, code in ((dict(rotary_dim=0), cs.ERR_INVALID_ARG), (dict(rotary_dim=144), cs.ERR_INVALID_ARG),
                       (dict(rotary_dim=24), cs.ERR_UNSUPPORTED), (dict(interleaved=2), cs.ERR_INVALID_ARG),
                       (dict(factor=0.0), cs.ERR_INVALID_ARG), (dict(factor=math.inf), cs.ERR_INVALID_ARG)):
        r = cs.CswattnRope(**{**dict(rotary_dim=128, interleaved=0, factor=1.0, frequencies=freq), **rope})
        assert bad(rope=ctypes.byref(r)) == code, rope
    freq[5] = math.nan
    r = cs.CswattnRope(128, 0, 1.0, freq)
    assert bad(rope=ctypes.byref(r)) == cs.ERR_INVALID_ARG and b"frequency 5" in lib.cswattn_last_error()


def test_weigh_workspace(lib):
    for max_new, some in ((1, False), (8, False), (9, True), (100, True)):  # 4 heads a group
        layer, paged = structs((), dict(max_new=max_new, n_tokens=300))
        need = lib.attn_paged_weigh_workspace_bytes(ctypes.byref(layer), ctypes.byref(paged))
        assert (need > 0) == some
        if some:
            assert call(lib, "attn_paged_weigh", layer, paged, size=need - 1) == cs.ERR_INVALID_ARG
            assert b"workspace" in lib.cswattn_last_error()
            assert call(lib, "attn_paged_weigh", layer, paged, workspace=None) == cs.ERR_INVALID_ARG
    layer, paged = structs(dict(window=0))
    assert lib.attn_paged_weigh_workspace_bytes(ctypes.byref(layer), ctypes.byref(paged)) == 0


def test_attend_refusals(lib):
    layer, paged = structs()
    need = lib.attn_paged_workspace_bytes(ctypes.byref(layer), ctypes.byref(paged))
    assert need > 0
    assert call(lib, "attn_paged", layer, paged, size=need - 1) == cs.ERR_INVALID_ARG
    assert b"workspace" in lib.cswattn_last_error()
    assert call(lib, "attn_paged", layer, paged, size=1 << 40, O=P) == cs.ERR_INVALID_ARG
    assert b"alias" in lib.cswattn_last_error()


@pytest.mark.parametrize("change", [dict(n_keep=0), dict(n_keep=101), dict(n_recent=-1), dict(n_recent=41),
                                    dict(new_len=256)])
def test_select_refusals(lib, change):
    assert call(lib, "attn_paged_select", *structs(), **change) == cs.ERR_INVALID_ARG


@pytest.mark.parametrize("change", [dict(n_keep=0), dict(n_keep=101), dict(v_pages=4 * P)])
def test_move_refusals(lib, change):
    assert call(lib, "attn_paged_move", *structs(), **change) == cs.ERR_INVALID_ARG


def test_rope_frequencies():
    plain = [10000.0 ** (-2 * i / 64) for i in range(32)]
    assert cs.RopeSpec(64).frequencies == pytest.approx(plain, rel=1e-15)
    assert cs.RopeSpec(64, scaling="linear", factor=4.0).frequencies == pytest.approx([f / 4 for f in plain], rel=1e-15)
    ntk = cs.RopeSpec(64, scaling="ntk", factor=4.0).frequencies
    # the fastest pair as it was, the slowest stretched by the factor
    assert ntk[0] == 1.0 and ntk[31] == pytest.approx(plain[31] / 4, rel=1e-12)
    y = cs.RopeSpec(64, scaling="yarn", factor=4.0, original_length=2048)
    for i, (a, b) in enumerate(zip(y.frequencies, plain)):
        turns = 2048 * b / (2 * math.pi)
        assert b / 4 <= a * (1 + 1e-12) and a <= b * (1 + 1e-12)
        if turns > 45:  # one pair past beta_fast
            assert a == b, i
        if turns < 0.7:
            assert a == pytest.approx(b / 4, rel=1e-12), i
    assert y.attention_factor == pytest.approx(1 + 0.1 * math.log(4))
    own = cs.RopeSpec(16, frequencies=[0.5] * 8, attention_factor=2.0)
    assert own.frequencies == (0.5,) * 8 and own.attention_factor == 2.0


@pytest.mark.parametrize("kw", [dict(rotary_dim=3), dict(rotary_dim=0), dict(rotary_dim=16, scaling="other"),
                                dict(rotary_dim=16, factor=0.0), dict(rotary_dim=16, frequencies=[1.0]),
                                dict(rotary_dim=16, scaling="yarn", factor=2.0), dict(rotary_dim=2, scaling="ntk", factor=2.0),
                                dict(rotary_dim=16, base=-1.0)])
def test_rope_refusals(kw):
    with pytest.raises(ValueError):
        cs.RopeSpec(**kw)


def test_tensor_checks():
    import torch
    spec = cs.LayerSpec(**LAYER)
    with pytest.raises(ValueError):  # not a CUDA tensor
        cs.PagedCache(spec, n_pages=4, page_size=16, device="cpu")
    with pytest.raises(ValueError):
        cs.PagedCache(spec)
    with pytest.raises(ValueError):  # int64
        cs.PagedBatch(torch.zeros(3, 7, dtype=torch.int64), torch.zeros(3, dtype=torch.int32))
