"""B200-native causal sliding-window RoPE attention (forward and backward).

A thin ctypes binding over libcswattn.so, the C ABI declared in
``include/cswattn.h``. Every step of the computation runs in the library's
CUDA kernels; this module only marshals pointers, sizes and the stream.
PyTorch provides device memory and streams.

The layer is the attention of a nanochat-style GPT block (page
"5만원으로 나만의 ChatGPT 훈련하는 방법", section "1. GPT 모델"): RoPE,
parameter-free QK RMSNorm, GQA, a per-layer sliding window ("SSSL") and the
value-embedding residual v + 3*sigmoid(gate)*ve.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
from dataclasses import dataclass

from .configs import WORKLOADS, Workload, alternating_ve, window_pattern  # noqa: F401

_HERE = os.path.dirname(os.path.abspath(__file__))
# CSWATTN_CHECK=1 in the environment selects the checked build (device-side
# bounds checks that report CSWATTN_ERR_BOUNDS instead of faulting); build it
# with `python -m causal_sliding_window_rope_b200.build --check`.
CHECKED = os.environ.get("CSWATTN_CHECK", "0") == "1"
LIB_PATH = os.path.join(_HERE, "libcswattn_check.so" if CHECKED else "libcswattn.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_TIMEOUT, ERR_BOUNDS = 0, 1, 2, 3, 4, 5
F32, BF16 = 0, 1

# Every symbol the header declares; the CPU tests check the library exports them.
EXPORTS = ("attn_prologue", "attn_prologue_gated", "attn_gate_bwd", "attn_qkv_prologue",
           "attn_qkv_fp8_workspace_bytes", "attn_qkv_prologue_fp8", "attn_qkv_bwd", "attn_fwd",
           "attn_bwd_workspace_bytes", "attn_bwd", "attn_bwd_noalloc",
           "attn_decode_workspace_bytes", "attn_decode", "attn_paged_append",
           "attn_paged_workspace_bytes", "attn_paged", "attn_paged_weigh",
           "attn_paged_weigh_workspace_bytes", "attn_paged_select", "attn_paged_move", "cswattn_gemm_bf16",
           "muon_ns_workspace_bytes", "muon_newton_schulz",
           "cswattn_sync_status", "cswattn_set_wait_limit_ns", "cswattn_set_timing",
           "cswattn_kernel_times", "cswattn_selftest_wait_timeout", "cswattn_last_error",
           "cswattn_version")
KERNEL_KINDS = ("prologue", "fwd", "bwd_pre", "bwd", "bwd_epi", "decode", "gate_bwd", "gemm")


class CswattnLayer(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int), ("T", ctypes.c_int), ("n_head", ctypes.c_int),
        ("n_kv_head", ctypes.c_int), ("head_dim", ctypes.c_int), ("window", ctypes.c_int),
        ("rope_base", ctypes.c_float), ("eps", ctypes.c_float), ("softmax_scale", ctypes.c_float),
        ("has_ve", ctypes.c_int), ("dtype", ctypes.c_int),
    ]


class CswattnPaged(ctypes.Structure):
    _fields_ = [
        ("page_size", ctypes.c_int), ("n_pages", ctypes.c_int), ("pages_per_seq", ctypes.c_int),
        ("n_tokens", ctypes.c_int), ("max_new", ctypes.c_int), ("page_table", ctypes.c_void_p),
        ("cache_len", ctypes.c_void_p), ("new_start", ctypes.c_void_p),
    ]


class CswattnRope(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int), ("interleaved", ctypes.c_int), ("factor", ctypes.c_float),
                ("frequencies", ctypes.POINTER(ctypes.c_double))]


class CswattnError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"cswattn status {status}: {message}")
        self.status = status


_lib = None


def lib():
    """The loaded library. Raises if it has not been built: there is no fallback."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing; build it with "
                               "`python -m causal_sliding_window_rope_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, fp, sz = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t
        lp = ctypes.POINTER(CswattnLayer)
        L.attn_prologue.argtypes = [lp] + [vp] * 8 + [fp, fp, vp]
        L.attn_fwd.argtypes = [lp, vp, vp, vp, vp, fp, vp]
        ll, ci = ctypes.c_longlong, ctypes.c_int
        L.attn_prologue_gated.argtypes = [lp] + [vp] * 5 + [ll, ci, vp, vp, vp, vp, vp, fp, fp, vp]
        L.attn_gate_bwd.argtypes = [lp, vp, ll, ci, vp, vp, vp, fp, vp]
        L.attn_qkv_prologue.argtypes = [lp, vp, ll, ci] + [vp] * 8 + [fp, fp, vp]
        L.attn_qkv_prologue.restype = ci
        L.attn_qkv_fp8_workspace_bytes.argtypes = [lp, ci]
        L.attn_qkv_fp8_workspace_bytes.restype = sz
        L.attn_qkv_prologue_fp8.argtypes = [lp, vp, ll, ci] + [vp] * 8 + [fp, fp, fp, vp, sz, vp]
        L.attn_qkv_prologue_fp8.restype = ci
        L.attn_qkv_bwd.argtypes = [lp, vp, ll, ci] + [vp] * 5 + [fp, vp]
        L.attn_qkv_bwd.restype = ci
        cf = ctypes.c_float
        L.cswattn_gemm_bf16.argtypes = [ci, ci, ci, ci, vp, ll, ci, vp, ll, cf, cf, vp, ll, vp, ll, vp]
        L.cswattn_gemm_bf16.restype = ci
        L.muon_ns_workspace_bytes.argtypes = [ci, ci]
        L.muon_ns_workspace_bytes.restype = sz
        L.muon_newton_schulz.argtypes = [ci, ci, ctypes.POINTER(cf), ci, vp, vp, vp, sz, vp]
        L.muon_newton_schulz.restype = ci
        L.attn_bwd_workspace_bytes.argtypes = [lp]
        L.attn_bwd_workspace_bytes.restype = sz
        L.attn_bwd.argtypes = [lp] + [vp] * 7 + [fp, fp, vp, fp, vp] + [vp] * 6 + [sz, vp]
        L.cswattn_sync_status.argtypes = [vp]
        L.cswattn_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
        L.cswattn_set_wait_limit_ns.restype = ctypes.c_uint64
        L.cswattn_last_error.restype = ctypes.c_char_p
        L.cswattn_set_timing.argtypes = [ctypes.c_int]
        L.cswattn_set_timing.restype = None
        L.cswattn_kernel_times.argtypes = [ctypes.POINTER(ctypes.c_double),
                                           ctypes.POINTER(ctypes.c_int)]
        L.cswattn_kernel_times.restype = ctypes.c_int
        L.cswattn_selftest_wait_timeout.argtypes = [ctypes.c_uint64, vp]
        L.cswattn_selftest_wait_timeout.restype = ctypes.c_int
        L.attn_bwd_noalloc.argtypes = [lp] + [vp] * 7 + [fp, fp, vp, fp, vp] + [vp] * 5 + [vp]
        L.attn_decode_workspace_bytes.argtypes = [lp]
        L.attn_decode_workspace_bytes.restype = sz
        L.attn_decode.argtypes = [lp] + [vp] * 5 + [vp, vp, vp, vp, fp, vp, sz, vp]
        pp, rp = ctypes.POINTER(CswattnPaged), ctypes.POINTER(CswattnRope)
        L.attn_paged_append.argtypes = [lp, pp, rp] + [vp] * 12
        L.attn_paged_workspace_bytes.argtypes = [lp, pp]
        L.attn_paged_workspace_bytes.restype = sz
        L.attn_paged.argtypes = [lp, pp] + [vp] * 6 + [sz, vp]
        L.attn_paged_weigh.argtypes = [lp, pp] + [vp] * 5 + [sz, vp]
        L.attn_paged_weigh_workspace_bytes.argtypes = [lp, pp]
        L.attn_paged_weigh_workspace_bytes.restype = sz
        L.attn_paged_select.argtypes = [lp, pp] + [vp] * 3 + [ci, ci] + [vp] * 5
        L.attn_paged_move.argtypes = [lp, pp] + [vp] * 3 + [ci] + [vp] * 5
        for name in ("attn_paged_append", "attn_paged", "attn_paged_weigh", "attn_paged_select",
                     "attn_paged_move"):
            getattr(L, name).restype = ci
        for name in ("attn_prologue", "attn_prologue_gated", "attn_gate_bwd", "attn_fwd", "attn_bwd",
                     "attn_bwd_noalloc", "cswattn_sync_status"):
            getattr(L, name).restype = ctypes.c_int
        _lib = L
    return _lib


@dataclass
class LayerSpec:
    """Arguments of one layer, as in the C struct ``cswattn_layer``."""
    B: int
    T: int
    n_head: int
    n_kv_head: int
    head_dim: int
    window: int
    has_ve: bool = True
    dtype: str = "bf16"          # "bf16" or "f32"
    rope_base: float = 10000.0
    eps: float = 1e-6
    softmax_scale: float = 0.0   # 0: 1/sqrt(head_dim)

    def c(self) -> CswattnLayer:
        return CswattnLayer(self.B, self.T, self.n_head, self.n_kv_head, self.head_dim,
                            self.window, self.rope_base, self.eps, self.softmax_scale,
                            int(bool(self.has_ve)), BF16 if self.dtype == "bf16" else F32)


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if not x.is_contiguous():
        raise ValueError("tensors passed to cswattn must be contiguous")
    return x.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int):
    if status != OK:
        raise CswattnError(status, lib().cswattn_last_error().decode())


def attn_prologue(spec: LayerSpec, q, k, v, ve, gate, q_out, k_out, v_out, rstd_q, rstd_k,
                  stream=None):
    layer = spec.c()
    _check(lib().attn_prologue(ctypes.byref(layer), _ptr(q), _ptr(k), _ptr(v), _ptr(ve),
                               _ptr(gate), _ptr(q_out), _ptr(k_out), _ptr(v_out),
                               _ptr(rstd_q), _ptr(rstd_k), _stream(stream)))


def attn_prologue_gated(spec: LayerSpec, q, k, v, ve, x, gate_channels, w_gate, gate_out, q_out,
                        k_out, v_out, rstd_q, rstd_k, stream=None):
    """attn_prologue with the gate logits computed from the block input:
    gate_out = x[..., :gate_channels] @ w_gate.T (x (B, T, X) contiguous)."""
    layer = spec.c()
    _check(lib().attn_prologue_gated(ctypes.byref(layer), _ptr(q), _ptr(k), _ptr(v), _ptr(ve),
                                     _ptr(x), int(x.shape[-1]), int(gate_channels), _ptr(w_gate),
                                     _ptr(gate_out), _ptr(q_out), _ptr(k_out), _ptr(v_out),
                                     _ptr(rstd_q), _ptr(rstd_k), _stream(stream)))


def attn_gate_bwd(spec: LayerSpec, x, gate_channels, w_gate, dgate, dx, dw_gate, stream=None):
    """dx (B, T, gate_channels) and float32 dw_gate (Hk, gate_channels) of the
    gate projection, from dgate (the attention backward's dgate)."""
    layer = spec.c()
    _check(lib().attn_gate_bwd(ctypes.byref(layer), _ptr(x), int(x.shape[-1]), int(gate_channels),
                               _ptr(w_gate), _ptr(dgate), _ptr(dx), _ptr(dw_gate), _stream(stream)))


def attn_qkv_prologue(spec: LayerSpec, x, C, w_qkv, ve, gate, q, k, q_out, k_out, v_out, rstd_q,
                      rstd_k, stream=None):
    """The QKV projection of x[..., :C] by the stacked weight w_qkv, fused with
    the prologue (see the C header); q and k receive the raw projections."""
    layer = spec.c()
    _check(lib().attn_qkv_prologue(ctypes.byref(layer), _ptr(x), int(x.shape[-1]), int(C), _ptr(w_qkv),
                                   _ptr(ve), _ptr(gate), _ptr(q), _ptr(k), _ptr(q_out), _ptr(k_out),
                                   _ptr(v_out), _ptr(rstd_q), _ptr(rstd_k), _stream(stream)))


def attn_qkv_fp8_workspace_bytes(spec: LayerSpec, C) -> int:
    layer = spec.c()
    return int(lib().attn_qkv_fp8_workspace_bytes(ctypes.byref(layer), int(C)))


def attn_qkv_prologue_fp8(spec: LayerSpec, x, C, w_qkv, ve, gate, q, k, q_out, k_out, v_out, rstd_q,
                          rstd_k, scales, workspace, workspace_bytes=None, stream=None):
    """attn_qkv_prologue with both operands quantized to E4M3 with tensor-wise
    scales (written to `scales`); `workspace` holds the codes afterwards."""
    layer = spec.c()
    nbytes = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    _check(lib().attn_qkv_prologue_fp8(ctypes.byref(layer), _ptr(x), int(x.shape[-1]), int(C), _ptr(w_qkv),
                                       _ptr(ve), _ptr(gate), _ptr(q), _ptr(k), _ptr(q_out), _ptr(k_out),
                                       _ptr(v_out), _ptr(rstd_q), _ptr(rstd_k), _ptr(scales), _ptr(workspace),
                                       int(nbytes), _stream(stream)))


def attn_qkv_bwd(spec: LayerSpec, x, C, w_qkv, dQ, dK, dV, dx, dw_qkv, stream=None):
    """dx (B, T, C) and float32 dw_qkv of the projection from attn_bwd's dQ, dK, dV."""
    layer = spec.c()
    _check(lib().attn_qkv_bwd(ctypes.byref(layer), _ptr(x), int(x.shape[-1]), int(C), _ptr(w_qkv),
                              _ptr(dQ), _ptr(dK), _ptr(dV), _ptr(dx), _ptr(dw_qkv), _stream(stream)))


def attn_fwd(spec: LayerSpec, q_out, k_out, v_out, O, lse, stream=None):
    layer = spec.c()
    _check(lib().attn_fwd(ctypes.byref(layer), _ptr(q_out), _ptr(k_out), _ptr(v_out),
                          _ptr(O), _ptr(lse), _stream(stream)))


def attn_bwd_workspace_bytes(spec: LayerSpec) -> int:
    layer = spec.c()
    return int(lib().attn_bwd_workspace_bytes(ctypes.byref(layer)))


def attn_bwd(spec: LayerSpec, q, k, ve, gate, q_out, k_out, v_out, rstd_q, rstd_k, O, lse,
             dO, dQ, dK, dV, dve, dgate, workspace, workspace_bytes=None, stream=None):
    layer = spec.c()
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    _check(lib().attn_bwd(ctypes.byref(layer), _ptr(q), _ptr(k), _ptr(ve), _ptr(gate),
                          _ptr(q_out), _ptr(k_out), _ptr(v_out), _ptr(rstd_q), _ptr(rstd_k),
                          _ptr(O), _ptr(lse), _ptr(dO), _ptr(dQ), _ptr(dK), _ptr(dV),
                          _ptr(dve), _ptr(dgate), _ptr(workspace), workspace_bytes,
                          _stream(stream)))


# Size of the fixed scratch array behind attn_bwd_noalloc (bytes).
NOALLOC_SCRATCH_BYTES = 32 << 20


def attn_bwd_noalloc(spec: LayerSpec, q, k, ve, gate, q_out, k_out, v_out, rstd_q, rstd_k, O,
                     lse, dO, dQ, dK, dV, dve, dgate, stream=None):
    """attn_bwd for callers that cannot allocate device memory: the scratch is
    a fixed array inside the library (see the C header for the limit and for
    why overlapping calls must be ordered)."""
    layer = spec.c()
    _check(lib().attn_bwd_noalloc(ctypes.byref(layer), _ptr(q), _ptr(k), _ptr(ve), _ptr(gate),
                                  _ptr(q_out), _ptr(k_out), _ptr(v_out), _ptr(rstd_q),
                                  _ptr(rstd_k), _ptr(O), _ptr(lse), _ptr(dO), _ptr(dQ), _ptr(dK),
                                  _ptr(dV), _ptr(dve), _ptr(dgate), _stream(stream)))


def attn_decode_workspace_bytes(spec: LayerSpec) -> int:
    """Scratch bytes of attn_decode; spec.T is the cache capacity."""
    layer = spec.c()
    return int(lib().attn_decode_workspace_bytes(ctypes.byref(layer)))


def attn_decode(spec: LayerSpec, q, k, v, ve, gate, cache_len, k_cache, v_cache, O, lse,
                workspace, workspace_bytes=None, stream=None):
    """One decode step with a KV cache (spec.T = cache capacity, cache_len an
    int32 device tensor of B lengths): writes the new token's k~ / v_eff rows
    into the caches and its attention output O (B,H,D) and lse (B,H)."""
    layer = spec.c()
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    _check(lib().attn_decode(ctypes.byref(layer), _ptr(q), _ptr(k), _ptr(v), _ptr(ve), _ptr(gate),
                             _ptr(cache_len), _ptr(k_cache), _ptr(v_cache), _ptr(O), _ptr(lse),
                             _ptr(workspace), workspace_bytes, _stream(stream)))


# ------------------------------------------------------------------ paged cache

@functools.lru_cache(maxsize=64)
def _rope(R, interleaved, scaling, factor, base, original_length, beta_fast, beta_slow, attention_factor, frequencies):
    """(frequencies, factor on cos and sin, C struct, its address) of a RopeSpec."""
    if R < 2 or R % 2:
        raise ValueError(f"rotary_dim must be even and >= 2, got {R}")
    if scaling not in RopeSpec.SCALINGS:
        raise ValueError(f"scaling must be one of {RopeSpec.SCALINGS}, got {scaling!r}")
    if not (math.isfinite(factor) and factor > 0) or not (math.isfinite(base) and base > 0):
        raise ValueError("factor and base must be finite and > 0")
    scale = 1.0
    if frequencies is not None:
        w = list(frequencies)
        if len(w) != R // 2:
            raise ValueError(f"{R // 2} frequencies are wanted, got {len(w)}")
    else:
        if scaling == "ntk":
            if R == 2:
                raise ValueError("ntk scaling needs rotary_dim > 2")
            base = base * factor ** (R / (R - 2))
        w = [base ** (-2.0 * i / R) for i in range(R // 2)]
        if scaling == "linear":
            w = [f / factor for f in w]
        elif scaling == "yarn":
            if not original_length or base == 1.0:
                raise ValueError("yarn scaling needs original_length and a base other than 1")

            def pair_of(turns):  # the pair that turns this often within original_length
                return R * math.log(original_length / (turns * 2 * math.pi)) / (2 * math.log(base))
            low = max(math.floor(pair_of(beta_fast)), 0)
            # (the line may end past the last pair, R / 2 - 1, which then keeps a part of its frequency)
            high = min(math.ceil(pair_of(beta_slow)), R - 1)
            for i in range(R // 2):
                ramp = min(max((i - low) / max(high - low, 0.001), 0.0), 1.0)
                w[i] = w[i] * (1 - ramp) + w[i] / factor * ramp
            scale = 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
    scale = float(scale if attention_factor is None else attention_factor)
    struct = CswattnRope(R, int(interleaved), scale, (ctypes.c_double * len(w))(*w))
    return tuple(w), scale, struct, ctypes.addressof(struct)


class RopeSpec:
    """Rotary positions of attn_paged_append: the layout (halves, or pairs of
    neighbours when interleaved), how much of the head turns, and the
    frequencies of a stretched context:

    "none"     base^(-2i/R)
    "linear"   the same, divided by ``factor`` (positions interpolated)
    "ntk"      base * factor^(R/(R-2)) in the place of base
    "yarn"     pairs that turn more than ``beta_fast`` times within
               ``original_length`` positions as they are, those below
               ``beta_slow`` turns divided by ``factor``, a ramp between, and
               cos and sin times 0.1 ln(factor) + 1 (1 for a factor below 1)

    or ``frequencies``: one angle per position for each pair, in their place.
    ``attention_factor`` replaces the factor on cos and sin. ``base`` None is
    the ``rope_base`` of the layer that a call is made with (``of``); until
    then ``frequencies`` are those of the usual 10000.
    """

    SCALINGS = ("none", "linear", "ntk", "yarn")

    DEFAULT_BASE = 10000.0

    def __init__(self, rotary_dim, interleaved=False, scaling="none", factor=1.0, base=None,
                 original_length=None, beta_fast=32.0, beta_slow=1.0, attention_factor=None, frequencies=None):
        self.rotary_dim, self.interleaved = int(rotary_dim), bool(interleaved)
        if frequencies is not None:
            frequencies = tuple(float(f) for f in frequencies)
        # the layer's base still to come: how to make this of another one
        self._open = None
        if base is None:
            base = self.DEFAULT_BASE
            if frequencies is None:
                self._open = (self.rotary_dim, self.interleaved, scaling, factor, original_length, beta_fast, beta_slow,
                              attention_factor)
        self.frequencies, self.attention_factor, self._c, self.address = _rope(
            self.rotary_dim, self.interleaved, scaling, factor, base, original_length, beta_fast, beta_slow,
            attention_factor, frequencies)

    def of(self, spec: LayerSpec) -> RopeSpec:
        """This rotation in a layer: with the layer's base where none was given."""
        if self._open is None or spec.rope_base == self.DEFAULT_BASE:
            return self
        R, interleaved, scaling, factor, *rest = self._open
        # the float32 that the layer's C struct holds
        return RopeSpec(R, interleaved, scaling, factor, ctypes.c_float(spec.rope_base).value, *rest)


_paged = None


def _paged_calls():
    """The module that checks and makes the paged calls, bound to the loaded
    library. Raises if it has not been built: there is no fallback."""
    global _paged
    if _paged is None:
        import torch  # (the module is linked against its libraries)

        from .build import binding_id
        rebuild = "build it with `python -m causal_sliding_window_rope_b200.build`"
        try:
            from . import _paged_binding as m
        except ImportError as e:
            raise RuntimeError(f"_paged_binding.so is missing or does not fit this PyTorch; {rebuild}") from e
        if m.built_for != binding_id(torch.__version__):
            raise RuntimeError(f"found {m.built_for}, wanted {binding_id(torch.__version__)}; {rebuild}")
        L = lib()
        m.bind(CswattnError, *(ctypes.cast(f, ctypes.c_void_p).value for f in (
            L.attn_paged_append, L.attn_paged, L.attn_paged_weigh, L.attn_paged_select, L.attn_paged_move,
            L.cswattn_last_error)))
        _paged = m
    return _paged


class PagedCache:
    """The pools of a paged cache: k and v (n_pages, page_size, n_kv_head,
    head_dim) bf16 and, for eviction, weight (float32) and position (int32),
    (n_pages, n_kv_head, page_size). Allocates them (weight and position only
    with track_weights), or takes the tensors given."""

    def __init__(self, spec: LayerSpec, n_pages=None, page_size=None, track_weights=False, k=None, v=None,
                 weight=None, position=None, device="cuda"):
        import torch
        if n_pages is not None:
            kv, term = (n_pages, page_size, spec.n_kv_head, spec.head_dim), (n_pages, spec.n_kv_head, page_size)
            k = torch.empty(*kv, device=device, dtype=torch.bfloat16) if k is None else k
            v = torch.empty(*kv, device=device, dtype=torch.bfloat16) if v is None else v
            if track_weights:
                weight = torch.zeros(*term, device=device) if weight is None else weight
                position = torch.zeros(*term, device=device, dtype=torch.int32) if position is None else position
        self.n_pages, self.page_size = (_paged or _paged_calls()).check_cache(spec.n_kv_head, spec.head_dim, k, v,
                                                                              weight, position)
        self.k, self.v, self.weight, self.position = k, v, weight, position


class PagedBatch:
    """The sequences of a paged call: page_table (B, pages_per_seq), cache_len
    (B) and new_start (B + 1), int32 device tensors; n_tokens rows of q, and
    max_new, which no sequence's new tokens exceed (new_start, n_tokens and
    max_new are not needed to select and move rows). max_new chooses the
    kernels, by max_new times the heads of a group: above 32 those of long
    chunks run, for single tokens too. A tight bound is the fast one:
    called alone, a step of 32 sequences of 2048 rows, 12 heads on 4 of 128,
    takes 39 us with max_new 1 and 49 us with 512, its row weights 18 and 28."""

    def __init__(self, page_table, cache_len, new_start=None, n_tokens=0, max_new=0):
        (_paged or _paged_calls()).check_batch(page_table, cache_len, new_start)
        self.page_table, self.cache_len, self.new_start = page_table, cache_len, new_start
        self.n_tokens, self.max_new = n_tokens, max_new

    def c(self, cache: PagedCache) -> CswattnPaged:
        return CswattnPaged(cache.page_size, cache.n_pages, self.page_table.shape[1], self.n_tokens, self.max_new,
                            self.page_table.data_ptr(), self.cache_len.data_ptr(),
                            None if self.new_start is None else self.new_start.data_ptr())


def attn_paged_append(spec: LayerSpec, batch: PagedBatch, cache: PagedCache, q, k, v, ve, gate, q_out,
                      positions=None, rope: RopeSpec | None = None, stream=None):
    """The prologue of the batch's new tokens: q_out, and their rows of the
    cache. rope None: the layer's plain RoPE."""
    if rope is not None:
        rope = rope.of(spec)
    (_paged or _paged_calls()).append(spec, batch, cache, q, k, v, ve, gate, q_out, positions, rope, stream)


def attn_paged_workspace_bytes(spec: LayerSpec, batch: PagedBatch, cache: PagedCache) -> int:
    """Scratch bytes of attn_paged for this layer and the batch's sizes."""
    return int(lib().attn_paged_workspace_bytes(ctypes.byref(spec.c()), ctypes.byref(batch.c(cache))))


def attn_paged(spec: LayerSpec, batch: PagedBatch, cache: PagedCache, q_out, O, lse, workspace,
               workspace_bytes=None, stream=None):
    """Attention of the new tokens (q_out of attn_paged_append) over the
    cache: O (n_tokens, H, D) and lse (n_tokens, H)."""
    (_paged or _paged_calls()).attend(spec, batch, cache, q_out, O, lse, workspace, workspace_bytes, stream)


def attn_paged_weigh_workspace_bytes(spec: LayerSpec, batch: PagedBatch, cache: PagedCache) -> int:
    """Scratch bytes of attn_paged_weigh; 0 for a call of few query rows."""
    return int(lib().attn_paged_weigh_workspace_bytes(ctypes.byref(spec.c()), ctypes.byref(batch.c(cache))))


def attn_paged_weigh(spec: LayerSpec, batch: PagedBatch, cache: PagedCache, q_out, lse, workspace=None, stream=None):
    """Adds the new tokens' attention weights to cache.weight. workspace:
    attn_paged_weigh_workspace_bytes of scratch; None: a call that needs some
    takes it from PyTorch's allocator on its stream."""
    if workspace is None and batch.max_new * spec.n_head > 32 * spec.n_kv_head:  # fewer query rows need none
        import torch
        nbytes, device = attn_paged_weigh_workspace_bytes(spec, batch, cache), batch.page_table.device
        if stream is None:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
        else:
            s = torch.cuda.ExternalStream(stream, device) if isinstance(stream, int) else stream
            with torch.cuda.stream(s):  # freed memory is reused in this stream's order
                workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    (_paged or _paged_calls()).weigh(spec, batch, cache, q_out, lse, workspace, stream)


def attn_paged_select(spec: LayerSpec, batch: PagedBatch, cache: PagedCache, next_pos, n_keep, n_recent, n_moves,
                      src, dst, new_len, stream=None):
    """Which rows each KV head keeps under a budget of n_keep rows, as moves
    (src, dst) of n_moves rows, and the sequences' new lengths."""
    (_paged or _paged_calls()).select(spec, batch, cache, next_pos, n_keep, n_recent, n_moves, src, dst, new_len, stream)


def attn_paged_move(spec: LayerSpec, batch: PagedBatch, cache: PagedCache, n_moves, src, dst, stream=None):
    """Moves the kept rows of attn_paged_select to their new places."""
    (_paged or _paged_calls()).move(spec, batch, cache, n_moves, src, dst, stream)


def cswattn_sync_status(stream=None):
    _check(lib().cswattn_sync_status(_stream(stream)))


def cswattn_set_wait_limit_ns(ns: int) -> int:
    """Sets the device-side wait limit; returns the limit applied (>= 1 ms)."""
    return int(lib().cswattn_set_wait_limit_ns(int(ns)))


def cswattn_set_timing(enable: bool):
    lib().cswattn_set_timing(1 if enable else 0)


def cswattn_kernel_times():
    """{kind: (total_ms, launches)} since the last read, for the kernel kinds."""
    n = len(KERNEL_KINDS)
    ms = (ctypes.c_double * n)()
    cnt = (ctypes.c_int * n)()
    _check(lib().cswattn_kernel_times(ms, cnt))
    return {k: (ms[i], cnt[i]) for i, k in enumerate(KERNEL_KINDS)}


def cswattn_selftest_wait_timeout(limit_ns: int, stream=None):
    """Launch the bounded-wait self-test kernel (its wait always runs out)."""
    _check(lib().cswattn_selftest_wait_timeout(int(limit_ns), _stream(stream)))


def cswattn_version() -> int:
    return int(lib().cswattn_version())


# ------------------------------------------------------------------ convenience

class LayerBuffers:
    """Device buffers of one layer (torch tensors), allocated once and reused."""

    def __init__(self, spec: LayerSpec, device="cuda"):
        import torch
        dt = torch.bfloat16 if spec.dtype == "bf16" else torch.float32
        B, T, H, Hk, D = spec.B, spec.T, spec.n_head, spec.n_kv_head, spec.head_dim
        e = dict(device=device, dtype=dt)
        f = dict(device=device, dtype=torch.float32)
        self.spec = spec
        self.q_out = torch.empty(B, T, H, D, **e)
        self.k_out = torch.empty(B, T, Hk, D, **e)
        self.v_out = torch.empty(B, T, Hk, D, **e)
        self.rstd_q = torch.empty(B, T, H, **f)
        self.rstd_k = torch.empty(B, T, Hk, **f)
        self.O = torch.empty(B, T, H, D, **e)
        self.lse = torch.empty(B, H, T, **f)
        self.dQ = torch.empty(B, T, H, D, **e)
        self.dK = torch.empty(B, T, Hk, D, **e)
        self.dV = torch.empty(B, T, Hk, D, **e)
        self.dve = torch.empty(B, T, Hk, D, **e) if spec.has_ve else None
        self.dgate = torch.empty(B, T, Hk, **e) if spec.has_ve else None
        nbytes = attn_bwd_workspace_bytes(spec)
        self.workspace = torch.empty(max(nbytes, 256), device=device, dtype=torch.uint8)


def layer_forward(spec: LayerSpec, buf: LayerBuffers, q, k, v, ve=None, gate=None, stream=None):
    attn_prologue(spec, q, k, v, ve, gate, buf.q_out, buf.k_out, buf.v_out, buf.rstd_q,
                  buf.rstd_k, stream)
    attn_fwd(spec, buf.q_out, buf.k_out, buf.v_out, buf.O, buf.lse, stream)


def layer_backward(spec: LayerSpec, buf: LayerBuffers, q, k, ve, gate, dO, stream=None):
    attn_bwd(spec, q, k, ve, gate, buf.q_out, buf.k_out, buf.v_out, buf.rstd_q, buf.rstd_k,
             buf.O, buf.lse, dO, buf.dQ, buf.dK, buf.dV, buf.dve, buf.dgate, buf.workspace,
             stream=stream)


# ------------------------------------------------------------------ Muon

def gemm_bf16(A, B, C, alpha=1.0, beta=0.0, D=None, a_mn=False, b_mn=True, stream=None):
    """C = alpha Aop Bop^T + beta D on the tensor cores (see the C header for
    Aop/Bop). Defaults: the plain product of row-major A (M x K), B (K x N)."""
    M, N = C.shape
    K = A.shape[0] if a_mn else A.shape[1]
    _check(lib().cswattn_gemm_bf16(M, N, K, int(a_mn), _ptr(A), A.stride(0), int(b_mn), _ptr(B),
                                   B.stride(0), float(alpha), float(beta), _ptr(D),
                                   D.stride(0) if D is not None else N, _ptr(C), C.stride(0),
                                   _stream(stream)))


def muon_ns_workspace_bytes(m: int, n: int) -> int:
    return int(lib().muon_ns_workspace_bytes(m, n))


def muon_newton_schulz(X, Y, coeffs, workspace, stream=None):
    """Muon's Newton-Schulz iteration, one step per (a, b, c) triple, from the
    bf16 m x n matrix X into Y (see the C header)."""
    m, n = X.shape
    flat = [float(v) for t in coeffs for v in t]
    arr = (ctypes.c_float * len(flat))(*flat)
    _check(lib().muon_newton_schulz(m, n, arr, len(coeffs), _ptr(X), _ptr(Y), _ptr(workspace),
                                    workspace.numel() * workspace.element_size(), _stream(stream)))
