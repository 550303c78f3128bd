"""The operators around the routed experts in a decoder layer, on torch tensors.

``add_rms_norm`` (moe_add_rmsnorm), ``fp4_linear`` / ``NVFP4Linear`` (moe_linear_fp4) and
``NVFP4KVCache`` (moe_kv_append, moe_kv_attend). The calls go through the native module
``_native`` (csrc/binding/native.cpp), which checks types, shapes, strides and device; they run on
torch's current stream, and only results that the caller did not bring are allocated.
"""
from __future__ import annotations

import threading
from operator import attrgetter

import torch

from . import _lib as L
from .moe import quantize_weights

_FP8 = {None: L.MOE_FP8_NONE, "token": L.MOE_FP8_PER_TOKEN, "group": L.MOE_FP8_PER_GROUP}
_BF16, _E4M3, _F32, _U8 = torch.bfloat16, torch.float8_e4m3fn, torch.float32, torch.uint8
_GATED = (L.MOE_ACT_SWIGLU, L.MOE_ACT_GEGLU)

_native = None


def _load():
    """The native module; raises if it has not been built."""
    global _native
    L.lib()
    try:
        from . import _native as native
    except ImportError as e:
        raise L.MoEError(f"the _native module is missing: build it first (nvfp4_routed_moe_sort_gb300.build): {e}") from e
    native.set_error(L.MoEError)
    _native = native
    return native


_scratch = threading.local()  # .of: (device, stream id) -> tensor; goes with its thread
_MOST_STREAMS = 8


def _workspace(nbytes: int, device) -> torch.Tensor | None:
    """Scratch of one call. Outside graph capture it is kept for the next call of the same host thread on
    the same stream, which runs after this one (a fresh tensor costs 5 us of host time a call)."""
    if nbytes == 0:
        return None
    if torch.cuda.is_current_stream_capturing():
        return torch.empty(nbytes, dtype=_U8, device=device)
    kept = _scratch.__dict__.setdefault("of", {})
    key = device, _native.stream_id()  # a handle may come back for another stream, an id does not
    t = kept.get(key)
    if t is None or t.numel() < nbytes:
        if t is None and len(kept) >= _MOST_STREAMS:
            kept.clear()
        t = kept[key] = torch.empty(nbytes, dtype=_U8, device=device)
    return t


def add_rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, eps: float = 1e-6,
                 fp8: str | None = None, out: tuple | None = None):
    """RMS norm of x [M, H] bf16, or of x + residual: (y, residual_out, y8, y8_scale).

    y [M, H] bf16; residual_out [M, H] bf16 = x + residual (None without a residual); with
    fp8 = "token" or "group" also y8 [M, H] float8_e4m3fn and its scales, f32 [M, 1] or
    [M, ceil(H / 128)] (None otherwise). x and residual may have a row stride. ``out``: the four
    results' own tensors (None in a place: that one is not written, for y and residual_out);
    residual_out may be ``residual``.
    """
    mode = _FP8.get(fp8)
    if mode is None:
        raise ValueError('fp8 must be None, "token" or "group"')
    if out is None:
        if x.dim() != 2:
            raise ValueError("x must be [M, H]")
        (M, H), dev = x.shape, x.device
        out = (torch.empty(M, H, dtype=_BF16, device=dev),
               torch.empty(M, H, dtype=_BF16, device=dev) if residual is not None else None,
               torch.empty(M, H, dtype=_E4M3, device=dev) if fp8 else None,
               torch.empty(M, 1 if fp8 == "token" else -(-H // L.MOE_FP8_GROUP), dtype=_F32, device=dev) if fp8 else None)
    y, r, y8, scale = out
    (_native or _load()).add_rms_norm(x, weight, residual, eps, mode, y, r, y8, scale)
    return y, r, y8, scale


def fp4_linear(x: torch.Tensor, w: torch.Tensor, w_sf: torch.Tensor, alpha: torch.Tensor,
               activation: str = "identity", x_scale: torch.Tensor | None = None, out: torch.Tensor | None = None):
    """act(x W^T) of a few tokens with one NVFP4 matrix: w [N, K/2] u8, w_sf [N, K/16] u8, alpha f32 [1].

    x [M, K]: bf16, or float8_e4m3fn with x_scale f32 [M, 1] or [M, ceil(K / 128)] (as add_rms_norm
    gives them); it may have a row stride. Gated activations take w rows [gate; up]. Returns [M, N]
    (gated: [M, N / 2]) bf16. alpha may be an element of a longer tensor; one that is not 16-byte aligned
    is copied in every call.
    """
    act = L.ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation must be one of {sorted(L.ACTIVATIONS)}")
    if out is None:
        out = torch.empty(x.shape[0], w.shape[0] // 2 if act in _GATED else w.shape[0], dtype=_BF16, device=x.device)
    (_native or _load()).fp4_linear(x, x_scale, w, w_sf, alpha, act, out)
    return out


class NVFP4Linear:
    """One dense NVFP4 matrix: a projection, a shared expert's matrix, an output head."""

    def __init__(self, w: torch.Tensor, w_sf: torch.Tensor, alpha: torch.Tensor, activation: str = "identity"):
        self.w, self.w_sf, self.alpha, self.activation = w, w_sf, alpha, activation

    @classmethod
    def from_bf16(cls, w: torch.Tensor, activation: str = "identity") -> "NVFP4Linear":
        """Encodes w [N, K] bf16 (K % 128 == 0) with moe_quantize_weights."""
        data, sf, alpha = quantize_weights(w.unsqueeze(0))
        return cls(data[0], sf[0], alpha, activation)

    def __call__(self, x, x_scale=None, out=None):
        return fp4_linear(x, self.w, self.w_sf, self.alpha, self.activation, x_scale, out)


class NVFP4KVCache:
    """A paged key/value cache in NVFP4 on the GPU (moe_kv_cache_t).

    k, v [num_pages, num_kv_heads, page_size, head_dim/2] u8; k_sf, v_sf [..., head_dim/16] u8;
    the pages of k and v (of k_sf and v_sf) have the same stride. k_scale, v_scale: static FP32
    encode scales. dev_status: an int32 tensor whose first element collects MOE_DEV_* bits. All of
    them stay what they are: other pages or scales are another cache.
    """

    k, k_sf, v, v_sf, k_scale, v_scale, dev_status = (
        property(attrgetter("_" + name)) for name in ("k", "k_sf", "v", "v_sf", "k_scale", "v_scale", "dev_status"))

    def __init__(self, k, k_sf, v, v_sf, k_scale: float = 1.0, v_scale: float = 1.0, dev_status=None):
        # holds the tensors' addresses, so the tensors are held beside it and never exchanged
        self._native = (_native or _load()).kv_cache(k, k_sf, v, v_sf, k_scale, v_scale, dev_status)
        self._k, self._k_sf, self._v, self._v_sf, self._dev_status = k, k_sf, v, v_sf, dev_status
        self._k_scale, self._v_scale = k_scale, v_scale

    @classmethod
    def allocate(cls, num_pages: int, page_size: int, num_kv_heads: int, head_dim: int, device="cuda",
                 k_scale: float = 1.0, v_scale: float = 1.0) -> "NVFP4KVCache":
        k, v = (torch.zeros(num_pages, num_kv_heads, page_size, head_dim // 2, dtype=_U8, device=device) for _ in "kv")
        k_sf, v_sf = (torch.zeros(num_pages, num_kv_heads, page_size, head_dim // 16, dtype=_U8, device=device)
                      for _ in "kv")
        return cls(k, k_sf, v, v_sf, k_scale, v_scale, torch.zeros(4, dtype=torch.int32, device=device))

    @property
    def c(self) -> L.KVCacheT:
        """The cache as the C entry points take it."""
        P, Hkv, ps, half = self.k.shape
        return L.KVCacheT(self.k.data_ptr(), self.k_sf.data_ptr(), self.v.data_ptr(), self.v_sf.data_ptr(), P, ps, Hkv,
                          2 * half, self.k.stride(0), self.k_sf.stride(0), self.k_scale, self.v_scale)

    def append(self, k_new, v_new, slots, seen: tuple | None = None):
        """Store N tokens' keys and values [N, num_kv_heads, head_dim] bf16 (a token stride is fine) at slots
        [N] int64 (page * page_size + place; negative: not stored). seen: two bf16 tensors of the same
        shape that get what the cache then holds for the tokens."""
        k_seen, v_seen = seen if seen is not None else (None, None)
        _native.kv_append(self._native, k_new, v_new, slots, k_seen, v_seen)

    def attend(self, q, page_table, seq_lens, softmax_scale: float | None = None, out=None, lse=None, workspace=None):
        """Attention of q [batch, q_len, num_q_heads, head_dim] bf16 (evenly spaced rows) over the sequences
        in page_table [batch, max_pages] int32 and seq_lens [batch] int32 (new tokens included): (out, lse),
        out like q and contiguous, lse f32 [batch, q_len, num_q_heads]."""
        if workspace is None:
            n = _native.kv_workspace(self._native, q, page_table)
            workspace = _workspace(n, q.device) if n else None
        if out is None:
            out = torch.empty(q.shape, dtype=_BF16, device=q.device)
        if lse is None:
            lse = torch.empty(q.shape[:3], dtype=_F32, device=q.device)
        if softmax_scale is None:
            softmax_scale = q.shape[3] ** -0.5
        _native.kv_attend(self._native, q, page_table, seq_lens, softmax_scale, out, lse, workspace)
        return out, lse
