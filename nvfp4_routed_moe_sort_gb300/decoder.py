"""The operators around the routed experts in a decoder layer, on torch tensors.

``add_rms_norm`` (moe_add_rmsnorm), ``fp4_linear`` / ``NVFP4Linear`` (moe_linear_fp4) and
``NVFP4KVCache`` (moe_kv_append, moe_kv_attend). They check what the C entry points cannot see
(types, shapes, strides), run on torch's current stream and allocate only the results that the
caller did not bring.
"""
from __future__ import annotations

import threading

import torch

from . import _lib as L
from .moe import quantize_weights

_FP8 = {None: L.MOE_FP8_NONE, "token": L.MOE_FP8_PER_TOKEN, "group": L.MOE_FP8_PER_GROUP}
_BF16, _E4M3, _F32, _U8 = torch.bfloat16, torch.float8_e4m3fn, torch.float32, torch.uint8


def _need(cond, what: str):
    if not cond:
        raise ValueError(what)


def _dense(t, dtype, shape, what: str):
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {tuple(shape)} on the GPU")


def _rows(t, dtype, shape, what: str):
    """t: rows of `shape` whose values lie side by side (any row stride)."""
    if t.dtype is not dtype or t.shape != shape or not t.is_cuda or (t.stride(1) != 1 and shape[1] != 1):
        raise ValueError(f"{what} must be {dtype} rows of shape {tuple(shape)} on the GPU, their values side by side")


_scratch: dict = {}


def _workspace(nbytes: int, device) -> torch.Tensor | None:
    """Scratch of one call. Outside graph capture it is kept for the next call of the same host thread on
    the same stream, which runs after this one (a fresh tensor costs 5 us of host time a call)."""
    if nbytes == 0:
        return None
    if torch.cuda.is_current_stream_capturing():
        return torch.empty(nbytes, dtype=_U8, device=device)
    key = device, L.current_stream(), threading.get_ident()
    t = _scratch.get(key)
    if t is None or t.numel() < nbytes:
        t = _scratch[key] = torch.empty(nbytes, dtype=_U8, device=device)
    return t


def add_rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, eps: float = 1e-6,
                 fp8: str | None = None, out: tuple | None = None):
    """RMS norm of x [M, H] bf16, or of x + residual: (y, residual_out, y8, y8_scale).

    y [M, H] bf16; residual_out [M, H] bf16 = x + residual (None without a residual); with
    fp8 = "token" or "group" also y8 [M, H] float8_e4m3fn and its scales, f32 [M, 1] or
    [M, ceil(H / 128)] (None otherwise). ``out``: the four results' own tensors (None in a
    place: that one is not written, for y and residual_out); residual_out may be ``residual``.
    """
    if fp8 not in _FP8:
        raise ValueError('fp8 must be None, "token" or "group"')
    _need(x.dim() == 2, "x must be [M, H]")
    M, H = shape = x.shape
    _rows(x, _BF16, shape, "x")
    _dense(weight, _BF16, (H,), "weight")
    if residual is not None:
        _rows(residual, _BF16, shape, "residual")
    groups = 1 if fp8 == "token" else -(-H // L.MOE_FP8_GROUP)
    if out is None:
        dev = x.device
        y = torch.empty(M, H, dtype=_BF16, device=dev)
        r = torch.empty(M, H, dtype=_BF16, device=dev) if residual is not None else None
        y8 = torch.empty(M, H, dtype=_E4M3, device=dev) if fp8 else None
        sc = torch.empty(M, groups, dtype=_F32, device=dev) if fp8 else None
    else:
        y, r, y8, sc = out
        if y is not None:
            _dense(y, _BF16, shape, "out[0]")
        if r is not None:
            _dense(r, _BF16, shape, "out[1]")
        _need((y8 is None) == (fp8 is None) and (sc is None) == (fp8 is None), "out[2] and out[3] go with fp8")
        if y8 is not None:
            _dense(y8, _E4M3, shape, "out[2]")
            _dense(sc, _F32, (M, groups), "out[3]")
    L.moe_add_rmsnorm(x, residual, weight, eps, _FP8[fp8], y, r, y8, sc)
    return y, r, y8, sc


def fp4_linear(x: torch.Tensor, w: torch.Tensor, w_sf: torch.Tensor, alpha: torch.Tensor,
               activation: str = "identity", x_scale: torch.Tensor | None = None, out: torch.Tensor | None = None):
    """act(x W^T) of a few tokens with one NVFP4 matrix: w [N, K/2] u8, w_sf [N, K/16] u8, alpha f32 [1].

    x [M, K]: bf16, or float8_e4m3fn with x_scale f32 [M, 1] or [M, ceil(K / 128)] (as add_rms_norm
    gives them). Gated activations take w rows [gate; up]. Returns [M, N] (gated: [M, N / 2]) bf16.
    """
    act = L.ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation must be one of {sorted(L.ACTIVATIONS)}")
    _need(x.dim() == 2 and w.dim() == 2, "x must be [M, K] and w [N, K/2]")
    M, K = shape = x.shape
    N = w.shape[0]
    _dense(w, _U8, (N, K // 2), "w")
    _dense(w_sf, _U8, (N, K // 16), "w_sf")
    _need(alpha.dtype is _F32 and alpha.numel() == 1 and alpha.is_cuda, "alpha must be one float32 value on the GPU")
    mode = L.MOE_FP8_NONE
    if x_scale is None:
        _rows(x, _BF16, shape, "x without x_scale")
    else:
        _rows(x, _E4M3, shape, "x with x_scale")
        groups = -(-K // L.MOE_FP8_GROUP)
        mode = L.MOE_FP8_PER_TOKEN if x_scale.shape[-1] == 1 else L.MOE_FP8_PER_GROUP
        _dense(x_scale, _F32, (M, 1 if mode == L.MOE_FP8_PER_TOKEN else groups), "x_scale")
    if act == L.MOE_ACT_SWIGLU or act == L.MOE_ACT_GEGLU:
        _need(N % 2 == 0, "a gated activation needs an even number of rows in w")
        N //= 2
    if out is None:
        out = torch.empty(M, N, dtype=_BF16, device=x.device)
    else:
        _dense(out, _BF16, (M, N), "out")
    L.moe_linear_fp4(x, x_scale, mode, w, w_sf, alpha, act, out)
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
    encode scales. dev_status: an int32 tensor whose first element collects MOE_DEV_* bits.
    """

    def __init__(self, k, k_sf, v, v_sf, k_scale: float = 1.0, v_scale: float = 1.0, dev_status=None):
        _need(k.dim() == 4, "k must be [num_pages, num_kv_heads, page_size, head_dim/2]")
        P, Hkv, ps, half = data = k.shape
        sf = (P, Hkv, ps, half // 8)
        inner, inner_sf = (ps * half, half, 1), (ps * (half // 8), half // 8, 1)
        if not (k.dtype is v.dtype is k_sf.dtype is v_sf.dtype is _U8 and v.shape == data and k_sf.shape == sf
                and v_sf.shape == sf and k.stride() == v.stride() and k_sf.stride() == v_sf.stride()
                and k.stride()[1:] == inner and k_sf.stride()[1:] == inner_sf):
            raise ValueError("k, v must be u8 [num_pages, num_kv_heads, page_size, head_dim/2] and k_sf, v_sf "
                             "[..., head_dim/16], each page contiguous, with the same strides for keys and values")
        _need(k.is_cuda and v.is_cuda and k_sf.is_cuda and v_sf.is_cuda
              and (dev_status is None or (dev_status.is_cuda and dev_status.dtype is torch.int32)),
              "the cache and dev_status (int32) must be on the GPU")
        self.k, self.k_sf, self.v, self.v_sf, self.dev_status = k, k_sf, v, v_sf, dev_status
        self.num_kv_heads, self.page_size, self.head_dim = Hkv, ps, 2 * half
        self.c = L.KVCacheT(k.data_ptr(), k_sf.data_ptr(), v.data_ptr(), v_sf.data_ptr(), P, ps, Hkv, 2 * half,
                            k.stride(0), k_sf.stride(0), k_scale, v_scale)

    @classmethod
    def allocate(cls, num_pages: int, page_size: int, num_kv_heads: int, head_dim: int, device="cuda",
                 k_scale: float = 1.0, v_scale: float = 1.0) -> "NVFP4KVCache":
        k, v = (torch.zeros(num_pages, num_kv_heads, page_size, head_dim // 2, dtype=_U8, device=device) for _ in "kv")
        k_sf, v_sf = (torch.zeros(num_pages, num_kv_heads, page_size, head_dim // 16, dtype=_U8, device=device)
                      for _ in "kv")
        return cls(k, k_sf, v, v_sf, k_scale, v_scale, torch.zeros(4, dtype=torch.int32, device=device))

    def _tokens(self, t, N, what):
        D = self.head_dim
        if t.dtype is not _BF16 or t.shape != (N, self.num_kv_heads, D) or t.stride()[1:] != (D, 1):
            raise ValueError(f"{what} must be bf16 [N, num_kv_heads, head_dim], each token's values contiguous")
        _need(t.is_cuda, f"{what} must be on the GPU")

    def append(self, k_new, v_new, slots, seen: tuple | None = None):
        """Store N tokens' keys and values [N, num_kv_heads, head_dim] bf16 at slots [N] int64 (page *
        page_size + place; negative: not stored). seen: two bf16 tensors of the same shape that get
        what the cache then holds for the tokens."""
        N = k_new.shape[0]
        self._tokens(k_new, N, "k_new")
        self._tokens(v_new, N, "v_new")
        _dense(slots, torch.int64, (N,), "slots")
        k_seen = v_seen = None
        if seen is not None:
            k_seen, v_seen = seen
            _dense(k_seen, _BF16, k_new.shape, "seen[0]")
            _dense(v_seen, _BF16, k_new.shape, "seen[1]")
        L.moe_kv_append(self.c, k_new, v_new, slots, k_seen, v_seen, self.dev_status)

    def attend(self, q, page_table, seq_lens, softmax_scale: float | None = None, out=None, lse=None, workspace=None):
        """Attention of q [batch, q_len, num_q_heads, head_dim] bf16 over the sequences in
        page_table [batch, max_pages] int32 and seq_lens [batch] int32 (new tokens included): (out, lse),
        out like q and contiguous, lse f32 [batch, q_len, num_q_heads]."""
        _need(q.dim() == 4, "q must be [batch, q_len, num_q_heads, head_dim]")
        B, T, Hq, D = shape = q.shape
        sb, st, sh, sd = q.stride()
        ld = st if T > 1 else sb
        if q.dtype is not _BF16 or D != self.head_dim or sd != 1 or sh != D or (B > 1 and sb != T * ld):
            raise ValueError("q must be bf16 [batch, q_len, num_q_heads, head_dim] with evenly spaced rows")
        if page_table.dtype is not torch.int32 or page_table.dim() != 2 or page_table.shape[0] != B \
                or (page_table.stride(1) != 1 and page_table.shape[1] > 1):
            raise ValueError("page_table must be int32 [batch, max_pages]")
        _need(q.is_cuda and page_table.is_cuda, "q and page_table must be on the GPU")
        _dense(seq_lens, torch.int32, (B,), "seq_lens")
        if out is None:
            out = torch.empty(shape, dtype=_BF16, device=q.device)
        else:
            _dense(out, _BF16, shape, "out")
        if lse is None:
            lse = torch.empty(B, T, Hq, dtype=_F32, device=q.device)
        else:
            _dense(lse, _F32, (B, T, Hq), "lse")
        if workspace is None:
            workspace = _workspace(L.moe_kv_attend_workspace_bytes(self.c, B, T, Hq, page_table.shape[1]), q.device)
        L.moe_kv_attend(self.c, q, ld, page_table, seq_lens, D ** -0.5 if softmax_scale is None else softmax_scale,
                        out, lse, workspace, self.dev_status)
        return out, lse
