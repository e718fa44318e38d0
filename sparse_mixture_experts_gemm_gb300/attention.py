"""The operators of a full-attention layer, over torch tensors.

Thin functions over the C ABI (include/moe.h: moe_qk_norm_rope,
moe_attention_prefill, moe_kv_write, moe_kv_read, moe_attention_decode), in the
manner of mixer.py: they check types, shapes and layouts, allocate what is not
given, and launch on `stream` (default: torch's current stream) of the current
device.  Tokens may be strided (slices of a fused projection).

A cache is a pair of tensors (codes, affine) from kv_cache; pages of it are given
out by the caller, in an int32 table [n][width] of page numbers per sequence.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import MoeError
from .mixer import _BF16, _device, _given, _lib, _on, _tokens, _vector

PAGE = 64   # tokens per page of a cache
GROUP = 64  # columns that share a scale and a bias

_I32 = torch.int32


def _check(rc, where):
    if rc:
        raise MoeError(rc, where)


def _heads(name, t):
    """(tokens, heads, width) of [..., heads, width]"""
    if t.dim() not in (2, 3, 4):
        raise ValueError(f"{name} must be [..., heads, head_dim]")
    shape = t.shape
    H, w = shape[-2], shape[-1]
    if H * w == 0:
        raise ValueError(f"{name} must have heads and columns")
    return t.numel() // (H * w), H, w


def _stride(name, t, H, w):
    """Token stride; a single token's [heads][width] counts as one of many."""
    return _tokens(name, t if t.dim() > 2 else t.unsqueeze(0), H, w)


def _offsets(name, t):
    if t.dtype != _I32 or t.dim() != 1 or not t.is_contiguous() or not t.is_cuda or t.shape[0] < 1:
        raise ValueError(f"{name} must be a contiguous CUDA int32 tensor [n + 1]")
    return t.shape[0] - 1, t.data_ptr()


def _empty(t):
    """An output of t's shape, contiguous."""
    return torch.empty_like(t) if t.is_contiguous() else torch.empty(t.shape, dtype=_BF16, device=t.device)


def qk_norm_rope(q, k, q_weight, k_weight, positions, inv_freq, eps=1e-6, q_out=None, k_out=None,
                 stream=None):
    """moe_qk_norm_rope: norm of every head's row of q [..., H_q, D] and
    k [..., H_k, D] (bf16) and the rotation of its first 2 len(inv_freq) columns
    by the token's position.  positions: int32 of q's leading shape; inv_freq:
    float64 [R / 2], radians per position (None: no rotation, positions unused).
    Returns (q, k); q_out may be q and k_out may be k."""
    N, Hq, D = _heads("q", q)
    Hk = k.shape[-2] if k.dim() > 1 else 0
    lead = q.shape[:-2]
    if Hk == 0 or k.shape[-1] != D or k.shape[:-2] != lead:
        raise ValueError("shapes of q and k do not agree")
    qs, ks = _stride("q", q, Hq, D), _stride("k", k, Hk, D)
    _vector("q_weight", q_weight, D, _BF16)
    _vector("k_weight", k_weight, D, _BF16)
    rot, pp, fp = 0, None, None
    if inv_freq is not None:
        _vector("inv_freq", inv_freq, inv_freq.numel(), torch.float64)
        rot = 2 * inv_freq.shape[0]
        if rot:
            _given("positions", positions, lead, _I32)
            pp, fp = positions.data_ptr(), inv_freq.data_ptr()
    ctx, handle = _on(stream, _device(q, k, q_weight, k_weight, positions, inv_freq, q_out, k_out))
    qos, kos = Hq * D, Hk * D
    with ctx:
        if q_out is None:
            q_out = _empty(q)
        elif q_out.shape != q.shape:
            raise ValueError("q_out must have the shape of q")
        else:
            qos = _stride("q_out", q_out, Hq, D)
        if k_out is None:
            k_out = _empty(k)
        elif k_out.shape != k.shape:
            raise ValueError("k_out must have the shape of k")
        else:
            kos = _stride("k_out", k_out, Hk, D)
    _check(_lib().moe_qk_norm_rope(q.data_ptr(), k.data_ptr(), q_weight.data_ptr(), k_weight.data_ptr(), pp, fp,
                                   N, Hq, Hk, D, rot, qs, ks, eps, q_out.data_ptr(), qos, k_out.data_ptr(), kos,
                                   handle), "moe_qk_norm_rope")
    return q_out, k_out


@functools.lru_cache(maxsize=1024)
def _prefill_workspace(N, M, n, Hq, Hk, D):
    """Bytes that moe_attention_prefill wants for these sizes."""
    need = ctypes.c_size_t(0)
    _check(_lib().moe_attention_prefill_workspace(N, M, n, Hq, Hk, D, ctypes.byref(need)),
           "moe_attention_prefill_workspace")
    return need.value


def attention_prefill(q, k, v, offsets=None, k_offsets=None, scale=None, out=None, stream=None):
    """moe_attention_prefill: causal attention of q bf16 [n][T][H_q][D] over
    k, v bf16 [n][M][H_kv][D] (n sequences, the queries being the last of the keys),
    or of packed q [N][H_q][D] over k, v [M][H_kv][D] with offsets (int32 [n + 1]
    on the GPU; one sequence without them) and k_offsets (None: those of q).
    scale: D ** -0.5 unless given.  Returns bf16 of q's shape."""
    dims = q.dim()
    if dims not in (3, 4) or k.dim() != dims or v.shape != k.shape or q.shape[-1] != k.shape[-1] \
            or (dims == 4 and q.shape[0] != k.shape[0]):
        raise ValueError("shapes of q, k, v do not agree")
    N, Hq, D = _heads("q", q)
    M, Hk, _ = _heads("k", k)
    op = kp = None
    if dims == 4:
        if offsets is not None or k_offsets is not None:
            raise ValueError("offsets go with packed tokens [N][H][D]")
        n = q.shape[0]
    elif offsets is None:
        if k_offsets is not None:
            raise ValueError("k_offsets go with offsets")
        n = 1
    else:
        n, op = _offsets("offsets", offsets)
        if k_offsets is not None:
            nk, kp = _offsets("k_offsets", k_offsets)
            if nk != n:
                raise ValueError("offsets and k_offsets must be of one length")
        elif N != M:
            raise ValueError("k and v must have q's tokens where there are no k_offsets")
    qs, ks, vs = _tokens("q", q, Hq, D), _tokens("k", k, Hk, D), _tokens("v", v, Hk, D)
    ctx, handle = _on(stream, _device(q, k, v, offsets, k_offsets, out))
    need, wp = _prefill_workspace(N, M, n, Hq, Hk, D), None
    with ctx:
        if out is None:
            out = _empty(q)
        else:
            _given("out", out, q.shape, _BF16)
        if need:
            ws = torch.empty(need, dtype=torch.uint8, device=q.device)
            wp = ws.data_ptr()
    _check(_lib().moe_attention_prefill(q.data_ptr(), k.data_ptr(), v.data_ptr(), op, kp, N, M, n, Hq, Hk, D, qs,
                                        ks, vs, D ** -0.5 if scale is None else scale, out.data_ptr(), wp, need,
                                        handle), "moe_attention_prefill")
    return out


def kv_cache(pages, heads, head_dim, device="cuda"):
    """The two tensors of a 4-bit cache of so many pages of 64 tokens, zeroed:
    codes uint8 [pages][2][heads][64][head_dim / 2], affine bf16
    [pages][2][heads][64][head_dim / 64][2]."""
    return (torch.zeros(pages, 2, heads, PAGE, head_dim // 2, dtype=torch.uint8, device=device),
            torch.zeros(pages, 2, heads, PAGE, head_dim // GROUP, 2, dtype=_BF16, device=device))


def _cache(cache):
    """(codes, affine, pages, heads, head_dim)"""
    codes, affine = cache
    shape = codes.shape
    if len(shape) != 5 or shape[1] != 2 or shape[3] != PAGE or codes.dtype != torch.uint8 \
            or not codes.is_contiguous() or not codes.is_cuda:
        raise ValueError("codes must be a contiguous CUDA uint8 tensor [pages][2][heads][64][head_dim / 2]")
    P, _, H, _, half = shape
    _given("affine", affine, (P, 2, H, PAGE, 2 * half // GROUP, 2), _BF16)
    return codes, affine, P, H, 2 * half


def _table(pages):
    if pages.dtype != _I32 or pages.dim() != 2 or not pages.is_contiguous() or not pages.is_cuda:
        raise ValueError("pages must be a contiguous CUDA int32 tensor [n][width]")
    return pages.shape


def kv_cache_write(cache, k, v, pages, starts=None, offsets=None, stream=None):
    """moe_kv_write: k, v bf16 [n][T][H][D], or packed [N][H][D] with offsets (int32
    [n + 1]; one sequence without them), quantised into the pages of each sequence
    from position starts[i] on (int32 [n]; None: 0)."""
    codes, affine, P, H, D = _cache(cache)
    n, width = _table(pages)
    dims = k.dim()
    shape = k.shape
    if dims not in (3, 4) or shape != v.shape or shape[-2] != H or shape[-1] != D:
        raise ValueError("k and v must be [n][T][H][D] or [N][H][D] with the cache's heads")
    N, op = shape[0] if dims == 3 else shape[0] * shape[1], None
    if dims == 4:
        if offsets is not None:
            raise ValueError("offsets go with packed tokens [N][H][D]")
        m = shape[0]
    elif offsets is None:
        m = 1
    else:
        m, op = _offsets("offsets", offsets)
    if m != n:
        raise ValueError("pages must have a row per sequence")
    if starts is not None:
        _vector("starts", starts, n, _I32)
    ks, vs = _tokens("k", k, H, D), _tokens("v", v, H, D)
    _, handle = _on(stream, _device(k, v, codes, affine, pages, starts, offsets))
    _check(_lib().moe_kv_write(codes.data_ptr(), affine.data_ptr(), P, k.data_ptr(), v.data_ptr(),
                               pages.data_ptr(), width, None if starts is None else starts.data_ptr(), op, N, n,
                               H, D, ks, vs, handle), "moe_kv_write")


def kv_cache_read(cache, pages, offsets, tokens, starts=None, k_out=None, v_out=None, stream=None):
    """moe_kv_read: sequence i's positions starts[i], .. (None: from 0) as the rows
    offsets[i] .. offsets[i + 1] - 1 of two bf16 tensors [tokens][H][D], returned.
    Rows of no sequence keep what a given k_out and v_out held."""
    codes, affine, P, H, D = _cache(cache)
    n, width = _table(pages)
    m, op = _offsets("offsets", offsets)
    if m != n:
        raise ValueError("pages must have a row per sequence")
    if starts is not None:
        _vector("starts", starts, n, _I32)
    ctx, handle = _on(stream, _device(codes, affine, pages, starts, offsets, k_out, v_out))
    shape = (tokens, H, D)
    with ctx:
        if k_out is None:
            k_out = torch.empty(shape, dtype=_BF16, device=codes.device)
        else:
            _given("k_out", k_out, shape, _BF16)
        if v_out is None:
            v_out = torch.empty_like(k_out)
        else:
            _given("v_out", v_out, shape, _BF16)
    _check(_lib().moe_kv_read(codes.data_ptr(), affine.data_ptr(), P, pages.data_ptr(), width,
                              None if starts is None else starts.data_ptr(), op, tokens, n, H, D,
                              k_out.data_ptr(), v_out.data_ptr(), handle), "moe_kv_read")
    return k_out, v_out


@functools.lru_cache(maxsize=1024)
def _decode_workspace(n, width, Hq, Hk, D):
    """Bytes that moe_attention_decode wants for these sizes."""
    need = ctypes.c_size_t(0)
    _check(_lib().moe_attention_decode_workspace(n, width, Hq, Hk, D, ctypes.byref(need)),
           "moe_attention_decode_workspace")
    return need.value


def attention_decode(q, cache, pages, lengths, scale=None, out=None, stream=None):
    """moe_attention_decode: attention of one query token per sequence, q bf16
    [n][H_q][D], over the first lengths[i] (int32 [n]) tokens of each sequence in
    the cache.  scale: D ** -0.5 unless given.  Returns bf16 of q's shape."""
    codes, affine, P, H, D = _cache(cache)
    n, width = _table(pages)
    shape = q.shape
    if len(shape) != 3 or shape[0] != n or shape[2] != D or shape[1] == 0:
        raise ValueError("q must be [n][H_q][D] with a row of pages per sequence and the cache's columns")
    Hq = shape[1]
    qs = _tokens("q", q, Hq, D)
    _vector("lengths", lengths, n, _I32)
    need = _decode_workspace(n, width, Hq, H, D)
    ctx, handle = _on(stream, _device(q, codes, affine, pages, lengths, out))
    with ctx:
        if out is None:
            out = _empty(q)
        else:
            _given("out", out, q.shape, _BF16)
        ws = torch.empty(need, dtype=torch.uint8, device=q.device) if need else None
    _check(_lib().moe_attention_decode(q.data_ptr(), qs, codes.data_ptr(), affine.data_ptr(), P, pages.data_ptr(),
                                       width, lengths.data_ptr(), n, Hq, H, D,
                                       D ** -0.5 if scale is None else scale, out.data_ptr(),
                                       None if ws is None else ws.data_ptr(), need, handle), "moe_attention_decode")
    return out
