"""The operators around a linear-attention mixer, over torch tensors.

Thin functions over the C ABI (include/moe.h: moe_add_rmsnorm,
moe_add_rmsnorm_fp8, moe_quantize_fp8, moe_matmul_fp8; include/gdn.h:
gdn_decay_scan): they check types, shapes and layouts, allocate what is not
given, and launch on `stream` (default: torch's current stream).  Results and
workspaces are allocated on that stream, so that the caching allocator hands
their memory on in its order.  The kernels run on the current device: tensors
or a stream of another one are refused.

One decoded token is a handful of such calls of a few microseconds each, so
the path of a call with contiguous tensors on the current stream is kept short:
torch's raw stream handle, no context managers, one size query per shape.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools

import torch

from . import MOE_BF16, MOE_F32, MoeError, lib

_BF16, _F32, _F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
_DTYPES = {_BF16: MOE_BF16, _F32: MOE_F32}
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_gpus = 0  # how many there are, once known
_NONE = contextlib.nullcontext()
_L = None


def _lib():
    global _L
    if _L is None:
        _L = lib()
    return _L


def _on(stream, device):
    """(context to allocate in, raw handle) of a caller's stream on `device`;
    None: the current one."""
    if stream is None:
        return _NONE, _raw_stream(device)
    if isinstance(stream, int):
        return torch.cuda.stream(torch.cuda.ExternalStream(stream)), stream
    if stream.device_index != device:
        raise ValueError(f"stream is on device {stream.device_index}, the tensors on {device}")
    return torch.cuda.stream(stream), stream.cuda_stream


def _device(first, *others):
    """The device of all these CUDA tensors (None: not given), which has to be
    the current one.  (Where there is one GPU it is that: asking every tensor
    costs a call 1 to 2 us.)"""
    global _gpus
    if _gpus == 1:
        return 0
    if not _gpus:
        _gpus = torch.cuda.device_count()
    device = first.get_device()
    for t in others:
        if t is not None and t.get_device() != device:
            raise ValueError(f"tensors on device {device} and on device {t.get_device()} in one call")
    if device != _current_device():
        raise ValueError(f"tensors on device {device}, current device {_current_device()}")
    return device


def _rows(name, t):
    """(rows, width, row stride in elements) of a tensor whose last dimension
    is contiguous and whose leading ones are evenly spaced rows."""
    shape = t.shape
    if not shape:
        raise ValueError(f"{name} must have at least one dimension")
    d = shape[-1]
    if t.is_contiguous():
        return (t.numel() // d if d else 0), d, d
    strides = t.stride()
    if strides[-1] != 1 and d > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    rows = t.numel() // d if d else 0
    step, stride = None, d
    for n, s in zip(reversed(shape[:-1]), reversed(strides[:-1])):
        if n == 1:
            continue
        if step is None:
            step, stride = s, s
        elif s != step:
            raise ValueError(f"{name}: rows must be evenly spaced")
        step *= n
    return rows, d, max(stride, d) if rows <= 1 else stride


def _vector(name, t, n, dtype):
    if t.dtype != dtype or not t.is_cuda or t.dim() != 1 or t.shape[0] != n \
            or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor [{n}]")


def _given(name, t, shape, dtype):
    """A caller's tensor of this shape and type, contiguous, on the GPU."""
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor of shape {tuple(shape)}")


def _norm(x, weight, residual, eps, out, scales, sum_out, stream, fp8):
    dtype = x.dtype
    dt = _DTYPES.get(dtype)
    if dt is None or not x.is_cuda:
        raise ValueError("x must be a CUDA bfloat16 or float32 tensor")
    rows, d, xs = _rows("x", x)
    _vector("weight", weight, d, dtype)
    rs, rp = d, None
    if residual is not None:
        if residual.dtype != dtype or not residual.is_cuda or residual.shape != x.shape:
            raise ValueError("residual must be a CUDA tensor of x's shape and type")
        _, _, rs = _rows("residual", residual)
        rp = residual.data_ptr()
    ctx, handle = _on(stream, _device(x, weight, residual, out, scales, sum_out))
    kind = _F8 if fp8 else dtype
    with ctx:
        plain = x.is_contiguous()
        if out is None:
            out = torch.empty_like(x, dtype=kind) if plain \
                else torch.empty(x.shape, dtype=kind, device=x.device)
        else:
            _given("codes" if fp8 else "out", out, x.shape, kind)
        if fp8:
            if scales is None:
                scales = torch.empty(x.shape[:-1], dtype=_F32, device=x.device)
            else:
                _given("scales", scales, x.shape[:-1], _F32)
        if sum_out is not None:
            _given("sum_out", sum_out, x.shape, dtype)
        elif residual is not None:
            sum_out = torch.empty_like(x) if plain \
                else torch.empty(x.shape, dtype=dtype, device=x.device)
    sp = None if sum_out is None else sum_out.data_ptr()
    if fp8:
        rc = _lib().moe_add_rmsnorm_fp8(x.data_ptr(), rp, weight.data_ptr(), dt, rows, d, xs, rs, eps,
                                        sp, out.data_ptr(), scales.data_ptr(), handle)
    else:
        rc = _lib().moe_add_rmsnorm(x.data_ptr(), rp, weight.data_ptr(), dt, rows, d, xs, rs, eps, sp,
                                    out.data_ptr(), handle)
    if rc:
        raise MoeError(rc, "moe_add_rmsnorm_fp8" if fp8 else "moe_add_rmsnorm")
    return out, scales, sum_out


def add_rmsnorm(x, weight, residual=None, eps=1e-6, out=None, sum_out=None, stream=None):
    """moe_add_rmsnorm over the last dimension of x (bf16 or float32): returns
    (out, sum) with sum = x + residual, None without a residual unless sum_out
    is given.  Rows may be strided (a slice of a wider tensor)."""
    out, _, s = _norm(x, weight, residual, eps, out, None, sum_out, stream, False)
    return out, s


def add_rmsnorm_fp8(x, weight, residual=None, eps=1e-6, codes=None, scales=None, sum_out=None,
                    stream=None):
    """moe_add_rmsnorm_fp8 over the last dimension of x: returns (codes
    float8_e4m3fn of x's shape, scales float32 of its leading shape, sum as in
    add_rmsnorm)."""
    return _norm(x, weight, residual, eps, codes, scales, sum_out, stream, True)


def quantize_fp8(w, codes=None, scales=None, stream=None):
    """moe_quantize_fp8 of the rows of w (bf16 or float32): (codes
    float8_e4m3fn, scales float32)."""
    dt = _DTYPES.get(w.dtype)
    if dt is None or not w.is_cuda:
        raise ValueError("w must be a CUDA bfloat16 or float32 tensor")
    rows, d, stride = _rows("w", w)
    ctx, handle = _on(stream, _device(w, codes, scales))
    with ctx:
        if codes is None:
            codes = torch.empty(w.shape, dtype=_F8, device=w.device)
        else:
            _given("codes", codes, w.shape, _F8)
        if scales is None:
            scales = torch.empty(w.shape[:-1], dtype=_F32, device=w.device)
        else:
            _given("scales", scales, w.shape[:-1], _F32)
    rc = _lib().moe_quantize_fp8(w.data_ptr(), dt, rows, d, stride, codes.data_ptr(),
                                 scales.data_ptr(), handle)
    if rc:
        raise MoeError(rc, "moe_quantize_fp8")
    return codes, scales


def matmul_fp8(x, x_scales, w, w_scales, out=None, stream=None):
    """moe_matmul_fp8: x float8_e4m3fn [..., K] with scales float32 [...], w
    float8_e4m3fn [N, K] with scales float32 [N] -> bf16 [..., N].  Rows of x, w
    and a given out may be strided."""
    if x.dtype != _F8 or w.dtype != _F8 or not x.is_cuda or not w.is_cuda:
        raise ValueError("x and w must be CUDA float8_e4m3fn tensors")
    T, K, xs = _rows("x", x)
    N, Kw, ws = _rows("w", w)
    if w.dim() != 2 or Kw != K:
        raise ValueError("w must be [N][K] with x's K")
    lead = x.shape[:-1]
    _given("x_scales", x_scales, lead, _F32)
    _vector("w_scales", w_scales, N, _F32)
    ctx, handle = _on(stream, _device(x, x_scales, w, w_scales, out))
    os_ = N
    if out is None:
        with ctx:
            out = torch.empty((*lead, N), dtype=_BF16, device=x.device)
    else:
        if out.dtype != _BF16 or not out.is_cuda or out.shape != (*lead, N):
            raise ValueError("out must be a CUDA bfloat16 tensor of x's leading shape and N columns")
        _, _, os_ = _rows("out", out)
    rc = _lib().moe_matmul_fp8(x.data_ptr(), x_scales.data_ptr(), T, xs, w.data_ptr(),
                               w_scales.data_ptr(), N, K, ws, out.data_ptr(), os_, handle)
    if rc:
        raise MoeError(rc, "moe_matmul_fp8")
    return out


def _tokens(name, t, H, w):
    """Token stride of bf16 [..., heads, width], tokens evenly spaced."""
    if t.dtype != _BF16 or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA bfloat16 tensor")
    if t.is_contiguous():
        return H * w
    strides, shape = t.stride(), t.shape
    if (w > 1 and strides[-1] != 1) or (H > 1 and strides[-2] != w):
        raise ValueError(f"{name}: heads and their width must be contiguous")
    step = strides[-3]
    if len(shape) == 4 and shape[0] > 1:
        if shape[1] == 1:
            step = strides[0]
        elif strides[0] != shape[1] * step:
            raise ValueError(f"{name}: tokens must be evenly spaced")
    return max(step, H * w) if t.numel() <= H * w else step


@functools.lru_cache(maxsize=1024)
def _decay_workspace(N, n, ragged, Hv, dk, dv):
    """Bytes that gdn_decay_scan wants for these sizes."""
    need = ctypes.c_size_t(0)
    rc = _lib().gdn_decay_workspace(N, n, ragged, Hv, dk, dv, ctypes.byref(need))
    if rc:
        raise MoeError(rc, "gdn_decay_workspace")
    return need.value


def gdn_decay_scan(q, k, v, decay, state=None, offsets=None, out=None, state_out=None,
                   stream=None):
    """Linear attention with a decay per value head (include/gdn.h).

    q, k: bf16 [n][T][H_k][d_k], v: bf16 [n][T][H_v][d_v] for n sequences of T
    tokens; or [N][H][d] for one sequence, or, with offsets (int32 [n + 1] on
    the GPU), for n packed ones.  Tokens may be strided (slices of a fused
    projection).  decay: float32 [H_v].  state: float32 [n][H_v][d_v][d_k]
    ([H_v][d_v][d_k] for one sequence of [N][H][d] tokens) or None (zeros).
    Returns (o bf16 of v's shape, final state); state_out may be `state`.
    """
    sq, sv = q.shape, v.shape
    dims = len(sq)
    if dims not in (3, 4) or sq != k.shape or len(sv) != dims or sv[:-2] != sq[:-2]:
        raise ValueError("shapes of q, k, v do not agree")
    Hk, dk = sq[-2:]
    Hv, dv = sv[-2:]
    _vector("decay", decay, Hv, _F32)
    op = None
    if dims == 4:
        if offsets is not None:
            raise ValueError("offsets go with packed tokens [N][H][d]")
        n, N = sq[0], sq[0] * sq[1]
        s_shape = (n, Hv, dv, dk)
    else:
        n, N, s_shape = 1, sq[0], (Hv, dv, dk)
        if offsets is not None:
            if offsets.dtype != torch.int32 or offsets.dim() != 1 or not offsets.is_contiguous() \
                    or not offsets.is_cuda or offsets.shape[0] < 1:
                raise ValueError("offsets must be a contiguous CUDA int32 tensor [n + 1]")
            n = offsets.shape[0] - 1
            s_shape = (n, Hv, dv, dk)
            op = offsets.data_ptr()
    qs, ks, vs = _tokens("q", q, Hk, dk), _tokens("k", k, Hk, dk), _tokens("v", v, Hv, dv)
    sp = None
    if state is not None:
        _given("state", state, s_shape, _F32)
        sp = state.data_ptr()
    need = _decay_workspace(N, n, op is not None, Hv, dk, dv)
    ctx, handle = _on(stream, _device(v, q, k, decay, state, offsets, out, state_out))
    with ctx:
        if out is None:
            out = torch.empty(sv, dtype=_BF16, device=v.device)
        else:
            _given("out", out, sv, _BF16)
        if state_out is None:
            state_out = torch.empty(s_shape, dtype=_F32, device=v.device)
        else:
            _given("state_out", state_out, s_shape, _F32)
        ws = torch.empty(need, dtype=torch.uint8, device=v.device) if need else None
    rc = _lib().gdn_decay_scan(q.data_ptr(), k.data_ptr(), v.data_ptr(), decay.data_ptr(), sp,
                               state_out.data_ptr(), out.data_ptr(), op, N, n, Hk, Hv, dk, dv, qs,
                               ks, vs, None if ws is None else ws.data_ptr(), need, handle)
    if rc:
        raise MoeError(rc, "gdn_decay_scan")
    return out, state_out
