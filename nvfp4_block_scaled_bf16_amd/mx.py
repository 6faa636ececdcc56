"""MXFP4 on AMD MI355X (gfx950): cast, products, and products by expert.

Blocks of 32 elements with E2M1 codes and one power-of-two (E8M0) scale, the
format that gfx950's matrix cores multiply directly (see the header for the
arithmetic).  R vectors of K elements are ``q`` uint8 [R, Kp/2] (Kp: K rounded
up to 128) and ``sf`` uint8 [cdiv(R, 128), Kp/128, 128, 4].  Like the rest of
the package these functions only check and marshal: outputs are allocated with
torch on the input's device and the work is enqueued on its current stream.

One linear layer, forward and backward::

    qx, qw, qd = nv.mx_quantize(x), nv.mx_quantize(w), nv.mx_quantize(dy)
    y = nv.mx_gemm(qx["row_q"], qx["row_sf"], qw["row_q"], qw["row_sf"])
    dx = nv.mx_gemm(qd["row_q"], qd["row_sf"], qw["col_q"], qw["col_sf"])
    dw = nv.mx_gemm(qd["col_q"], qd["col_sf"], qx["col_q"], qx["col_sf"], torch.float32)
"""
from __future__ import annotations

import ctypes

import torch

from . import _check, _ptr, _stream, _u8, lib

_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


def _up(n, m):
    return -(-n // m) * m


def mx_sf_shape(R: int, K: int) -> tuple:
    """Shape of the scale codes of R vectors of K elements."""
    return (_up(R, 128) // 128, _up(K, 128) // 128, 128, 4)


def mx_padded_rows(R: int, num_groups: int) -> int:
    """Length of a columnwise vector over R rows in groups: each group begins
    a 128-element step of its own."""
    return (R + 127 * min(num_groups, R)) // 128 * 128


def _type(dtype, name):
    try:
        return _TYPES[dtype]
    except KeyError:
        raise ValueError(f"{name} must be float32, bfloat16 or float16 (got {dtype})") from None


def _matrix(x, name="x"):
    """A 2-D tensor with adjacent columns: its row pitch in elements."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2 or not x.is_cuda:
        raise ValueError(f"{name} must be a 2-D CUDA tensor")
    _type(x.dtype, name)
    if x.shape[1] > 1 and x.stride(1) != 1:
        raise ValueError(f"{name} must have adjacent columns (stride 1 in its last dimension)")
    return x.stride(0) if x.shape[0] > 1 else x.shape[1]


def _tensor(t, dtype, device, name, shape=None):
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor on {device}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have the shape {tuple(shape)} (got {tuple(t.shape)})")
    return t


def _codes(q, sf, name, batch=False):
    """Vectors and padded length of one operand (``batch``: one per group)."""
    dims = 3 if batch else 2
    if not isinstance(q, torch.Tensor) or q.dim() != dims or not q.is_cuda or q.shape[-1] % 64:
        raise ValueError(f"{name}_q must be a {dims}-D uint8 CUDA tensor with rows of a multiple of 64 bytes")
    _tensor(q, torch.uint8, q.device, f"{name}_q")
    rows, Kp = q.shape[-2], 2 * q.shape[-1]
    _tensor(sf, torch.uint8, q.device, f"{name}_sf", (q.shape[0],) * batch + mx_sf_shape(rows, Kp))
    return rows, Kp


def _groups(offsets, rows, R, device):
    if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1 or offsets.numel() < 1:
        raise ValueError("offsets must be a 1-D int32 tensor of num_groups + 1 values")
    _tensor(offsets, torch.int32, device, "offsets")
    if rows is not None:
        _tensor(rows, torch.int32, device, "rows", (rows.numel(),))
        R = rows.numel()
    return offsets.numel() - 1, R


def mx_quantize(x: torch.Tensor, rowwise: bool = True, columnwise: bool = True) -> dict:
    """MXFP4 cast of x [M, K] (float32, bfloat16 or float16; any row pitch, or
    the transpose of such a tensor): ``row_q`` [M, Kp/2] and ``row_sf`` for its
    rows, ``col_q`` [K, Mp/2] and ``col_sf`` for its columns, from one read."""
    if isinstance(x, torch.Tensor) and x.dim() == 2 and x.shape[1] > 1 and x.stride(1) != 1 and x.stride(0) == 1:
        t = mx_quantize(x.t(), columnwise, rowwise)
        swap = {"row": "col", "col": "row"}
        return {swap[k[:3]] + k[3:]: v for k, v in t.items()}
    ldx = _matrix(x)
    M, K = x.shape
    dev, out = x.device, {}
    if rowwise:
        out.update(row_q=_u8((M, _up(K, 128) // 2), dev), row_sf=_u8(mx_sf_shape(M, K), dev))
    if columnwise:
        out.update(col_q=_u8((K, _up(M, 128) // 2), dev), col_sf=_u8(mx_sf_shape(K, M), dev))
    g = out.get
    if not out:
        raise ValueError("no output direction requested")
    if M and K:
        _check(lib().nvfp4_mx_quantize(_ptr(x), _TYPES[x.dtype], M, K, ldx, _ptr(g("row_q")), _ptr(g("row_sf")),
                                       _ptr(g("col_q")), _ptr(g("col_sf")), _stream(dev)))
    return out


def mx_quantize_grouped(x: torch.Tensor, offsets: torch.Tensor, rows: torch.Tensor | None = None,
                        rowwise: bool = True, columnwise: bool = True) -> dict:
    """MXFP4 cast of the R rows x[rows] (all of x without ``rows``) that groups
    hold: group e those from offsets[e] to offsets[e + 1], int32 on the device.
    Columnwise vectors have :func:`mx_padded_rows` elements, each group
    beginning a step of 128 of its own, for :func:`mx_wgrad_grouped`."""
    ldx = _matrix(x)
    M, K = x.shape
    dev, out = x.device, {}
    E, R = _groups(offsets, rows, M, dev)
    if rowwise:
        out.update(row_q=_u8((R, _up(K, 128) // 2), dev), row_sf=_u8(mx_sf_shape(R, K), dev))
    if columnwise:
        Tp = mx_padded_rows(R, E)
        out.update(col_q=_u8((K, Tp // 2), dev), col_sf=_u8(mx_sf_shape(K, Tp), dev))
    g = out.get
    if not out:
        raise ValueError("no output direction requested")
    if R and K and (rowwise or E):
        _check(lib().nvfp4_mx_quantize_grouped(_ptr(x), _TYPES[x.dtype], M, K, ldx, _ptr(rows), R, _ptr(offsets), E,
                                               _ptr(g("row_q")), _ptr(g("row_sf")), _ptr(g("col_q")),
                                               _ptr(g("col_sf")), _stream(dev)))
    return out


def mx_dequantize(q: torch.Tensor, sf: torch.Tensor, K: int, out_dtype=torch.float32) -> torch.Tensor:
    """The values [R, K] that codes and scales stand for."""
    R, Kp = _codes(q, sf, "mx")
    t = _type(out_dtype, "out_dtype")
    if not 0 <= K <= Kp or Kp != _up(K, 128):
        raise ValueError(f"K={K} does not fit rows of {Kp} codes")
    out = torch.empty((R, K), dtype=out_dtype, device=q.device)
    _check(lib().nvfp4_mx_dequantize(_ptr(q), _ptr(sf), R, K, t, _ptr(out), _stream(q.device)))
    return out


def mx_gemm(a_q, a_sf, b_q, b_sf, out_dtype=torch.bfloat16) -> torch.Tensor:
    """out [M, N] = a b^T for M vectors a and N vectors b, summed in fp32."""
    M, K = _codes(a_q, a_sf, "a")
    N, Kb = _codes(b_q, b_sf, "b")
    if K != Kb or a_q.device != b_q.device:
        raise ValueError("a and b differ in length or device")
    t = _type(out_dtype, "out_dtype")
    out = torch.empty((M, N), dtype=out_dtype, device=a_q.device)
    _check(lib().nvfp4_mx_gemm(_ptr(a_q), _ptr(a_sf), _ptr(b_q), _ptr(b_sf), M, N, K, t, _ptr(out),
                               _stream(a_q.device)))
    return out


def mx_gemm_grouped(a_q, a_sf, b_q, b_sf, offsets, rows=None, row_scale=None,
                    out_dtype=torch.bfloat16) -> torch.Tensor:
    """out [R, N]: for the rows r of group e, row_scale[r] * a[rows[r]] b_e^T.
    b_q [E, N, Kp/2] and b_sf hold one operand per group; rows of out that no
    group holds are not written."""
    A, K = _codes(a_q, a_sf, "a")
    N, Kb = _codes(b_q, b_sf, "b", batch=True)
    dev = a_q.device
    if K != Kb or b_q.device != dev:
        raise ValueError("a and b differ in length or device")
    E, R = _groups(offsets, rows, A, dev)
    if E != b_q.shape[0]:
        raise ValueError(f"offsets are for {E} groups, b for {b_q.shape[0]}")
    if row_scale is not None:
        _tensor(row_scale, torch.float32, dev, "row_scale", (R,))
    t = _type(out_dtype, "out_dtype")
    out = torch.empty((R, N), dtype=out_dtype, device=dev)
    _check(lib().nvfp4_mx_gemm_grouped(_ptr(a_q), _ptr(a_sf), A, _ptr(rows), R, _ptr(offsets), E, _ptr(b_q),
                                       _ptr(b_sf), N, K, _ptr(row_scale), t, _ptr(out), _stream(dev)))
    return out


def mx_wgrad_grouped(a_q, a_sf, b_q, b_sf, offsets, out_dtype=torch.float32) -> torch.Tensor:
    """out [E, N, K]: for each group the sum over its rows of a[n][r] b[k][r],
    from the columnwise outputs of :func:`mx_quantize_grouped` with the same
    offsets.  An empty group gives zeros."""
    N, Tp = _codes(a_q, a_sf, "a")
    K, Tb = _codes(b_q, b_sf, "b")
    dev = a_q.device
    if Tp != Tb or b_q.device != dev:
        raise ValueError("a and b differ in length or device")
    E, _ = _groups(offsets, None, 0, dev)
    t = _type(out_dtype, "out_dtype")
    out = torch.empty((E, N, K), dtype=out_dtype, device=dev)
    _check(lib().nvfp4_mx_wgrad_grouped(_ptr(a_q), _ptr(a_sf), _ptr(b_q), _ptr(b_sf), N, K, Tp, _ptr(offsets), E, t,
                                        _ptr(out), _stream(dev)))
    return out


def _workspace(n, dev):
    return _u8(n, dev) if n else None


def mx_linear(x: torch.Tensor, w_q, w_sf, out_dtype=None) -> torch.Tensor:
    """y [M, N] = Q(x) W^T for x [M, K] (cast on the way) and N weight vectors;
    of x's type unless ``out_dtype`` is given."""
    ldx = _matrix(x)
    M, K = x.shape
    N, Kp = _codes(w_q, w_sf, "w")
    dev = x.device
    if Kp != _up(K, 128) or w_q.device != dev:
        raise ValueError(f"x of {K} columns does not fit weights of {Kp} codes on {w_q.device}")
    out_dtype = out_dtype or x.dtype
    t = _type(out_dtype, "out_dtype")
    out = torch.empty((M, N), dtype=out_dtype, device=dev)
    L = lib()
    n = L.nvfp4_mx_linear_workspace(M, N, K)
    ws = _workspace(n, dev)
    _check(L.nvfp4_mx_linear(_ptr(x), _TYPES[x.dtype], M, K, ldx, _ptr(w_q), _ptr(w_sf), N, t, _ptr(out), _ptr(ws), n,
                             _stream(dev)))
    return out


def mx_linear_grouped(x: torch.Tensor, w_q, w_sf, offsets, rows=None, row_scale=None,
                      out_dtype=None) -> torch.Tensor:
    """:func:`mx_gemm_grouped` on x [M, K], each of its rows cast once on the
    way: out[r] = row_scale[r] * Q(x[rows[r]]) W_e^T for the rows r of e."""
    ldx = _matrix(x)
    M, K = x.shape
    N, Kp = _codes(w_q, w_sf, "w", batch=True)
    dev = x.device
    if Kp != _up(K, 128) or w_q.device != dev:
        raise ValueError(f"x of {K} columns does not fit weights of {Kp} codes on {w_q.device}")
    E, R = _groups(offsets, rows, M, dev)
    if E != w_q.shape[0]:
        raise ValueError(f"offsets are for {E} groups, w for {w_q.shape[0]}")
    if row_scale is not None:
        _tensor(row_scale, torch.float32, dev, "row_scale", (R,))
    out_dtype = out_dtype or x.dtype
    t = _type(out_dtype, "out_dtype")
    out = torch.empty((R, N), dtype=out_dtype, device=dev)
    L = lib()
    n = L.nvfp4_mx_linear_grouped_workspace(M, R, N, K)
    ws = _workspace(n, dev)
    _check(L.nvfp4_mx_linear_grouped(_ptr(x), _TYPES[x.dtype], M, K, ldx, _ptr(rows), R, _ptr(offsets), E, _ptr(w_q),
                                     _ptr(w_sf), N, _ptr(row_scale), t, _ptr(out), _ptr(ws), n, _stream(dev)))
    return out
