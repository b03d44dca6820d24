"""Torch-facing wrappers of libdsv's row calls (argument marshalling only):
norms of rows, and activations kept in 8 bits for the backward pass.

Tensors are CUDA bf16, fp16 or fp32 of shape [B, H, S, D], [H, S, D] or
[S, D] with unit stride along D; the other strides are free, so a head of a
fused projection is read (and its gradient written) where it lies. Calls run
on the current stream of the tensors' device.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import NamedTuple, Optional, Tuple, Union

import torch

from . import native as N
from .api import _ptr, _workspace

_TYPES = {torch.bfloat16: N.DSV_BF16, torch.float16: N.DSV_FP16, torch.float32: N.DSV_FP32}
_BLOCK = 32
_NO_ROWS = N.dsv_rows(None, None, N.DSV_PACKED, 0, 0, 0)


class PackedAct(NamedTuple):
    """An 8-bit checkpoint of an activation x: q int8 in x's shape, e uint8 with
    one exponent per 32 channels ([..., ceil(D / 32)]), both contiguous. A channel
    stands for q * 2^(e - 133), a block with e = 255 for NaN."""

    q: torch.Tensor
    e: torch.Tensor

    @property
    def shape(self):
        return self.q.shape

    @property
    def device(self):
        return self.q.device


def _extent(shape) -> N.dsv_extent:
    if len(shape) not in (2, 3, 4):
        raise ValueError("expected [B, H, S, D], [H, S, D] or [S, D]")
    return N.dsv_extent(*([1] * (4 - len(shape)) + list(shape)))


def _rows(t: Union[torch.Tensor, PackedAct], shape, device, what: str) -> N.dsv_rows:
    """The dsv_rows of a tensor (or a checkpoint) that must have this shape and device."""
    if isinstance(t, PackedAct):
        q, e = t
        if not q.is_cuda or q.device != device or e.device != device:
            raise ValueError(f"{what}: expected CUDA tensors on {device}")
        if q.dtype != torch.int8 or e.dtype != torch.uint8 or not q.is_contiguous() or not e.is_contiguous():
            raise ValueError(f"{what}: expected contiguous int8 values and uint8 exponents")
        if q.shape != shape or tuple(e.shape) != tuple(shape[:-1]) + ((shape[-1] + _BLOCK - 1) // _BLOCK,):
            raise ValueError(f"{what}: values {tuple(q.shape)} and exponents {tuple(e.shape)} do not match {tuple(shape)}")
        return N.dsv_rows(q.data_ptr(), e.data_ptr(), N.DSV_PACKED, 0, 0, 0)
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype not in _TYPES:
        raise ValueError(f"{what}: expected a CUDA bf16, fp16 or fp32 tensor")
    if t.device != device:
        raise ValueError(f"{what} is on {t.device}, expected {device}")
    if t.shape != shape:
        raise ValueError(f"{what} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    st = t.stride()
    if shape[-1] > 1 and st[-1] != 1:
        raise ValueError(f"{what}: channels must have unit stride")
    return N.dsv_rows(t.data_ptr(), None, _TYPES[t.dtype], *([0] * (4 - len(st)) + list(st[:-1])))


def _param_layout(p: torch.Tensor, shape) -> Tuple[int, int, int, int]:
    """(per_batch, per_head, batch stride, head stride) of a weight or bias:
    [D], or x's dimensions with 1 for S and 1 or x's size for B and H."""
    D = shape[-1]
    if p.shape[-1:] != (D,) or (D > 1 and p.stride(-1) != 1):
        raise ValueError(f"weight and bias hold {D} channels of unit stride, got {tuple(p.shape)}")
    if p.dim() == 1:
        return 0, 0, 0, 0
    if p.dim() != len(shape) or p.shape[-2] != 1 or any(a not in (1, b) for a, b in zip(p.shape, shape)):
        raise ValueError(f"weight and bias broadcast over S: got {tuple(p.shape)} for {tuple(shape)}")
    lead = list(zip(p.shape[:-2], p.stride()[:-2]))
    (nb, sb), (nh, sh) = [(1, 0)] * (2 - len(lead)) + lead
    # an empty dimension of x (size 0) keeps its empty gradient
    return int(nb != 1), int(nh != 1), sb, sh


def _params(weight, bias, base: float, shape, device) -> N.dsv_norm_params:
    given = [p for p in (weight, bias) if p is not None]
    for p in given:
        if not p.is_cuda or p.device != device or p.dtype not in _TYPES:
            raise ValueError(f"weight and bias: expected bf16, fp16 or fp32 tensors on {device}")
    if len(given) == 2 and (weight.dtype != bias.dtype or weight.shape != bias.shape):
        raise ValueError("weight and bias must have one type and shape")
    if not given:
        return N.dsv_norm_params(None, None, N.DSV_FP32, 0, 0, 0, 0, 0, 0, 1.0)
    lw = _param_layout(weight, shape) if weight is not None else (0, 0, 0, 0)
    lb = _param_layout(bias, shape) if bias is not None else (0, 0, 0, 0)
    per = lw if weight is not None else lb
    return N.dsv_norm_params(weight.data_ptr() if weight is not None else None,
                             bias.data_ptr() if bias is not None else None, _TYPES[given[0].dtype], per[0], per[1],
                             lw[2], lw[3], lb[2], lb[3], float(base))


def _on(device):
    """The device's context, entered only where another device is current."""
    if device.index is None or device.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(device)


def _stream_of(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _source(x) -> Tuple[torch.Size, torch.device]:
    t = x.q if isinstance(x, PackedAct) else x
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("expected a CUDA tensor or a PackedAct")
    return t.shape, t.device


def _stats(t, shape, device, what):
    if t is not None and (t.dtype != torch.float32 or t.shape != shape[:-1] or not t.is_contiguous() or
                          t.device != device):
        raise ValueError(f"{what}: expected a contiguous float32 tensor {tuple(shape[:-1])} on {device}")
    return t


def _new_packed(shape, device) -> PackedAct:
    return PackedAct(torch.empty(shape, dtype=torch.int8, device=device),
                     torch.empty(tuple(shape[:-1]) + ((shape[-1] + _BLOCK - 1) // _BLOCK,), dtype=torch.uint8,
                                 device=device))


def layer_norm_fwd(x, weight=None, bias=None, eps: float = 1e-6, center: bool = True, weight_base: float = 0.0,
                   dtype: Optional[torch.dtype] = None, y=None, pack: Union[bool, PackedAct] = False):
    """dsv_layer_norm_fwd. x: a tensor or a PackedAct. weight, bias: [D], or x's
    dimensions with 1 for S and 1 or x's size for B and H; the factor is
    weight_base + weight. center=False: root mean square norm. y's type is
    dtype (x's by default, bf16 for a PackedAct). pack=True (or a PackedAct to
    fill) keeps x's 8-bit checkpoint from the same pass.
    Returns (y, mean or None, rstd, PackedAct or None)."""
    shape, device = _source(x)
    n = _extent(shape)
    xr = _rows(x, shape, device, "x")
    par = _params(weight, bias, weight_base, shape, device)
    if y is None:
        y = torch.empty(shape, dtype=dtype or (torch.bfloat16 if isinstance(x, PackedAct) else x.dtype), device=device)
    elif dtype is not None and y.dtype != dtype:
        raise ValueError("y does not have the type asked for")
    yr = _rows(y, shape, device, "y")
    mean = torch.empty(shape[:-1], dtype=torch.float32, device=device) if center else None
    rstd = torch.empty(shape[:-1], dtype=torch.float32, device=device)
    kept = pack if isinstance(pack, PackedAct) else _new_packed(shape, device) if pack else None
    kr = _rows(kept, shape, device, "pack") if kept is not None else _NO_ROWS
    with _on(device):
        code = N.load().dsv_layer_norm_fwd(xr, n, par, float(eps), int(bool(center)), yr, _ptr(mean), _ptr(rstd), kr,
                                           _stream_of(device))
    N.check(code, "dsv_layer_norm_fwd")
    return y, mean, rstd, kept


def layer_norm_bwd_workspace_size(x, weight=None) -> int:
    """Bytes of workspace layer_norm_bwd takes for x and this weight (or bias)."""
    shape, _ = _source(x)
    per = _param_layout(weight, shape) if weight is not None else (0, 0)
    return int(N.load().dsv_layer_norm_bwd_workspace_size(_extent(shape), per[0], per[1]))


def layer_norm_bwd(dy, x, mean, rstd, weight=None, bias=None, weight_base: float = 0.0, dx=None, workspace=None):
    """dsv_layer_norm_bwd. x: the forward's input or its PackedAct; mean (None
    for the root mean square norm) and rstd as the forward returned them.
    weight, bias, weight_base as given to the forward (the bias's values are not
    read). Returns (dx, dweight, dbias): dx of x's type (dy's for a PackedAct),
    the others fp32 in the parameters' shape, None without the parameter."""
    shape, device = _source(x)
    n = _extent(shape)
    xr = _rows(x, shape, device, "x")
    dyr = _rows(dy, shape, device, "dy")
    par = _params(weight, bias, weight_base, shape, device)
    _stats(mean, shape, device, "mean")
    if rstd is None:
        raise ValueError("rstd is needed")
    _stats(rstd, shape, device, "rstd")
    if dx is None:
        dx = torch.empty(shape, dtype=dy.dtype if isinstance(x, PackedAct) else x.dtype, device=device)
    dxr = _rows(dx, shape, device, "dx")
    dw = torch.empty(weight.shape, dtype=torch.float32, device=device) if weight is not None else None
    db = torch.empty(bias.shape, dtype=torch.float32, device=device) if bias is not None else None
    lib = N.load()
    ws = None
    if dw is not None or db is not None:
        need = int(lib.dsv_layer_norm_bwd_workspace_size(n, par.per_batch, par.per_head))
        if need or workspace is not None:
            ws = _workspace(need, device, workspace)
    with _on(device):
        code = lib.dsv_layer_norm_bwd(dyr, xr, n, par, _ptr(mean), _ptr(rstd), dxr, _ptr(dw), _ptr(db), _ptr(ws),
                                      ws.numel() if ws is not None else 0, _stream_of(device))
    N.check(code, "dsv_layer_norm_bwd")
    return dx, dw, db


def act_pack(x, out: Optional[PackedAct] = None) -> PackedAct:
    """dsv_act_pack: x kept in 8 bits (blocks of 32 channels share an exponent)."""
    if isinstance(x, PackedAct):
        raise ValueError("x is packed already")
    shape, device = _source(x)
    n = _extent(shape)
    xr = _rows(x, shape, device, "x")
    out = _new_packed(shape, device) if out is None else out
    if not isinstance(out, PackedAct):
        raise ValueError("out: expected a PackedAct")
    pr = _rows(out, shape, device, "out")
    with _on(device):
        code = N.load().dsv_act_pack(xr, n, pr, _stream_of(device))
    N.check(code, "dsv_act_pack")
    return out


def act_unpack(packed: PackedAct, dtype: torch.dtype = torch.bfloat16, out=None) -> torch.Tensor:
    """dsv_act_unpack: the values a checkpoint stands for (exact in bf16 and fp32)."""
    if not isinstance(packed, PackedAct):
        raise ValueError("expected a PackedAct")
    shape, device = _source(packed)
    n = _extent(shape)
    pr = _rows(packed, shape, device, "packed")
    out = torch.empty(shape, dtype=dtype, device=device) if out is None else out
    yr = _rows(out, shape, device, "out")
    with _on(device):
        code = N.load().dsv_act_unpack(pr, n, yr, _stream_of(device))
    N.check(code, "dsv_act_unpack")
    return out
