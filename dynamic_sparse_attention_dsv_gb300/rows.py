"""Torch-facing wrappers of libdsv's row calls (argument marshalling only):
norms of rows, and activations kept in 8 bits for the backward pass.

Tensors are CUDA bf16, fp16 or fp32 of shape [B, H, S, D], [H, S, D] or
[S, D] with unit stride along D; the other strides are free, so a head of a
fused projection is read (and its gradient written) where it lies. Calls run
on the current stream of the tensors' device.
"""
from __future__ import annotations

import functools
from typing import Optional, Tuple, Union

import torch

from . import native as N
from .api import PackedAct, _workspace

_TYPES = {torch.bfloat16: N.DSV_BF16, torch.float16: N.DSV_FP16, torch.float32: N.DSV_FP32}
_BLOCK = 32
_NO_ROWS = N.dsv_rows(None, None, N.DSV_PACKED, 0, 0, 0)
_NO_PARAMS = N.dsv_norm_params(None, None, N.DSV_FP32, 0, 0, 0, 0, 0, 0, 1.0)
_stream_of = torch._C._cuda_getCurrentRawStream     # of a device index


@functools.lru_cache(maxsize=512)
def _extent(shape) -> N.dsv_extent:
    if len(shape) not in (2, 3, 4):
        raise ValueError("expected [B, H, S, D], [H, S, D] or [S, D]")
    return N.dsv_extent(*([1] * (4 - len(shape)) + list(shape)))


@functools.lru_cache(maxsize=512)
def _bwd_workspace(shape, per_batch: int, per_head: int) -> int:
    return int(N.load().dsv_layer_norm_bwd_workspace_size(_extent(shape), per_batch, per_head))


def _packed_rows(t: PackedAct, shape, dev: int, what: str) -> N.dsv_rows:
    q, e = t
    if q.get_device() != dev or e.get_device() != dev:
        raise ValueError(f"{what}: expected CUDA tensors on device {dev}")
    if q.dtype != torch.int8 or e.dtype != torch.uint8 or not q.is_contiguous() or not e.is_contiguous():
        raise ValueError(f"{what}: expected contiguous int8 values and uint8 exponents")
    if q.shape != shape or e.shape[:-1] != shape[:-1] or e.shape[-1] != (shape[-1] + _BLOCK - 1) // _BLOCK:
        raise ValueError(f"{what}: values {tuple(q.shape)} and exponents {tuple(e.shape)} do not match {tuple(shape)}")
    return N.dsv_rows(q.data_ptr(), e.data_ptr(), N.DSV_PACKED, 0, 0, 0)


def _rows(t: Union[torch.Tensor, PackedAct], shape, dev: int, what: str) -> N.dsv_rows:
    """The dsv_rows of a tensor (or a checkpoint) that must have this shape and device."""
    if isinstance(t, PackedAct):
        return _packed_rows(t, shape, dev, what)
    kind = _TYPES.get(t.dtype) if isinstance(t, torch.Tensor) else None
    if kind is None or t.get_device() != dev:
        raise ValueError(f"{what}: expected a bf16, fp16 or fp32 tensor on CUDA device {dev}")
    if t.shape != shape:
        raise ValueError(f"{what} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    st = t.stride()
    if st[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{what}: channels must have unit stride")
    if len(st) == 4:
        return N.dsv_rows(t.data_ptr(), None, kind, st[0], st[1], st[2])
    return N.dsv_rows(t.data_ptr(), None, kind, 0, st[0] if len(st) == 3 else 0, st[-2])


def _param_layout(p: torch.Tensor, shape) -> Tuple[int, int, int, int]:
    """(per_batch, per_head, batch stride, head stride) of a weight or bias:
    [D], or x's dimensions with 1 for S and 1 or x's size for B and H."""
    D, ps, st = shape[-1], p.shape, p.stride()
    if len(ps) == 0 or ps[-1] != D or (D > 1 and st[-1] != 1):
        raise ValueError(f"weight and bias hold {D} channels of unit stride, got {tuple(ps)}")
    if len(ps) == 1:
        return 0, 0, 0, 0
    if len(ps) != len(shape) or ps[-2] != 1 or any(a != 1 and a != b for a, b in zip(ps, shape)):
        raise ValueError(f"weight and bias broadcast over S: got {tuple(ps)} for {tuple(shape)}")
    nh, sh = (ps[-3], st[-3]) if len(ps) > 2 else (1, 0)
    nb, sb = (ps[-4], st[-4]) if len(ps) > 3 else (1, 0)
    return int(nb != 1), int(nh != 1), sb, sh


def _params(weight, bias, base: float, shape, dev: int) -> N.dsv_norm_params:
    if weight is None and bias is None:
        return _NO_PARAMS
    first = weight if weight is not None else bias
    kind = _TYPES.get(first.dtype)
    if kind is None or first.get_device() != dev:
        raise ValueError(f"weight and bias: expected bf16, fp16 or fp32 tensors on CUDA device {dev}")
    b, h, sb, sh = _param_layout(first, shape)
    if first is bias:
        return N.dsv_norm_params(None, bias.data_ptr(), kind, b, h, 0, 0, sb, sh, base)
    if bias is None:
        return N.dsv_norm_params(weight.data_ptr(), None, kind, b, h, sb, sh, 0, 0, base)
    if bias.dtype != weight.dtype or bias.shape != weight.shape or bias.get_device() != dev:
        raise ValueError("weight and bias must have one type, shape and device")
    _, _, bb, bh = _param_layout(bias, shape)
    return N.dsv_norm_params(weight.data_ptr(), bias.data_ptr(), kind, b, h, sb, sh, bb, bh, base)


def _source(x):
    """(shape, device, device index) of a tensor or checkpoint."""
    t = x.q if isinstance(x, PackedAct) else x
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("expected a CUDA tensor or a PackedAct")
    device = t.device
    return t.shape, device, device.index


def _call(fn, dev: int, where: str, *args) -> None:
    """fn(*args, stream) on the device's current stream; another current device is left as it was."""
    if dev == torch.cuda.current_device():
        code = fn(*args, _stream_of(dev))
    else:
        with torch.cuda.device(dev):
            code = fn(*args, _stream_of(dev))
    if code:
        N.check(code, where)


def _stats(t, shape, dev: int, what: str) -> int:
    if t.dtype != torch.float32 or t.shape != shape[:-1] or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"{what}: expected a contiguous float32 tensor {tuple(shape[:-1])} on CUDA device {dev}")
    return t.data_ptr()


def _new_packed(shape, device) -> PackedAct:
    return PackedAct(torch.empty(shape, dtype=torch.int8, device=device),
                     torch.empty(shape[:-1] + ((shape[-1] + _BLOCK - 1) // _BLOCK,), dtype=torch.uint8, device=device))


def layer_norm_fwd(x, weight=None, bias=None, eps: float = 1e-6, center: bool = True, weight_base: float = 0.0,
                   dtype: Optional[torch.dtype] = None, y=None, pack: Union[bool, PackedAct] = False):
    """dsv_layer_norm_fwd. x: a tensor or a PackedAct. weight, bias: [D], or x's
    dimensions with 1 for S and 1 or x's size for B and H; the factor is
    weight_base + weight. center=False: root mean square norm. y's type is
    dtype (x's by default, bf16 for a PackedAct). pack=True (or a PackedAct to
    fill) keeps x's 8-bit checkpoint from the same pass.
    Returns (y, mean or None, rstd, PackedAct or None)."""
    shape, device, dev = _source(x)
    n = _extent(shape)
    xr = _rows(x, shape, dev, "x")
    par = _params(weight, bias, weight_base, shape, dev)
    if y is None:
        y = torch.empty(shape, dtype=dtype or (torch.bfloat16 if isinstance(x, PackedAct) else x.dtype), device=device)
    elif dtype is not None and y.dtype != dtype:
        raise ValueError("y does not have the type asked for")
    yr = _rows(y, shape, dev, "y")
    rstd = torch.empty(shape[:-1], dtype=torch.float32, device=device)
    mean = torch.empty_like(rstd) if center else None
    kept = pack if isinstance(pack, PackedAct) else _new_packed(shape, device) if pack else None
    kr = _packed_rows(kept, shape, dev, "pack") if kept is not None else _NO_ROWS
    _call(N.load().dsv_layer_norm_fwd, dev, "dsv_layer_norm_fwd", xr, n, par, eps, 1 if center else 0, yr,
          mean.data_ptr() if center else None, rstd.data_ptr(), kr)
    return y, mean, rstd, kept


def layer_norm_bwd_workspace_size(x, weight=None) -> int:
    """Bytes of workspace layer_norm_bwd takes for x and this weight (or bias)."""
    shape = _source(x)[0]
    per = _param_layout(weight, shape) if weight is not None else (0, 0)
    return _bwd_workspace(shape, per[0], per[1])


def layer_norm_bwd(dy, x, mean, rstd, weight=None, bias=None, weight_base: float = 0.0, dx=None, workspace=None):
    """dsv_layer_norm_bwd. x: the forward's input or its PackedAct; mean (None
    for the root mean square norm) and rstd as the forward returned them.
    weight, bias, weight_base as given to the forward (the bias's values are not
    read). Returns (dx, dweight, dbias): dx of x's type (dy's for a PackedAct),
    the others fp32 in the parameters' shape, None without the parameter."""
    shape, device, dev = _source(x)
    n = _extent(shape)
    xr = _rows(x, shape, dev, "x")
    dyr = _rows(dy, shape, dev, "dy")
    par = _params(weight, bias, weight_base, shape, dev)
    mean_at = _stats(mean, shape, dev, "mean") if mean is not None else None
    if rstd is None:
        raise ValueError("rstd is needed")
    rstd_at = _stats(rstd, shape, dev, "rstd")
    if dx is None:
        dx = torch.empty(shape, dtype=dy.dtype if isinstance(x, PackedAct) else x.dtype, device=device)
    dxr = _rows(dx, shape, dev, "dx")
    dw = torch.empty(weight.shape, dtype=torch.float32, device=device) if weight is not None else None
    db = torch.empty(bias.shape, dtype=torch.float32, device=device) if bias is not None else None
    ws = None
    if dw is not None or db is not None:
        need = _bwd_workspace(shape, par.per_batch, par.per_head)
        if need or workspace is not None:
            ws = _workspace(need, device, workspace)
    _call(N.load().dsv_layer_norm_bwd, dev, "dsv_layer_norm_bwd", dyr, xr, n, par, mean_at, rstd_at, dxr,
          dw.data_ptr() if dw is not None else None, db.data_ptr() if db is not None else None,
          ws.data_ptr() if ws is not None else None, ws.numel() if ws is not None else 0)
    return dx, dw, db


def act_pack(x, out: Optional[PackedAct] = None) -> PackedAct:
    """dsv_act_pack: x kept in 8 bits (blocks of 32 channels share an exponent)."""
    if isinstance(x, PackedAct):
        raise ValueError("x is packed already")
    shape, device, dev = _source(x)
    n = _extent(shape)
    xr = _rows(x, shape, dev, "x")
    out = _new_packed(shape, device) if out is None else out
    if not isinstance(out, PackedAct):
        raise ValueError("out: expected a PackedAct")
    _call(N.load().dsv_act_pack, dev, "dsv_act_pack", xr, n, _packed_rows(out, shape, dev, "out"))
    return out


def act_unpack(packed: PackedAct, dtype: torch.dtype = torch.bfloat16, out=None) -> torch.Tensor:
    """dsv_act_unpack: the values a checkpoint stands for (exact in bf16 and fp32)."""
    if not isinstance(packed, PackedAct):
        raise ValueError("expected a PackedAct")
    shape, device, dev = _source(packed)
    n = _extent(shape)
    pr = _packed_rows(packed, shape, dev, "packed")
    out = torch.empty(shape, dtype=dtype, device=device) if out is None else out
    _call(N.load().dsv_act_unpack, dev, "dsv_act_unpack", pr, n, _rows(out, shape, dev, "out"))
    return out
