"""Torch-facing wrappers of libdsv's row calls: norms of rows, and activations
kept in 8 bits for the backward pass. They only marshal arguments, through the
native binding (csrc/rows_binding.cpp): these calls are also made on small
tensors, where the marshalling is the time.

Tensors are CUDA bf16, fp16 or fp32 of shape [B, H, S, D], [H, S, D] or
[S, D] with unit stride along D; the other strides are free, so a head of a
fused projection is read (and its gradient written) where it lies. Calls run
on the current stream of the tensors' device.
"""
from __future__ import annotations

import importlib.util
import os
from typing import Optional, Union

import torch

from . import native as N
from .api import PackedAct

BINDING_PATH = os.path.join(N.PKG, "_rows.so")
_binding = None


def _load():
    """The native binding (loaded once). Raises if it is not built."""
    global _binding
    if _binding is None:
        N.load()          # the same libdsv.so, which the binding links against
        if not os.path.exists(BINDING_PATH):
            raise RuntimeError(f"_rows.so not built ({BINDING_PATH}); run `python -c 'import __graft_entry__ as g; "
                               "g.build()'`")
        spec = importlib.util.spec_from_file_location(__package__ + "._rows", BINDING_PATH)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        module.init(PackedAct, N.DsvError)
        _binding = module
    return _binding


def layer_norm_fwd(x, weight=None, bias=None, eps: float = 1e-6, center: bool = True, weight_base: float = 0.0,
                   dtype: Optional[torch.dtype] = None, y=None, pack: Union[bool, PackedAct] = False):
    """dsv_layer_norm_fwd. x: a tensor or a PackedAct. weight, bias: [D], or x's
    dimensions with 1 for S and 1 or x's size for B and H; the factor is
    weight_base + weight. center=False: root mean square norm. y's type is
    dtype (x's by default, bf16 for a PackedAct). pack=True (or a PackedAct to
    fill) keeps x's 8-bit checkpoint from the same pass.
    Returns (y, mean or None, rstd, PackedAct or None)."""
    return (_binding or _load()).layer_norm_fwd(x, weight, bias, eps, center, weight_base, dtype, y, pack)


def layer_norm_bwd_workspace_size(x, weight=None) -> int:
    """Bytes of workspace layer_norm_bwd takes for x and this weight (or bias)."""
    return (_binding or _load()).layer_norm_bwd_workspace_size(x, weight)


def layer_norm_bwd(dy, x, mean, rstd, weight=None, bias=None, weight_base: float = 0.0, dx=None, workspace=None):
    """dsv_layer_norm_bwd. x: the forward's input or its PackedAct; mean (None
    for the root mean square norm) and rstd as the forward returned them.
    weight, bias, weight_base as given to the forward (the bias's values are not
    read). Returns (dx, dweight, dbias): dx of x's type (dy's for a PackedAct),
    the others fp32 in the parameters' shape, None without the parameter."""
    return (_binding or _load()).layer_norm_bwd(dy, x, mean, rstd, weight, bias, weight_base, dx, workspace)


def act_pack(x, out: Optional[PackedAct] = None) -> PackedAct:
    """dsv_act_pack: x kept in 8 bits (blocks of 32 channels share an exponent)."""
    return (_binding or _load()).act_pack(x, out)


def act_unpack(packed: PackedAct, dtype: torch.dtype = torch.bfloat16, out=None) -> torch.Tensor:
    """dsv_act_unpack: the values a checkpoint stands for (exact in bf16 and fp32)."""
    return (_binding or _load()).act_unpack(packed, dtype, out)
