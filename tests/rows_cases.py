"""Inputs and tolerances shared by the tests of the row calls."""
import torch

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32

#: [B, H, S, D]: one row, one channel, every lane layout (8, 16 and 32 lanes a
#: row, two chunks, several warps), widths no vector load divides, the widest
SHAPES = [(1, 1, 1, 1), (1, 2, 3, 2), (1, 1, 1, 64), (2, 3, 5, 64), (1, 2, 257, 128), (1, 24, 130, 128), (3, 1, 33, 200),
          (2, 2, 7, 40), (1, 3, 70, 33), (1, 1, 9, 264), (1, 1, 5, 512), (1, 1, 3, 520), (2, 1, 4, 2048), (2, 1, 3, 517),
          (1, 1, 3, 1003), (1, 2, 300, 8), (1, 1, 2, 8192), (1, 1, 2, 8191), (2, 2, 40, 1024), (2, 3, 37, 12), (1, 2, 67, 61), (1, 1, 300, 31), (2, 24, 3, 64),
          (30, 2, 4, 40)]
LAYOUTS = ["bhsd", "qkv", "shifted", "padded"]
PARAMS = ["none", "weight", "shared", "batch", "head", "both"]
#: (x, y) types the norms take; None: an 8-bit checkpoint
TYPES = [(BF16, BF16), (FP16, FP16), (FP32, FP32), (FP32, BF16), (FP32, FP16), (None, BF16), (None, FP16), (None, FP32)]


def half_step(t):
    return torch.finfo(t).eps / 2


def lay(t, layout):
    """The values of t [B, H, S, D] with other strides (device kept)."""
    B, H, S, D = t.shape
    if layout == "qkv":
        out = torch.zeros(B, S, 3, H, D, dtype=t.dtype, device=t.device)[:, :, 1].permute(0, 2, 1, 3)
    elif layout == "shifted":   # contiguous, one element off any 16-byte boundary
        out = torch.zeros(t.numel() + 1, dtype=t.dtype, device=t.device)[1:].view(B, H, S, D)
    elif layout == "padded":    # rows of D + 16 channels, planes with a gap
        out = torch.zeros(B, H, S + 2, D + 16, dtype=t.dtype, device=t.device)[:, :, 1:S + 1, 8:8 + D]
    else:
        return t.contiguous()
    out.copy_(t)
    return out


def guarded(shape, dtype, layout, device="cuda"):
    """(view of that shape and layout, the memory it lies in), the memory filled with 7."""
    B, H, S, D = shape
    if layout == "qkv":
        mem = torch.full((B, S, 3, H, D), 7, dtype=dtype, device=device)
        return mem[:, :, 1].permute(0, 2, 1, 3), mem
    if layout == "shifted":
        mem = torch.full((B * H * S * D + 9,), 7, dtype=dtype, device=device)
        return mem[1:1 + B * H * S * D].view(B, H, S, D), mem
    if layout == "padded":
        mem = torch.full((B, H, S + 2, D + 16), 7, dtype=dtype, device=device)
        return mem[:, :, 1:S + 1, 8:8 + D], mem
    mem = torch.full((B, H, S + 1, D), 7, dtype=dtype, device=device) if B * H == 1 else \
        torch.full((B, H, S, D), 7, dtype=dtype, device=device)
    return mem[:, :, :S], mem


def outside_kept(view, mem):
    """Whether nothing of mem but the view's elements was written."""
    was = view.clone()
    view.fill_(7)
    ok = bool((mem == 7).all())
    view.copy_(was)
    return ok


def inputs(shape, seed, spread=1.0, offset=0.3):
    g = torch.Generator().manual_seed(seed)
    B, H, S, D = shape
    x = torch.randn(shape, generator=g) * torch.exp(0.5 * torch.randn(1, H, 1, D, generator=g)) * spread
    return x + offset * torch.randn(1, H, 1, D, generator=g), torch.randn(shape, generator=g), g


def params(kind, shape, dtype, g, base):
    """(weight, bias) on the CPU."""
    B, H, S, D = shape
    if kind == "none":
        return None, None
    ps = {"weight": (D,), "shared": (D,), "batch": (B, 1, 1, D), "head": (1, H, 1, D), "both": (B, H, 1, D)}[kind]
    w = (0.3 * torch.randn(ps, generator=g) + 1 - base).to(dtype)
    return w, None if kind == "weight" else (0.2 * torch.randn(ps, generator=g)).to(dtype)
