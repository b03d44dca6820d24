"""The cases on which the row norms and the 8-bit activation checkpoints are measured.

``run`` computes a case in its plain form (elementary torch operations, fp32)
or, with ``own`` set, through the calls a training step makes: layer_norm_fwd,
layer_norm_bwd, act_pack and act_unpack.

A case names one pass: "fwd" and "bwd" are the norm's two directions, "bwd8"
the backward from an 8-bit checkpoint of the input, "step8" the forward that
also writes that checkpoint followed by the backward that reads it, "keep" a
checkpoint written and restored, "restore" the restoring alone.
"""
import math

import torch

own = False

BLOCK = 32                     # channels that share one exponent
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6


def _case(op, B, H, S, D, x, y=None, params="shared", center=True, layout="bhsd", base=0.0, name=None):
    """x, y: types of the input and of the output (or its gradient). params:
    "none", "shared" [D], "batch" [B,1,1,D] or "head" [1,H,1,D]. layout of the
    input (and of its gradient): contiguous [B,H,S,D], or "qkv", one of the
    three slices of a fused projection's [B,S,3,H,D]."""
    c = dict(op=op, B=B, H=H, S=S, D=D, x=x, y=y or x, params=params, center=center, layout=layout, base=base)
    return dict(c, name=name) if name else c


def listed():
    return [
        # per-head query norm of the oracle-scale layer, straight from its fused projection: the launch counts
        _case("fwd", 1, 1, 1024, 64, "bf16", center=False, layout="qkv", name="fwd_qk_1k"),
        # query norm of the S = 64K video layer, which also turns the projection's layout into [B,H,S,d]
        _case("fwd", 1, 24, 65536, 128, "bf16", layout="qkv", name="fwd_qk_64k"),
        # token norm over an fp32 residual stream with a modulation per clip, an odd number of tokens
        _case("fwd", 2, 1, 32767, 2048, "fp32", "bf16", params="batch", base=1.0, name="fwd_tokens_mod"),
        # a width that no vector load divides
        _case("fwd", 3, 1, 4001, 517, "fp16", name="fwd_odd_517"),
        # the small query norm's gradient
        _case("bwd", 1, 1, 1024, 64, "bf16", center=False, layout="qkv", name="bwd_qk_1k"),
        # token norm's gradient with a modulation per clip, of which each clip has its own gradient
        _case("bwd", 2, 1, 32768, 2048, "bf16", params="batch", base=1.0, name="bwd_tokens_mod"),
        # odd width, fp32, bias and weight shared by all rows
        _case("bwd", 1, 1, 9001, 1003, "fp32", name="bwd_odd_1003"),
        # query norm's gradient of a 256K-token layer from the 8-bit checkpoint of its input, weights per head
        _case("bwd8", 1, 16, 262144, 128, "bf16", params="head", center=False, name="bwd8_qk_256k"),
        # a 16K-token layer's query norm, forward with its checkpoint and backward from it
        _case("step8", 1, 8, 16384, 64, "bf16", layout="qkv", name="step8_qk_16k"),
        # values of the S = 64K layer kept in 8 bits between the forward and the backward pass
        _case("keep", 1, 24, 65536, 128, "bf16", params="none", name="keep_64k"),
        # ragged blocks: the last one of a row holds 8 channels
        _case("keep", 1, 3, 1037, 200, "fp32", params="none", layout="qkv", name="keep_ragged_200"),
        # a 256K-token layer's keys restored
        _case("restore", 1, 16, 262144, 128, "bf16", params="none", name="restore_256k"),
    ]


def draw(rng):
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "bwd8", "step8", "keep", "restore"])
    heads = rng.random() < 0.6
    B = rng.randint(1, 4)
    H = rng.randint(1, 24) if heads else 1
    D = rng.choice([64, 128, 80, 96, log(8, 256)]) if heads else log(8, 1024) * rng.choice([1, 1, 8])
    most = (1 << 27) // (B * H * D)
    S = log(1, max(2, min(most, 262144)))
    x = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    y = rng.choice(["bf16", "fp16", "fp32"]) if x == "fp32" else x
    kept = op in ("keep", "restore")
    return _case(op, B, H, S, D, x, x if kept else y, params="none" if kept else rng.choice(["none", "shared", "batch", "head"]),
                 center=rng.random() < 0.6, layout=rng.choice(["bhsd", "qkv"]) if op != "restore" else "bhsd",
                 base=rng.choice([0.0, 1.0]))


def _param_shape(c):
    return {"none": None, "shared": (c["D"],), "batch": (c["B"], 1, 1, c["D"]), "head": (1, c["H"], 1, c["D"])}[c["params"]]


def _laid(t, layout):
    """The [B,H,S,D] values of t in the case's layout."""
    if layout == "bhsd":
        return t
    B, H, S, D = t.shape
    qkv = torch.empty(B, S, 3, H, D, dtype=t.dtype, device=t.device)
    out = qkv[:, :, 1].permute(0, 2, 1, 3)
    out.copy_(t)
    return out


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    B, H, S, D = c["B"], c["H"], c["S"], c["D"]
    # projections: channels of different spread and offset, a few of them wide
    spread = torch.exp(0.5 * randn(1, H, 1, D))
    x = _laid((randn(B, H, S, D) * spread + 0.3 * randn(1, H, 1, D)).to(TYPES[c["x"]]), c["layout"])
    s = dict(c, x=x, x_type=TYPES[c["x"]], y_type=TYPES[c["y"]], weight=None, bias=None)
    shape = _param_shape(c)
    if shape is not None:
        s["weight"] = (0.2 * randn(*shape) + 1.0 - c["base"]).to(s["y_type"])
        s["bias"] = (0.1 * randn(*shape)).to(s["y_type"])
    if c["op"] in ("bwd", "bwd8", "step8"):
        s["dy"] = randn(B, H, S, D).to(s["y_type"])
        s["dx_type"] = s["y_type"] if c["op"] in ("bwd8", "step8") else s["x_type"]
        # the projection's gradient buffer, of which this call fills its slice
        s["dx"] = _laid(torch.zeros(B, H, S, D, dtype=s["dx_type"], device="cuda"), c["layout"])
    if c["op"] in ("bwd", "bwd8"):
        s["mean"], s["rstd"] = _stats(x.float(), c["center"])
        s["mean"], s["rstd"] = (v.reshape(B, H, S) if v is not None else None for v in (s["mean"], s["rstd"]))
    if c["op"] in ("bwd8", "restore"):
        s["q"], s["e"] = _pack(x)
        del s["x"]
    return s


# ------------------------------------------------------------- plain forms
def _stats(x, center):
    mean = x.mean(-1, keepdim=True) if center else None
    var = ((x - mean) if center else x).square().mean(-1, keepdim=True)
    return mean, 1.0 / torch.sqrt(var + EPS)


def _pack(x):
    """(q int8 [B,H,S,D], e uint8 [B,H,S,ceil(D/32)]): x to the nearest q 2^(e-133), ties to even."""
    x = x.float()
    D = x.shape[-1]
    nb = -(-D // BLOCK)
    xb = torch.nn.functional.pad(x, (0, nb * BLOCK - D)).reshape(*x.shape[:-1], nb, BLOCK)
    e = (xb.abs().amax(-1, keepdim=True).view(torch.int32) >> 23).clamp(min=7)
    inv = ((260 - e) << 23).view(torch.float32)              # 2^(133 - e)
    q = torch.round(xb * inv).clamp(-127, 127).to(torch.int8).reshape(*x.shape[:-1], nb * BLOCK)[..., :D]
    return q.contiguous(), e.squeeze(-1).to(torch.uint8)


def _unpack(q, e):
    step = ((e.int() - 6) << 23).view(torch.float32)         # 2^(e - 133)
    return q.float() * step.repeat_interleave(BLOCK, -1)[..., :q.shape[-1]]


def _affine(s):
    w = s["weight"].float() + s["base"] if s["weight"] is not None else 1.0
    b = s["bias"].float() if s["bias"] is not None else 0.0
    return w, b


def _rows_of(s, t):
    """Sum over the rows that share one row of parameters."""
    if s["weight"] is None:
        return None
    return t.sum({"shared": (0, 1, 2), "batch": (1, 2), "head": (0, 2)}[s["params"]]).reshape(s["weight"].shape)


def _fwd(s, x):
    mean, rstd = _stats(x, s["center"])
    w, b = _affine(s)
    xhat = (x - mean if mean is not None else x) * rstd
    return (xhat * w + b).to(s["y_type"]), mean.squeeze(-1) if mean is not None else None, rstd.squeeze(-1)


def _bwd(s, dy, x, mean, rstd):
    w, _ = _affine(s)
    rstd = rstd.unsqueeze(-1)
    xhat = (x - mean.unsqueeze(-1) if mean is not None else x) * rstd
    dy = dy.float()
    g = dy * w
    c2 = (g * xhat).mean(-1, keepdim=True)
    dx = g - xhat * c2
    if s["center"]:
        dx = dx - g.mean(-1, keepdim=True)
    return (dx * rstd).to(s["dx_type"]), _rows_of(s, dy * xhat), _rows_of(s, dy)


def _outputs(**named):
    return {k: v for k, v in named.items() if v is not None}


def run(state):
    s = state
    if own:
        return _run_own(s)
    op = s["op"]
    if op == "fwd":
        y, mean, rstd = _fwd(s, s["x"].float())
        return _outputs(y=y, mean=mean, rstd=rstd)
    if op in ("bwd", "bwd8"):
        x = s["x"].float() if op == "bwd" else _unpack(s["q"], s["e"])
        dx, dw, db = _bwd(s, s["dy"], x, s["mean"], s["rstd"])
        return _outputs(dx=dx, dweight=dw, dbias=db)
    if op == "step8":
        y, mean, rstd = _fwd(s, s["x"].float())
        dx, dw, db = _bwd(s, s["dy"], _unpack(*_pack(s["x"])), mean, rstd)
        return _outputs(y=y, mean=mean, rstd=rstd, dx=dx, dweight=dw, dbias=db)
    q, e = _pack(s["x"]) if op == "keep" else (s["q"], s["e"])
    return {"x": _unpack(q, e).to(s["x_type"])}


# ---------------------------------------------------------- the framework's
def _run_own(s):
    import dynamic_sparse_attention_dsv_gb300 as dsv
    op, affine = s["op"], dict(weight=s["weight"], bias=s["bias"], weight_base=s["base"])
    if op in ("fwd", "step8"):
        y, mean, rstd, kept = dsv.layer_norm_fwd(s["x"], eps=EPS, center=s["center"], dtype=s["y_type"],
                                                 pack=op == "step8", **affine)
        if op == "fwd":
            return _outputs(y=y, mean=mean, rstd=rstd)
        dx, dw, db = dsv.layer_norm_bwd(s["dy"], kept, mean, rstd, dx=s["dx"], **affine)
        return _outputs(y=y, mean=mean, rstd=rstd, dx=dx, dweight=dw, dbias=db)
    if op in ("bwd", "bwd8"):
        x = s["x"] if op == "bwd" else dsv.PackedAct(s["q"], s["e"])
        dx, dw, db = dsv.layer_norm_bwd(s["dy"], x, s["mean"], s["rstd"], dx=s["dx"], **affine)
        return _outputs(dx=dx, dweight=dw, dbias=db)
    kept = dsv.act_pack(s["x"]) if op == "keep" else dsv.PackedAct(s["q"], s["e"])
    return {"x": dsv.act_unpack(kept, dtype=s["x_type"])}


def work(case):
    c = case
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    rows = c["B"] * c["H"] * c["S"]
    n, x, y = rows * c["D"], size[c["x"]], size[c["y"]]
    kept = n + rows * -(-c["D"] // BLOCK)
    stats = rows * (8 if c["center"] else 4)
    shape = _param_shape(c)
    p = math.prod(shape) if shape else 0
    fwd = n * (x + y) + stats + 2 * p * y
    bwd = n * y + stats + p * (y + 8)
    return {"fwd": dict(bytes=fwd, flops=8 * n),
            "bwd": dict(bytes=bwd + 2 * n * x, flops=14 * n),
            "bwd8": dict(bytes=bwd + kept + n * y, flops=16 * n),
            "step8": dict(bytes=fwd + bwd + 2 * kept + n * y, flops=28 * n),
            "keep": dict(bytes=2 * n * x + 2 * kept, flops=6 * n),
            "restore": dict(bytes=n * x + kept, flops=n)}[c["op"]]


# ------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op, D, center = s["op"], s["D"], s["center"]
    f64 = lambda t: t.to(torch.float64)  # noqa: E731
    x = f64(s["x"]) if "x" in s else None
    if op in ("keep", "step8"):
        kept = torch.empty_like(x)
        for lo in range(0, D, BLOCK):
            part = x[..., lo:lo + BLOCK]
            _, power = torch.frexp(part.abs().amax(-1, keepdim=True))       # top in [2^(power-1), 2^power)
            step = torch.exp2((power - 1).clamp(min=-120).double() - 6)
            kept[..., lo:lo + BLOCK] = torch.round(part / step).clamp(-127, 127) * step
    elif op in ("bwd8", "restore"):
        kept = torch.empty_like(s["q"], dtype=torch.float64)
        for b in range(s["e"].shape[-1]):
            at = slice(b * BLOCK, (b + 1) * BLOCK)
            kept[..., at] = f64(s["q"][..., at]) * torch.exp2(f64(s["e"][..., b:b + 1]) - 133)
    if op in ("keep", "restore"):
        return {"x": kept}
    gain = f64(s["weight"]) + s["base"] if s["weight"] is not None else torch.ones(D, dtype=torch.float64, device="cuda")
    found = {}
    if op in ("fwd", "step8"):
        mean = x.sum(-1) / D if center else torch.zeros(x.shape[:-1], dtype=torch.float64, device="cuda")
        dev = x - mean[..., None]
        rstd = (torch.einsum("bhsd,bhsd->bhs", dev, dev) / D + EPS) ** -0.5
        y = dev * rstd[..., None] * gain
        found = {"y": y + f64(s["bias"]) if s["bias"] is not None else y, "rstd": rstd}
        if center:
            found["mean"] = mean
        if op == "fwd":
            return found
    else:
        mean = f64(s["mean"]) if center else torch.zeros(s["rstd"].shape, dtype=torch.float64, device="cuda")
        rstd = f64(s["rstd"])
    u = (kept if op != "bwd" else x) - mean[..., None]
    u *= rstd[..., None]
    dy = f64(s["dy"])
    back = dy * gain
    along = torch.einsum("bhsd,bhsd->bhs", back, u) / D
    found["dx"] = back - u * along[..., None]
    if center:
        found["dx"] -= back.sum(-1, keepdim=True) / D
    found["dx"] *= rstd[..., None]
    if s["weight"] is not None:
        over = {"shared": "d", "batch": "bd", "head": "hd"}[s["params"]]
        found["dweight"] = torch.einsum("bhsd,bhsd->" + over, dy, u).reshape(s["weight"].shape)
        found["dbias"] = torch.einsum("bhsd->" + over, dy).reshape(s["weight"].shape)
    return found
