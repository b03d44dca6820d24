"""What the row calls refuse, through the C ABI and in the binding. Pointers are
made up, so every call here has to be one that is refused before a launch."""
import ctypes

import pytest
import torch

import dynamic_sparse_attention_dsv_gb300 as dsv
from dynamic_sparse_attention_dsv_gb300 import native as N
from dynamic_sparse_attention_dsv_gb300 import rows as R

A = 1 << 20                       # any aligned address: nothing reads it
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
NONE = N.dsv_rows(None, None, N.DSV_PACKED, 0, 0, 0)


def ext(B=2, H=3, S=5, D=64):
    return N.dsv_extent(B, H, S, D)


def rows(n=None, type=N.DSV_BF16, data=A, exp=None, strides=None):
    n = n or ext()
    st = strides or (n.H * n.S * n.D, n.S * n.D, n.D)
    return N.dsv_rows(data, exp, type, *st)


def packed(data=A, exp=A):
    return N.dsv_rows(data, exp, N.DSV_PACKED, 0, 0, 0)


def par(weight=None, bias=None, type=N.DSV_FP32, per=(0, 0), strides=(0, 0, 0, 0), base=0.0):
    return N.dsv_norm_params(weight, bias, type, *per, *strides, base)


@pytest.fixture(scope="module")
def lib():
    return N.load()


def fwd(lib, x=None, n=None, p=None, eps=1e-6, y=None, mean=A, rstd=A, pack=NONE):
    return lib.dsv_layer_norm_fwd(x or rows(n), n or ext(), p or par(), eps, 1, y or rows(n), mean, rstd, pack, None)


def bwd(lib, dy=None, x=None, n=None, p=None, mean=A, rstd=A, dx=None, dw=A, db=A, ws=A, ws_bytes=1 << 40):
    return lib.dsv_layer_norm_bwd(dy or rows(n), x or rows(n), n or ext(), p or par(), mean, rstd, dx or rows(n), dw, db, ws,
                                  ws_bytes, None)


@pytest.mark.parametrize("n,code", [(ext(B=-1), INVALID), (ext(D=0), INVALID), (ext(D=8193), UNSUPPORTED),
                                    (ext(B=1 << 31, H=0), UNSUPPORTED), (ext(B=1 << 16, H=1 << 15), UNSUPPORTED),
                                    (ext(B=1 << 30, H=1 << 30, S=1 << 30), UNSUPPORTED),
                                    (ext(B=1 << 20, H=8, S=8, D=8192), UNSUPPORTED)])
def test_extents(lib, n, code):
    assert fwd(lib, n=n) == code and bwd(lib, n=n) == code
    assert lib.dsv_act_pack(rows(n), n, packed(), None) == code
    assert lib.dsv_act_unpack(packed(), n, rows(n), None) == code
    assert lib.dsv_layer_norm_bwd_workspace_size(n, 1, 1) == 0


@pytest.mark.parametrize("bad", [rows(data=None), rows(data=A + 1), rows(type=7), rows(exp=A), rows(strides=(-64, 64, 64)),
                                 rows(strides=(1 << 57, 64, 64)), packed(data=None), packed(exp=None), packed(data=A + 4)])
def test_tensors(lib, bad):
    assert fwd(lib, x=bad) == INVALID and fwd(lib, y=bad) == INVALID
    assert bwd(lib, x=bad) == INVALID and bwd(lib, dy=bad) == INVALID and bwd(lib, dx=bad) == INVALID
    if bad.type == N.DSV_PACKED:
        assert lib.dsv_act_pack(rows(), ext(), bad, None) == INVALID and lib.dsv_act_unpack(bad, ext(), rows(), None) == INVALID
        if bad.data:              # data NULL asks for no checkpoint
            assert fwd(lib, pack=bad) == INVALID
    else:
        assert lib.dsv_act_pack(bad, ext(), packed(), None) == INVALID
        assert lib.dsv_act_unpack(packed(), ext(), bad, None) == INVALID


@pytest.mark.parametrize("strides", [(0, 320, 64), (960, 320, 32), (960, 64, 64), (64, 64, 64), (320, 320, 64)])
def test_output_rows_may_not_overlap(lib, strides):
    over = rows(strides=strides)
    assert fwd(lib, y=over) == INVALID and bwd(lib, dx=over) == INVALID
    assert lib.dsv_act_unpack(packed(), ext(), over, None) == INVALID


def test_types(lib):
    f16, f32 = rows(type=N.DSV_FP16), rows(type=N.DSV_FP32)
    assert fwd(lib, y=f16) == UNSUPPORTED and fwd(lib, y=f32) == UNSUPPORTED     # bf16 in, another type out
    assert fwd(lib, y=packed()) == INVALID and bwd(lib, dy=packed()) == INVALID and bwd(lib, dx=packed()) == INVALID
    assert bwd(lib, dx=f32) == INVALID                                           # dx has x's type
    assert bwd(lib, dy=f32, dx=rows()) == UNSUPPORTED
    assert bwd(lib, x=packed(), dx=f32) == INVALID                               # dx has dy's type
    assert fwd(lib, x=packed(), pack=packed()) == INVALID                        # kept already
    assert fwd(lib, pack=rows()) == INVALID
    assert lib.dsv_act_pack(packed(), ext(), packed(), None) == INVALID
    assert lib.dsv_act_pack(rows(), ext(), rows(), None) == INVALID


def test_numbers_and_parameters(lib):
    for eps in (0.0, -1e-6, float("nan"), float("inf")):
        assert fwd(lib, eps=eps) == INVALID
    assert fwd(lib, mean=A + 2) == INVALID and fwd(lib, rstd=A + 2) == INVALID
    assert bwd(lib, rstd=None) == INVALID and bwd(lib, dw=A + 1) == INVALID and bwd(lib, mean=A + 1) == INVALID
    for p in (par(weight=A, type=N.DSV_PACKED), par(weight=A + 2), par(bias=A + 2), par(weight=A, base=float("nan")),
              par(weight=A, base=float("inf")), par(weight=A, per=(1, 0), strides=(-1, 0, 0, 0)),
              par(bias=A, per=(0, 1), strides=(0, 0, 0, 1 << 50))):
        assert fwd(lib, p=p) == INVALID and bwd(lib, p=p) == INVALID


def test_workspace(lib):
    n = ext(1, 4, 3000, 128)
    need = lib.dsv_layer_norm_bwd_workspace_size(n, 0, 0)
    assert need > 0
    assert bwd(lib, n=n, ws_bytes=need - 1) == WORKSPACE and bwd(lib, n=n, ws=None) == WORKSPACE
    assert bwd(lib, n=n, ws=A + 8) == WORKSPACE
    # it holds sums of the thread blocks, not of the rows
    many = lib.dsv_layer_norm_bwd_workspace_size(ext(4, 24, 65536, 128), 0, 0)
    assert many < 16 << 20
    # one row is one block, which writes its sums as the result
    assert lib.dsv_layer_norm_bwd_workspace_size(ext(1, 1, 1, 128), 1, 1) == 0


def test_nothing_to_do(lib):
    """No rows: accepted without a launch, whatever the pointers."""
    n = ext(S=0)
    none = rows(n, data=None)
    assert fwd(lib, n=n, x=none, y=none) == 0
    assert lib.dsv_act_pack(none, n, NONE, None) == 0 and lib.dsv_act_unpack(NONE, n, none, None) == 0
    assert bwd(lib, n=n, dy=none, x=none, dx=none, dw=None, db=None, ws=None, ws_bytes=0) == 0


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 3, 64, dtype=torch.bfloat16)
    for call in (lambda: dsv.layer_norm_fwd(x), lambda: dsv.layer_norm_bwd(x, x, None, x[..., 0].float()),
                 lambda: dsv.act_pack(x), lambda: dsv.act_unpack(dsv.PackedAct(x.to(torch.int8), x.to(torch.uint8))),
                 lambda: dsv.act_unpack(x), lambda: dsv.act_pack("x")):
        with pytest.raises(ValueError):
            call()


def test_structures_match_the_header():
    assert ctypes.sizeof(N.dsv_rows) == 48 and ctypes.sizeof(N.dsv_norm_params) == 72 and ctypes.sizeof(N.dsv_extent) == 32


def test_binding_is_required(monkeypatch, tmp_path):
    """No fallback: without its native binding a row call raises."""
    monkeypatch.setattr(R, "_binding", None)
    monkeypatch.setattr(R, "BINDING_PATH", str(tmp_path / "_rows.so"))
    with pytest.raises(RuntimeError, match="not built"):
        dsv.act_pack(torch.zeros(2, 3, 64))


def test_packed_backward(lib):
    """dsv_sparse_attn_bwd_packed: what it refuses, and its workspace beside the backward's."""
    s, g = N.dsv_shape(1, 2, 8, 16, 16, 128), N.dsv_group(2, 8, 8)
    ks, offs = (ctypes.c_int32 * 2)(100, 100), (ctypes.c_int64 * 2)(0, 100 * 16)
    own, least = (f(s, g, ks, offs) for f in (lib.dsv_sparse_attn_bwd_workspace_size, lib.dsv_sparse_attn_bwd_min_workspace_size))
    one = 2 * 2 * 2048 * 128
    for n in range(5):
        assert lib.dsv_sparse_attn_bwd_packed_workspace_size(s, g, ks, offs, n) == own + n * one
        assert lib.dsv_sparse_attn_bwd_packed_min_workspace_size(s, g, ks, offs, n) == least + n * one
    assert lib.dsv_sparse_attn_bwd_packed_workspace_size(s, g, ks, offs, 5) == 0
    bf = N.dsv_rows(A, None, N.DSV_BF16, 0, 0, 0)

    def call(Q=packed(), K=packed(), V=bf, O=packed(), LSE=A, dO=A, idx=A, k=ks, o=offs, shape=s, scale=0.1, dK=A, ws=A,
             size=least + 3 * one):
        return lib.dsv_sparse_attn_bwd_packed(Q, K, V, O, LSE, dO, idx, k, o, shape, g, scale, A, dK, A, ws, size, None, None)

    assert call(size=least + 3 * one - 1) == WORKSPACE and call(ws=None) == WORKSPACE and call(ws=A + 64) == WORKSPACE
    for bad in (dict(Q=rows(type=N.DSV_FP16)), dict(V=N.dsv_rows(A, A, N.DSV_BF16, 0, 0, 0)), dict(K=packed(exp=None)),
                dict(O=packed(data=None)), dict(O=packed(data=A + 4)), dict(K=packed(data=A + 8)), dict(V=N.dsv_rows(A + 8, None, N.DSV_BF16, 0, 0, 0)),
                dict(V=N.dsv_rows(None, None, N.DSV_BF16, 0, 0, 0)), dict(LSE=None), dict(dO=A + 8), dict(scale=0.0),
                dict(k=None), dict(dK=None), dict(k=(ctypes.c_int32 * 2)(100, 4096))):
        assert call(**bad) == INVALID, bad
    assert call(shape=N.dsv_shape(1, 2, 8, 16, 16, 96)) == UNSUPPORTED
