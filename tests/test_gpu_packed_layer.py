"""The row calls where an attention layer uses them: the sparse backward from
8-bit checkpoints, and a layer's training step from its fused projection to the
projection's gradient."""
import math

import numpy as np
import pytest
import torch

import dynamic_sparse_attention_dsv_gb300 as dsv
from dynamic_sparse_attention_dsv_gb300 import synthetic as syn
from oracle import dsv_oracle as ora
from oracle import rows_oracle as rora

from .parity import GRAD_REL_L2, rel_l2

pytestmark = pytest.mark.gpu

W = {
    "oracle_scale": syn.workload(0, backward=True),
    "ragged_d128": syn.Workload("ragged", 101, 2, 4, 16, 32, 128, 32, 2, 8, 8, 300, ("uniform", 2.0, 8.0), True),
}


def _forward(w, dense=False):
    d = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in syn.make_inputs(w).items()}
    grid, group = (w.T, w.Y, w.X), (w.gt, w.gy, w.gx)
    idx = ks = offs = None
    if not dense:
        idx, ks, offs = dsv.lowrank_topk(d["Q"], d["K"], d["Wq"], d["Wk"], grid, group, w.k)
    O, L = dsv.sparse_attn_fwd(d["Q"], d["K"], d["V"], idx, ks, offs, grid, group)
    return d, O, L, (idx, ks, offs, grid, group)


@pytest.mark.parametrize("dense", [False, True])
@pytest.mark.parametrize("which", ["QKVO", "QO", "V", "K"])
@pytest.mark.parametrize("name", list(W))
def test_packed_backward_is_the_backward_of_the_restored(name, which, dense):
    w = W[name]
    d, O, L, plan = _forward(w, dense)
    kept = dict(Q=d["Q"], K=d["K"], V=d["V"], O=O)
    kept = {k: dsv.act_pack(t) if k in which else t for k, t in kept.items()}
    back = {k: dsv.act_unpack(t) if k in which else t for k, t in kept.items()}
    st = dsv.new_status()
    got = dsv.sparse_attn_bwd(kept["Q"], kept["K"], kept["V"], kept["O"], L, d["dO"], *plan, status=st)
    ref = dsv.sparse_attn_bwd(back["Q"], back["K"], back["V"], back["O"], L, d["dO"], *plan, status=st)
    dsv.check_status(st, "packed backward")
    assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_packed_backward_workspaces():
    """The smallest workspace gives the same bits; one byte less is refused before anything is written."""
    w = W["ragged_d128"]
    d, O, L, plan = _forward(w)
    idx, ks, offs, grid, group = plan
    kept = [dsv.act_pack(t) for t in (d["Q"], d["K"], d["V"], O)]
    ref = dsv.sparse_attn_bwd(*kept, L, d["dO"], *plan)
    least = dsv.sparse_attn_bwd_packed_min_workspace_size(O, grid, group, ks, offs)
    full = dsv.sparse_attn_bwd_packed_workspace_size(O, grid, group, ks, offs)
    assert least < full
    assert least - dsv.sparse_attn_bwd_min_workspace_size(O, grid, group, ks, offs) == 4 * O.numel() * 2
    for n in (least, full):
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        got = dsv.sparse_attn_bwd(*kept, L, d["dO"], *plan, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
    ws = torch.full((least,), 7, dtype=torch.uint8, device="cuda")
    with pytest.raises(dsv.DsvError) as err:
        dsv.sparse_attn_bwd(*kept, L, d["dO"], *plan, workspace=ws[:least - 256])
    assert err.value.code == 3 and bool((ws == 7).all())
    with pytest.raises(dsv.DsvError) as err:      # refused by the backward's own checks, before the restoring
        dsv.sparse_attn_bwd(*kept, L, d["dO"], idx, [w.S + 1] * w.H, offs, grid, group, workspace=ws)
    assert err.value.code == 1 and bool((ws == 7).all())


def _bwd64(q, k, v, o, lse, do, idx, mem, scale):
    """dQ, dK, dV in fp64 at the values and the LSE given (numpy, one head)."""
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for g in range(mem.shape[0]):
        m, i = mem[g], idx[g]
        p = np.exp(scale * q[m] @ k[i].T - lse[m][:, None])
        ds = p * (do[m] @ v[i].T - (do[m] * o[m]).sum(-1, keepdims=True))
        dq[m] = scale * ds @ k[i]
        np.add.at(dk, i, scale * ds.T @ q[m])
        np.add.at(dv, i, p.T @ do[m])
    return dq, dk, dv


@pytest.mark.parametrize("center", [False, True])
def test_layer_step(center):
    """One layer's training step as a user runs it: Q and K normed straight from
    the fused projection with their inputs' checkpoints written on the way, top-k
    and sparse attention, V, O and the normed Q, K kept in 8 bits, the backward
    from the checkpoints, and the norms' gradients written into the projection's."""
    w = W["ragged_d128"]
    H, S, D = w.H, w.S, w.d
    inp = syn.make_inputs(w)
    grid, group = (w.T, w.Y, w.X), (w.gt, w.gy, w.gx)
    g = torch.Generator().manual_seed(9)
    qkv = torch.empty(1, S, 3, H, D, dtype=torch.bfloat16, device="cuda")
    for i, n in enumerate("QKV"):
        qkv[0, :, i] = inp[n].permute(1, 0, 2).cuda()
    q, k, v = (qkv[:, :, i].permute(0, 2, 1, 3) for i in range(3))
    par = [(torch.rand(D, generator=g) + 0.5).to(torch.bfloat16).cuda() for _ in range(4)]
    gain, shift = (par[0], par[1]), (par[2], par[3]) if center else (None, None)
    Wq, Wk, dO = inp["Wq"].cuda(), inp["Wk"].cuda(), inp["dO"].cuda().view(1, H, S, D)

    normed = [dsv.layer_norm_fwd(t, gain[i], shift[i], center=center, pack=True) for i, t in enumerate((q, k))]
    qn, kn = normed[0][0], normed[1][0]
    vn = v.contiguous()
    st = dsv.new_status()
    idx, ks, offs = dsv.lowrank_topk(qn, kn, Wq, Wk, grid, group, w.k, status=st)
    O, L = dsv.sparse_attn_fwd(qn, kn, vn, idx, ks, offs, grid, group, status=st)
    kept = [dsv.act_pack(t) for t in (qn, kn, vn, O)]
    dqn, dkn, dv = dsv.sparse_attn_bwd(*kept, L, dO, idx, ks, offs, grid, group, status=st)
    dqkv = torch.full_like(qkv, float("nan"))
    dq_in, dk_in, dv_in = (dqkv[:, :, i].permute(0, 2, 1, 3) for i in range(3))
    grads = []
    for i, (dy, out) in enumerate(((dqn, dq_in), (dkn, dk_in))):
        _, mean, rstd, x8 = normed[i]
        grads.append(dsv.layer_norm_bwd(dy, x8, mean, rstd, gain[i], shift[i], dx=out))
    dv_in.copy_(dv)
    dsv.check_status(st, "layer step")
    assert torch.isfinite(dqkv).all()

    # the norms against the oracle
    scale = 1.0 / math.sqrt(D)
    mem = ora.group_members(w.T, w.Y, w.X, w.gt, w.gy, w.gx)
    for i, t in enumerate((q, k)):
        b = shift[i].cpu() if center else None
        ref, _, _ = rora.norm_fwd(t.cpu(), gain[i].cpu(), b, 1e-6, center, 0.0)
        assert rel_l2(normed[i][0].double().cpu().numpy(), ref.numpy()) < 2 ** -8
    # the attention's gradients at the restored values
    rows = [idx[offs[h]: offs[h] + w.n_groups * w.k].view(w.n_groups, w.k).cpu().numpy().astype(np.int64) for h in range(H)]
    back = [dsv.act_unpack(t, dtype=torch.float32)[0].double().cpu().numpy() for t in kept]
    for h in range(H):
        ref = _bwd64(*(b[h] for b in back), L[0, h].double().cpu().numpy(), dO[0, h].double().cpu().numpy(), rows[h], mem, scale)
        for got, r in zip((dqn, dkn, dv), ref):
            assert rel_l2(got[0, h].double().cpu().numpy(), r) < GRAD_REL_L2
    # the norms' gradients at the restored inputs
    for i, (dy, out) in enumerate(((dqn, dq_in), (dkn, dk_in))):
        _, mean, rstd, x8 = normed[i]
        x = rora.unpack(x8.q.cpu().long(), x8.e.cpu().long())
        ref = rora.norm_bwd(dy.cpu(), x, mean.cpu() if center else None, rstd.cpu(), gain[i].cpu(),
                            shift[i].cpu() if center else None, 0.0)
        assert rel_l2(out.double().cpu().numpy(), ref[0].numpy()) < 2 ** -8
        assert rel_l2(grads[i][1].double().cpu().numpy(), ref[1].numpy()) < 1e-5
