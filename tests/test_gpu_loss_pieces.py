"""Losses through the head in pieces of the vocabulary: the logits are computed again
piece by piece.  Small shapes are brought to it by the size of their workspace, and
checked as test_gpu_losses.py checks the others."""

import numpy as np
import pytest
import torch

from oracle import dense_labels, dense_teacher
from test_gpu_losses import BF16, DEV, F16, F32, check_head, f64, half_step, head_inputs, ssv  # noqa: F401

pytestmark = pytest.mark.gpu

CASES = [
    # N, V, H, dtype, grad dtype, T, k (0: cross entropy), reduction, weighted
    (300, 6100, 712, BF16, BF16, 0.8, 20, "mean", True),    # three pieces, lists across their borders, two splits
    (300, 6100, 712, F16, F16, 0.8, 20, "mean", True),
    (129, 6144, 264, F16, F32, 1.7, 0, "sum", True),
    (257, 4099, 520, BF16, F32, 1.0, 0, "mean", True),      # a last piece of a few tokens
    (33, 20011, 1024, F16, F16, 1.0, 64, "mean", False),
    (7, 9000, 72, BF16, BF16, 0.7, 256, "sum", True),
    (1, 5000, 64, F16, F32, 1.0, 3, "mean", False),
    (700, 4097, 136, BF16, BF16, 1.0, 0, "sum", False),     # a last piece of one token
]


@pytest.mark.parametrize("N,V,H,dt,gdt,T,k,red,weighted", CASES)
def test_head_with_a_bounded_workspace(ssv, N, V, H, dt, gdt, T, k, red, weighted):  # noqa: F811
    x, w, y, rw = head_inputs(N, V, H, dt, N + V + H)
    xd, wd, rd = x.to(DEV), w.to(DEV), rw.to(DEV) if weighted else None
    scale = 2.0 if dt == BF16 else 2.0 * 512
    if k == 0:
        y[::3] = -100
        target = dense_labels(y.numpy(), V, -100)
        a, both = (xd, wd, y.to(DEV), T), ssv.linear_cross_entropy_fwd_bwd
    else:
        full = f64(x) @ f64(w).T + np.random.Generator(np.random.PCG64(1)).normal(0, 0.5, (N, V))
        ids = np.argsort(-full, axis=1)[:, :k].astype(np.int32)
        ids[:, -1] = np.arange(N) % 3 + np.where(np.arange(N) % 2, 2046, 4094)  # next to borders of pieces
        ids[:, -1] = np.where((ids[:, :-1] == ids[:, -1:]).any(1), -1, ids[:, -1])
        tx = np.take_along_axis(full, np.maximum(ids, 0), axis=1).astype(np.float32)
        if N > 4:
            ids[::3, : k // 2] = -1
            ids[1] = -1
        target = dense_teacher(ids, tx, T, V)
        a = (xd, wd, torch.from_numpy(ids).to(DEV), torch.from_numpy(tx).to(DEV), T)
        both = ssv.linear_topk_distill_fwd_bwd
    kw = dict(row_weight=rd, reduction=red, grad_dtype=gdt)
    full = both(*a, scale, **kw)
    for gh, gw in ((True, True), (True, False), (False, True)):
        size = [ssv.linear_loss_workspace_bytes(N, V, H, dt, max(k, 1), want_grad_hidden=gh, want_grad_weight=gw, least=b)
                for b in (True, False)]
        assert size[0] < size[1]
        for nbytes in (size[0], (size[0] + size[1]) // 2, size[1] - 1):
            ws = torch.full((nbytes,), 255, dtype=torch.uint8, device=DEV)
            o = both(*a, scale, want_grad_hidden=gh, want_grad_weight=gw, workspace=ws, **kw)
            torch.cuda.synchronize()
            assert int(o.status) == 0
            assert torch.equal(o.loss, full.loss) and torch.equal(o.row_loss, full.row_loss) and torch.equal(o.lse, full.lse)
            if gh and gw:
                check_head(o, x, w, target, T, rw.numpy() if weighted else None, red, scale, gdt)
            elif nbytes == size[0]:  # the same pieces as with both gradients
                least = both(*a, scale, workspace=torch.empty(ssv.linear_loss_workspace_bytes(
                    N, V, H, dt, max(k, 1), least=True), dtype=torch.uint8, device=DEV), **kw)
                assert gh == (o.grad_hidden is not None) and gw == (o.grad_weight is not None)
                assert (torch.equal(o.grad_hidden, least.grad_hidden) if gh
                        else torch.equal(o.grad_weight, least.grad_weight))
    with pytest.raises(ssv.SpecError):
        both(*a, scale, workspace=torch.empty(size[0] // 2, dtype=torch.uint8, device=DEV), **kw)


@pytest.mark.parametrize("dt", [BF16, F16])
def test_left_out_rows_may_hold_anything_in_pieces(ssv, dt):  # noqa: F811
    N, V, H, kept = 300, 4500, 72, 65
    x, w, y, rw = head_inputs(N, V, H, dt, 3)
    order = torch.randperm(N, generator=torch.Generator().manual_seed(3))
    y[order[kept:]] = -100
    clean = x.clone()
    clean[y < 0] = 0
    x[y < 0] = torch.tensor([float("nan"), float("inf"), -float("inf"), 7.0], dtype=dt).repeat(H // 4)
    ws = torch.empty(ssv.linear_loss_workspace_bytes(N, V, H, dt, least=True), dtype=torch.uint8, device=DEV)
    kw = dict(row_weight=rw.to(DEV), reduction="sum", grad_dtype=F32, workspace=ws)
    o = ssv.linear_cross_entropy_fwd_bwd(x.to(DEV), w.to(DEV), y.to(DEV), 1.0, 64.0, **kw)
    c = ssv.linear_cross_entropy_fwd_bwd(clean.to(DEV), w.to(DEV), y.to(DEV), 1.0, 64.0, **kw)
    torch.cuda.synchronize()
    assert torch.equal(o.grad_hidden, c.grad_hidden) and torch.equal(o.grad_weight, c.grad_weight)
    check_head(c, clean, w, dense_labels(y.numpy(), V, -100), 1.0, rw.numpy(), "sum", 64.0, F32)


@pytest.mark.parametrize("dt,least", [(F16, False), (BF16, True)])
def test_a_batch_that_is_cut_by_itself(ssv, dt, least):  # noqa: F811
    """An fp16 batch of more than 4 GB (and a bf16 one bounded to the least workspace), weighted, at T = 0.8, with
    several pieces and several splits, against fp64 products on the GPU."""
    N, V, H, T = 5500, 151936, 256, 0.8
    g = torch.Generator(device=DEV).manual_seed(4)
    w = (torch.randn(V, H, generator=g, device=DEV) * (2.0 / H ** 0.5)).to(dt)
    y = torch.randint(0, V, (N,), generator=g, device=DEV)
    x = (torch.randn(N, H, generator=g, device=DEV) + 2 * w[y].float()).to(dt)
    y = torch.where(torch.rand(N, generator=g, device=DEV) < 0.2, -100, y)
    rw = 0.8 ** torch.randint(0, 7, (N,), generator=g, device=DEV).float()
    scale = 256.0
    ws = None
    if least:
        ws = torch.empty(ssv.linear_loss_workspace_bytes(N, V, H, dt, least=True), dtype=torch.uint8, device=DEV)
    o = ssv.linear_cross_entropy_fwd_bwd(x, w, y.int(), T, scale, row_weight=rw, reduction="sum", grad_dtype=F32,
                                         workspace=ws)
    torch.cuda.synchronize()
    assert int(o.status) == 0
    X, W = x.double(), w.double()
    gw, tw = torch.zeros_like(W), torch.zeros_like(W)
    u, E = half_step(dt), 2e-5
    tiny = 2.0 ** -25 / 2.0 ** 15 if dt == F16 else 0.0
    for r in range(0, N, 500):
        rows = slice(r, r + 500)
        z = X[rows] @ W.T / T
        lse = torch.logsumexp(z, dim=1)
        dz = (H / 16 + 1) * 2.0 ** -23 * (X[rows].abs() @ W.abs().T).amax(dim=1) / T
        keep = y[rows] >= 0
        c = (scale * rw[rows].double() * keep / T)[:, None]
        q = torch.exp(z - lse[:, None])
        t = torch.zeros_like(q)
        t[torch.nonzero(keep)[:, 0], y[rows][keep]] = 1.0
        d = (q - t) * c
        err = c * (q + t) * (2 * dz[:, None] + E) + u * d.abs() + tiny * scale / T * keep[:, None]
        size = d.abs() + err
        gx = d @ W
        tol = err @ W.abs() + (V / 16 + V / 1024 + 40) * 2.0 ** -23 * (size @ W.abs()) + half_step(F32) * gx.abs()
        assert ((o.grad_hidden[rows].double() - gx).abs() <= tol).all()
        gw += d.T @ X[rows]
        tw += err.T @ X[rows].abs() + (N / 16 + 40) * 2.0 ** -23 * (size.T @ X[rows].abs())
    assert ((o.grad_weight.double() - gw).abs() <= tw + half_step(F32) * gw.abs()).all()
