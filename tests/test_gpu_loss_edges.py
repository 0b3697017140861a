"""Edges of the drafter-training losses: infinite losses, masked tiles, weights at the
end of the range, batches that reuse every buffer of a kernel.  Oracle and tolerances
are those of test_gpu_losses.py."""

import threading

import numpy as np
import pytest
import torch

from oracle import dense_labels, dense_teacher, listed_loss
from test_gpu_losses import (BAD_LOGITS, BF16, DEV, E, F16, F32, check_head, check_kd, f64, head_inputs, kd_inputs,
                             ssv)  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [3, 8, 9, 40, 5000])
@pytest.mark.parametrize("red", ["mean", "sum"])
def test_infinite_row_losses_make_the_loss_infinite(ssv, N, red):  # noqa: F811
    """A student that gives a listed token no mass has an infinite loss, and so has
    its batch; only opposite infinities make NaN."""
    V, k = 64, 3
    z, ids, x, lse, w = kd_inputs(N, V, k, F32, N, 1.0)
    z[1, ids[1, 0].long()] = float("-inf")
    w[2] = -0.5
    d = [t.to(DEV) for t in (z, ids, x, w)]
    o = ssv.topk_distill_fwd_bwd(*d[:3], 1.0, row_weight=d[3], reduction=red)
    r = listed_loss(f64(z), dense_teacher(ids.numpy(), x.numpy(), 1.0, V), 1.0, row_weight=w.numpy(), reduction=red)
    assert np.isposinf(r.loss) and float(o.loss) == float("inf") and int(o.status) == 0
    z[2, ids[2, 1].long()] = float("-inf")
    o = ssv.topk_distill(z.to(DEV), *d[1:3], 1.0, row_weight=d[3], reduction=red)
    assert np.isnan(float(o.loss)) and np.isposinf(f64(o.row_loss)[1:3]).all()
    w[1] = -1.0
    o = ssv.topk_distill(z.to(DEV), *d[1:3], 1.0, row_weight=w.to(DEV), reduction=red)
    assert float(o.loss) == float("-inf")


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("N", [4, 30])
def test_rows_masked_with_the_lowest_value_keep_their_loss(ssv, dt, N):  # noqa: F811
    """One token left that the teacher does not list: a large and finite loss."""
    V, k = 500, 3
    z, ids, x, lse, w = kd_inputs(N, V, k, dt, 11, 1.0)
    z[1, torch.arange(V) != 17] = torch.finfo(dt).min
    ids[1] = torch.tensor([3, 4, 5])
    o = ssv.topk_distill_fwd_bwd(*(t.to(DEV) for t in (z, ids, x)), 1.0, reduction="sum")
    r = listed_loss(f64(z), dense_teacher(ids.numpy(), x.numpy(), 1.0, V), 1.0, reduction="sum")
    assert (np.abs(f64(o.row_loss) - r.row_loss) <= E + 2e-6 * np.abs(r.row_loss)).all()
    assert abs(float(o.loss) - r.loss) <= E * N + 4e-6 * abs(r.loss)


@pytest.mark.parametrize("cut", [slice(0, 256), slice(256, 512), slice(512, 513), slice(256, 513)])
def test_head_tiles_without_a_finite_logit(ssv, cut):  # noqa: F811
    """Tokens whose logits are -inf have no part in a row's results, also where
    they fill a tile of the product (here 256, 256 and 1 tokens)."""
    N, V, H = 40, 513, 64
    x, w, y, rw = head_inputs(N, V, H, BF16, 7)
    gone = torch.zeros(V, dtype=torch.bool)
    gone[cut] = True
    x[:, 0], w[:, 0] = 1e20, 0.0
    w[gone, 0] = -1e20                      # logits of -1e40
    left = torch.nonzero(~gone)[:, 0]
    pick = torch.randint(0, len(left), (N,), generator=torch.Generator().manual_seed(1))
    y = left[pick].to(torch.int32)
    a = [t.to(DEV) for t in (x, w, y)]
    o = ssv.linear_cross_entropy_fwd_bwd(*a, 1.0, row_weight=rw.to(DEV), reduction="sum", grad_dtype=F32)
    f = ssv.linear_cross_entropy(*a, 1.0, row_weight=rw.to(DEV), reduction="sum")
    assert int(o.status) == 0 and torch.equal(f.loss, o.loss) and torch.equal(f.row_loss, o.row_loss)
    assert (f64(o.grad_weight)[gone.numpy()] == 0).all()
    o.grad_weight = o.grad_weight[left.to(DEV)]
    check_head(o, x, w[left], dense_labels(pick.numpy(), len(left), -100), 1.0, rw.numpy(), "sum", 1.0, F32)
    # a label among them: an infinite loss (or the least logit's), no NaN
    y[5] = int(torch.nonzero(gone)[0])
    o = ssv.linear_cross_entropy_fwd_bwd(a[0], a[1], y.to(DEV), 1.0, reduction="sum", grad_dtype=F32)
    assert float(o.row_loss[5]) > 3e38 and float(o.loss) > 3e38
    assert not o.grad_hidden.isnan().any() and not o.grad_weight.isnan().any()
    # nothing but such tokens is a row that cannot be normalised
    w[:, 0] = -1e20
    o = ssv.linear_cross_entropy(a[0], w.to(DEV), a[2], 1.0)
    assert o.row_loss.isnan().all() and int(o.status) == BAD_LOGITS


@pytest.mark.parametrize("N", [1, 20])
def test_head_weights_below_the_normal_range(ssv, N):  # noqa: F811
    """Row weights that have decayed to subnormal numbers still give the gradient's value."""
    V, H = 300, 64
    x, w, y, _ = head_inputs(N, V, H, BF16, 21)
    rw = torch.full((N,), 1e-39) * torch.linspace(1, 2, N)
    o = ssv.linear_cross_entropy_fwd_bwd(x.to(DEV), w.to(DEV), y.to(DEV), 1.0, 2.0 ** 126, row_weight=rw.to(DEV),
                                         reduction="sum", grad_dtype=F32)
    check_head(o, x, w, dense_labels(y.numpy(), V, -100), 1.0, rw.numpy(), "sum", 2.0 ** 126, F32)
    assert (f64(o.grad_hidden) != 0).any()


def test_two_host_threads_on_one_stream(ssv):  # noqa: F811
    """Calls of different sizes from two threads: each gets what it gets alone."""
    def job(N, V, H, k, seed):
        x, w, y, rw = (t.to(DEV) for t in head_inputs(N, V, H, BF16, seed))
        z, ids, tx, lse, kw = (t.to(DEV) for t in kd_inputs(N, V, k, BF16, seed, 1.0, padded=True))

        def call():
            a = ssv.linear_cross_entropy_fwd_bwd(x, w, y, 1.0, row_weight=rw)
            b = ssv.linear_topk_distill_fwd_bwd(x, w, ids, tx, 1.0, row_weight=rw)
            c = ssv.topk_distill_fwd_bwd(z, ids, tx, 1.0, teacher_lse=lse, row_weight=kw)
            return [a.loss, a.row_loss, a.grad_hidden, a.grad_weight, b.loss, b.grad_hidden, b.grad_weight, c.loss,
                    c.row_loss, c.grad, a.status, b.status, c.status]
        return call

    jobs = [job(70, 3001, 136, 12, 1), job(300, 5003, 200, 40, 2)]
    want = [j() for j in jobs]
    torch.cuda.synchronize()
    got, failed = [[], []], []

    def work(i):
        try:
            for _ in range(40):
                got[i].append(jobs[i]())
        except Exception as e:  # noqa: BLE001
            failed.append(repr(e))

    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for i in (0, 1):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(want[i], g))


# ---------------------------------------------------------------------------
# every buffer used again: several live rows a cluster, at every cluster size
# ---------------------------------------------------------------------------

REUSE_CASES = [
    # N, V, k, dtype, grad dtype, tail, padded, masked, gradients off a vector's boundary
    (400, 40003, 40, BF16, BF16, True, True, True, False),    # two CTAs a row
    (330, 60008, 64, F16, F32, False, False, False, False),
    (190, 120001, 33, BF16, F32, True, True, False, False),   # four
    (150, 70001, 100, F32, F32, True, False, False, False),
    (100, 129280, 64, F32, F32, True, True, False, False),    # eight
    (60, 160001, 20, F32, F32, True, False, True, False),     # sixteen
    (40, 300000, 256, F32, F32, False, True, False, False),
    (200, 80003, 16, BF16, BF16, True, True, False, True),    # from shared memory, two stages
    (100, 100000, 30, F32, F32, True, False, False, True),
    (30, 800001, 9, F32, F32, True, False, False, False),     # one stage
]


@pytest.mark.parametrize("N,V,k,dt,gdt,tail,padded,masked,off", REUSE_CASES)
def test_distill_many_rows_a_cluster(ssv, N, V, k, dt, gdt, tail, padded, masked, off):  # noqa: F811
    z, ids, x, lse, w = kd_inputs(N, V, k, dt, N + V, 1.0, padded, masked)
    scale = 3.0 if gdt != F16 else 3.0 * 4096
    grad = torch.empty(N * V + 1, dtype=gdt, device=DEV)[1 if off else 0:][:N * V].view(N, V)
    out = ssv.DistillOutput(torch.empty(1, device=DEV), torch.empty(N, device=DEV), grad,
                            torch.zeros(1, dtype=torch.int32, device=DEV))
    d = [t.to(DEV) for t in (z, ids, x, lse, w)]
    kw = dict(teacher_lse=d[3] if tail else None, row_weight=d[4])
    o = ssv.topk_distill_fwd_bwd(d[0], d[1], d[2], 1.0, scale, grad_dtype=gdt, out=out, **kw)
    f = ssv.topk_distill(d[0], d[1], d[2], 1.0, **kw)
    torch.cuda.synchronize()
    assert int(o.status) == 0
    for n0 in range(0, N, 50):  # the oracle's arrays are long
        rows = slice(n0, n0 + 50)
        r = listed_loss(f64(z[rows]), dense_teacher(ids[rows].numpy(), x[rows].numpy(), 1.0, V,
                                                    f64(lse[rows]) if tail else None), 1.0,
                        row_weight=w[rows].numpy(), reduction="sum", grad_scale=scale / int((ids >= 0).any(1).sum()))
        check_kd(o, r, 1.0, gdt, rows=rows)
        check_kd(f, r, 1.0, rows=rows)


def test_head_lists_of_many_rows(ssv):  # noqa: F811
    """More than 8192 rows: a CTA of the kernels that look at every row takes several blocks of them."""
    N, V, H, k = 9001, 520, 64, 5
    x, w, y, rw = head_inputs(N, V, H, BF16, 31)
    full = f64(x) @ f64(w).T
    ids = np.argsort(-full, axis=1)[:, :k].astype(np.int32)
    tx = np.take_along_axis(full, ids, axis=1).astype(np.float32)
    ids[::3] = -1
    ids[1::5, 2:] = -1
    for target, call in ((dense_teacher(ids, tx, 1.0, V),
                          lambda **kw: ssv.linear_topk_distill_fwd_bwd(x.to(DEV), w.to(DEV), torch.from_numpy(ids).to(DEV),
                                                                       torch.from_numpy(tx).to(DEV), 1.0, **kw)),
                         (dense_labels(np.where(np.arange(N) % 4 == 0, -100, y.numpy()), V, -100),
                          lambda **kw: ssv.linear_cross_entropy_fwd_bwd(
                              x.to(DEV), w.to(DEV), torch.where(torch.arange(N) % 4 == 0, -100, y).int().to(DEV), 1.0,
                              **kw))):
        o = call(row_weight=rw.to(DEV), reduction="sum", grad_dtype=F32)
        torch.cuda.synchronize()
        assert int(o.status) == 0
        check_head(o, x, w, target, 1.0, rw.numpy(), "sum", 1.0, F32)


@pytest.mark.parametrize("vecs", [1, 3, 4, 5, 7, 8, 10, 11, 13, 14, 16, 17, 19])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_distill_every_slice_length(ssv, vecs, dt):  # noqa: F811
    """Rows of one CTA each whose threads hold 1 to 19 vectors, not all of them full."""
    V = (vecs * 256 - 37) * (8 if dt == BF16 else 4) + 3
    N, k = 160, 24
    z, ids, x, lse, w = kd_inputs(N, V, k, dt, vecs, 1.0)
    d = [t.to(DEV) for t in (z, ids, x, lse)]
    o = ssv.topk_distill_fwd_bwd(*d[:3], 1.0, 3.0, teacher_lse=d[3], reduction="sum")
    f = ssv.topk_distill(*d[:3], 1.0, teacher_lse=d[3], reduction="sum")
    torch.cuda.synchronize()
    assert torch.equal(o.row_loss, f.row_loss) and int(o.status) == 0
    for rows in (slice(0, 20), slice(N - 20, N)):
        r = listed_loss(f64(z[rows]), dense_teacher(ids[rows].numpy(), x[rows].numpy(), 1.0, V, f64(lse[rows])), 1.0,
                        reduction="sum", grad_scale=3.0)
        check_kd(o, r, 1.0, dt, rows=rows)
