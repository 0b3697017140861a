"""GPU parity of the drafter-training losses against the fp64 oracle.

Tolerances, from the kernels' arithmetic (worst cases, not fitted):

* Each exponent x = (z - m) s is formed with two roundings of 2^-24 |x| and
  2^x with the hardware ex2 (2^-22 relative).  |x| <= 64 for every term above
  2^-64 of its row, so a term is off by at most 64 * 2^-23 * ln 2 + 2^-22 =
  5.6e-6 relative; a sum of positive terms keeps that and adds its depth (at
  most 150 additions of 2^-24 here: 9e-6).  E = 2e-5 bounds both, for the
  normaliser and for every probability.
* A row loss is a sum of t_i (log t_i - log q_i) with sum t_i + t_r <= 1:
  E absolute from log q, and 2e-6 relative from t and its own sums.
* A gradient entry of given logits is the difference of M q_v and t_v (or
  M q_v and q_v t_r / q_r): E (of their sum) times the row's coefficient, and
  half a step of the output type.
* Through the head, a logit is a sum over H of exact products, accumulated 16
  at a time in fp32: dz = (H / 16 + 1) 2^-23 max_v sum_h |x_h w_vh|.  It adds
  dz / T to the errors of lse and 2 dz / T to the relative ones of q.
  D is rounded to the 16-bit type (half a step u, and a quarter of the least
  subnormal of fp16 after its scaling by 2^15), and the products sum
  |D| |W| with (V / 16 + V / 1024 + 40) 2^-23 more (16 at a time, then over splits).
"""

import numpy as np
import pytest
import torch

from oracle import dense_labels, dense_teacher, head_loss, listed_loss

pytestmark = pytest.mark.gpu

DEV = "cuda"
E = 2e-5
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
BAD_TOKEN, BAD_LOGITS = 1, 2


def half_step(dt):
    return torch.finfo(dt).eps / 2


def tiny(dt):  # half the least subnormal
    f = torch.finfo(dt)
    return f.tiny * f.eps / 2


def f64(t):
    return t.detach().double().cpu().numpy()


@pytest.fixture(scope="module")
def ssv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sampling_spec_verify_gb300 as m
    m.lib()
    return m


# ---------------------------------------------------------------------------
# distillation of given logits
# ---------------------------------------------------------------------------

def kd_inputs(N, V, k, dt, seed, T, padded=False, masked=False):
    g = torch.Generator().manual_seed(seed)
    z = (2.0 * torch.randn(N, V, generator=g)).to(dt)
    full = z.float() + 0.5 * torch.randn(N, V, generator=g)
    x, ids = torch.topk(full, k, dim=1)
    lse = torch.logsumexp(full.double() / T, dim=1).float()
    ids = ids.to(torch.int32)
    if padded:
        n = torch.randint(0, k + 1, (N, 1), generator=g)
        hole = torch.rand(N, k, generator=g) < 0.2  # unused slots anywhere
        ids = torch.where((torch.arange(k)[None] < n) & ~hole, ids, -1)
    if masked:
        drop = torch.rand(N, V, generator=g) < 0.5
        for r in range(N):
            drop[r, ids[r][ids[r] >= 0].long()] = False
        z = z.masked_fill(drop, float("-inf"))
    w = 0.8 ** torch.randint(0, 7, (N,), generator=g).float()
    return z, ids.contiguous(), x.contiguous(), lse, w


def check_kd(o, r, T, grad_dtype=None, rows=None):
    rows = slice(None) if rows is None else rows
    tol = E + 2e-6 * np.abs(r.row_loss)
    assert (np.abs(f64(o.row_loss)[rows] - r.row_loss) <= tol).all(), np.abs(f64(o.row_loss)[rows] - r.row_loss).max()
    if grad_dtype is None:
        return
    g = f64(o.grad)[rows]
    mass = (r.t.sum(axis=1) + r.rest)[:, None]
    with np.errstate(divide="ignore", invalid="ignore"):
        qr = np.where(r.listed, 0.0, r.q).sum(axis=1)
        ratio = np.where(r.rest > 0, r.rest / qr, 0.0)[:, None]
    parts = np.where(r.listed, mass * r.q + r.t, r.q * (mass + ratio))
    tol = (E * parts * np.abs(r.coef[:, None]) / T + half_step(grad_dtype) * np.abs(r.grad) + tiny(grad_dtype)
           + 1e-37)
    assert (np.abs(g - r.grad) <= tol).all(), (np.abs(g - r.grad) / tol).max()


KD_CASES = [
    # N, V, k, dtype, grad dtype, T, tail, padded, masked, reduction
    (1, 1, 1, F32, F32, 1.0, False, False, False, "mean"),
    (1, 5, 3, BF16, BF16, 1.0, False, False, False, "sum"),
    (2, 7, 7, BF16, F32, 0.7, True, False, False, "mean"),      # the whole vocabulary listed
    (3, 9, 2, F16, F16, 1.0, True, False, False, "sum"),
    (4, 1024, 8, F32, F32, 1.0, False, False, False, "mean"),
    (5, 1001, 256, F32, F32, 1.7, True, True, False, "mean"),
    (9, 2049, 1, BF16, BF16, 1.0, False, False, True, "mean"),
    (8, 2047, 50, BF16, F32, 0.6, True, True, True, "sum"),
    (37, 4099, 33, F16, F32, 1.0, False, True, True, "mean"),
    (64, 20011, 64, F16, F16, 2.0, True, True, False, "sum"),
    (6, 50257, 100, BF16, BF16, 1.0, True, False, False, "mean"),
    (5, 151936, 128, BF16, F32, 1.0, False, False, False, "mean"),
    (3, 151937, 128, F32, F32, 1.0, True, False, False, "mean"),
    (2, 800001, 20, F32, F32, 1.0, False, False, False, "mean"),  # one stage per CTA
    (700, 513, 16, BF16, BF16, 1.0, True, True, False, "mean"),   # more rows than clusters
]


@pytest.mark.parametrize("N,V,k,dt,gdt,T,tail,padded,masked,red", KD_CASES)
def test_distill(ssv, N, V, k, dt, gdt, T, tail, padded, masked, red):
    z, ids, x, lse, w = kd_inputs(N, V, k, dt, N + V, T, padded, masked)
    d = [t.to(DEV) for t in (z, ids, x, lse, w)]
    kw = dict(teacher_lse=d[3] if tail else None, row_weight=d[4], reduction=red)
    scale = -3.0 if gdt != F16 else -3.0 * 4096
    o = ssv.topk_distill_fwd_bwd(d[0], d[1], d[2], T, scale, grad_dtype=gdt, **kw)
    f = ssv.topk_distill(d[0], d[1], d[2], T, **kw)
    torch.cuda.synchronize()
    r = listed_loss(f64(z), dense_teacher(ids.numpy(), x.numpy(), T, V, f64(lse) if tail else None), T,
                    row_weight=w.numpy(), reduction=red, grad_scale=scale)
    check_kd(o, r, T, gdt)
    check_kd(f, r, T)
    assert torch.equal(o.row_loss, f.row_loss) and torch.equal(o.loss, f.loss)
    wsum = (w.numpy() * r.keep).sum() / (max(r.keep.sum(), 1) if red == "mean" else 1)
    assert abs(float(o.loss) - r.loss) <= E * wsum + 4e-6 * abs(r.loss)
    assert int(o.status) == 0


def test_distill_views_that_start_off_a_boundary(ssv):
    V = 1003
    z, ids, x, lse, w = kd_inputs(9, V, 12, BF16, 3, 1.0)
    zd = z.to(DEV)
    for first in (1, 2, 3, 5):
        n = 9 - first
        grad = torch.zeros(n * V + 1, dtype=BF16, device=DEV)[1:].view(n, V)  # another offset than the logits'
        a = [t[first:].contiguous().to(DEV) for t in (ids, x, lse)]
        out = ssv.DistillOutput(torch.empty(1, device=DEV), torch.empty(n, device=DEV), grad,
                                torch.zeros(1, dtype=torch.int32, device=DEV))
        o = ssv.topk_distill_fwd_bwd(zd[first:], a[0], a[1], 1.0, teacher_lse=a[2], out=out)
        torch.cuda.synchronize()
        r = listed_loss(f64(z[first:]), dense_teacher(ids[first:].numpy(), x[first:].numpy(), 1.0, V, f64(lse[first:])),
                        1.0)
        check_kd(o, r, 1.0, BF16)


def test_distill_rows_left_out_and_bad_rows(ssv):
    N, V, k = 10, 777, 4
    z, ids, x, lse, w = kd_inputs(N, V, k, F32, 9, 1.0)
    nan, inf = float("nan"), float("inf")
    ids[0] = -1                      # nothing listed
    ids[1, 2] = V                    # outside the vocabulary
    ids[2, 3] = ids[2, 0]            # listed twice
    ids[3, 1] = -7
    x[4, 0] = nan                    # teacher
    x[5] = -inf
    z[0, 5] = nan                    # a left-out row's own logits do not matter
    target = dense_teacher(ids.numpy(), x.numpy(), 1.0, V)
    assert target[3].tolist() == [False] * 6 + [True] * 4
    o = ssv.topk_distill_fwd_bwd(*(t.to(DEV) for t in (z, ids, x)), 1.0)
    torch.cuda.synchronize()
    clean = z.clone()
    clean[0, 5] = 0
    r = listed_loss(f64(clean), target, 1.0)
    check_kd(o, r, 1.0, F32)
    assert (f64(o.grad)[:6] == 0).all() and (f64(o.row_loss)[:6] == 0).all()
    assert int(o.status) == BAD_TOKEN | BAD_LOGITS

    # student rows that cannot be normalised: NaN in their results, and only there
    z, ids, x, lse, w = kd_inputs(N, V, k, BF16, 10, 1.0)
    z[1, 700] = nan
    z[2, 3] = inf
    z[3] = -inf
    z[4, ids[4, 0].long()] = nan
    good = [0, 5, 6, 7, 8, 9]
    for tail in (None, lse.to(DEV)):
        o = ssv.topk_distill_fwd_bwd(*(t.to(DEV) for t in (z, ids, x)), 1.0, teacher_lse=tail, reduction="sum")
        torch.cuda.synchronize()
        assert np.isnan(f64(o.row_loss)[1:5]).all() and np.isnan(f64(o.grad)[1:5]).all()
        assert np.isnan(float(o.loss)) and int(o.status) == BAD_LOGITS
        r = listed_loss(f64(z[good]), dense_teacher(ids[good].numpy(), x[good].numpy(), 1.0, V,
                                                    None if tail is None else f64(lse[good])), 1.0, reduction="sum")
        check_kd(o, r, 1.0, BF16, rows=good)


def test_distill_masks(ssv):
    """Rows masked with the type's lowest value, and listed tokens that the
    student gives no mass."""
    V, k = 500, 3
    for dt in (F32, BF16, F16):
        z, ids, x, lse, w = kd_inputs(4, V, k, dt, 11, 1.0)
        low = torch.finfo(dt).min
        z[0] = low                                   # a uniform row
        z[1, torch.arange(V) != 17] = low            # one token left, not listed
        ids[1] = torch.tensor([3, 4, 5])
        z[2, ids[2, 1].long()] = float("-inf")       # listed with t > 0, q = 0: infinite loss, finite gradient
        o = ssv.topk_distill_fwd_bwd(*(t.to(DEV) for t in (z, ids, x)), 1.0, grad_dtype=F32, reduction="sum")
        torch.cuda.synchronize()
        r = listed_loss(f64(z), dense_teacher(ids.numpy(), x.numpy(), 1.0, V), 1.0, reduction="sum")
        assert np.isposinf(r.row_loss[2]) and np.isposinf(f64(o.row_loss)[2])
        rows = [0, 3]
        assert (np.abs(f64(o.row_loss)[rows] - r.row_loss[rows]) <= E + 2e-6 * np.abs(r.row_loss[rows])).all()
        tol = E * (r.q + r.t) + half_step(F32) * np.abs(r.grad) + 1e-37
        assert (np.abs(f64(o.grad) - r.grad) <= tol).all()


def test_distill_extremes(ssv):
    z, ids, x, lse, w = kd_inputs(3, 300, 5, F32, 12, 1.0)
    d = [t.to(DEV) for t in (z, ids, x)]
    # no rows; all rows left out; zero weights
    o = ssv.topk_distill_fwd_bwd(d[0][:0], d[1][:0], d[2][:0], 1.0)
    assert float(o.loss) == 0.0 and o.grad.shape == (0, 300)
    o = ssv.topk_distill_fwd_bwd(d[0], torch.full_like(d[1], -1), d[2], 1.0)
    assert float(o.loss) == 0.0 and (o.grad == 0).all() and int(o.status) == 0
    o = ssv.topk_distill_fwd_bwd(d[0], d[1], d[2], 1.0, row_weight=torch.zeros(3, device=DEV))
    assert float(o.loss) == 0.0 and (o.grad == 0).all() and (o.row_loss > 0).all()


def test_distill_offsets_past_32_bits(ssv):
    """More than 2^31 logits: the last rows against the oracle."""
    N, V, k = 15000, 151936, 8
    z = torch.empty(N, V, dtype=BF16, device=DEV)
    z.normal_(0, 2, generator=torch.Generator(device=DEV).manual_seed(1))
    ids = torch.full((N, k), -1, dtype=torch.int32, device=DEV)
    x = torch.zeros(N, k, device=DEV)
    last = slice(N - 3, N)
    x[last], i = torch.topk(z[last].float() + 0.3, k, dim=1)
    ids[last] = i.to(torch.int32)
    o = ssv.topk_distill_fwd_bwd(z, ids, x, 1.0)
    torch.cuda.synchronize()
    r = listed_loss(f64(z[last]), dense_teacher(ids[last].cpu().numpy(), f64(x[last]), 1.0, V), 1.0)
    o.row_loss, o.grad = o.row_loss[last], o.grad[last]
    check_kd(o, r, 1.0, BF16)


def test_distill_repeats_streams_and_graphs(ssv):
    z, ids, x, lse, w = (t.to(DEV) for t in kd_inputs(300, 4001, 40, BF16, 13, 1.0, padded=True))
    a = ssv.topk_distill_fwd_bwd(z, ids, x, 1.0, teacher_lse=lse, row_weight=w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = ssv.topk_distill_fwd_bwd(z, ids, x, 1.0, teacher_lse=lse, row_weight=w, stream=s)
    torch.cuda.synchronize()
    ws = torch.full((ssv.lib().spec_topk_distill_workspace_bytes(300, 4001, 40),), 255, dtype=torch.uint8, device=DEV)
    out = ssv.DistillOutput(torch.empty(1, device=DEV), torch.empty(300, device=DEV), torch.empty_like(z),
                            torch.zeros(1, dtype=torch.int32, device=DEV))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ssv.topk_distill_fwd_bwd(z, ids, x, 1.0, teacher_lse=lse, row_weight=w, out=out, workspace=ws)
    for _ in range(2):
        out.grad.zero_()
        g.replay()
    torch.cuda.synchronize()
    for o in (b, out):
        assert torch.equal(a.loss, o.loss) and torch.equal(a.row_loss, o.row_loss) and torch.equal(a.grad, o.grad)


# ---------------------------------------------------------------------------
# losses through the head
# ---------------------------------------------------------------------------

def head_inputs(N, V, H, dt, seed):
    g = torch.Generator().manual_seed(seed)
    w = (torch.randn(V, H, generator=g) * (2.0 / H ** 0.5)).to(dt)
    y = torch.randint(0, V, (N,), generator=g)
    x = (torch.randn(N, H, generator=g) + 4 * torch.rand(N, 1, generator=g) * w[y].float()).to(dt)
    rw = 0.8 ** torch.randint(0, 7, (N,), generator=g).float()
    return x, w, y.to(torch.int32), rw


def check_head(o, x, w, target, T, rw, red, scale, gdt, weight=True):
    dt = x.dtype
    X, W = f64(x), f64(w)
    (N, H), V = X.shape, W.shape[0]
    r, gx, gw = head_loss(X, W, target, T, row_weight=rw, reduction=red, grad_scale=scale)
    dz = (H / 16 + 1) * 2.0 ** -23 * (np.abs(X) @ np.abs(W).T).max(axis=1) / T  # per row, in exponents
    assert (np.abs(f64(o.lse) - r.lse) <= dz + E + half_step(F32) * np.abs(r.lse)).all()
    tol = np.where(r.keep, 2 * dz + E + 2e-6 * np.abs(r.row_loss), 0.0)
    assert (np.abs(f64(o.row_loss) - r.row_loss) <= tol).all()
    weights = np.where(r.keep, 1.0 if rw is None else np.abs(rw), 0.0) / (max(r.keep.sum(), 1) if red == "mean" else 1)
    assert abs(float(o.loss) - r.loss) <= (weights * (2 * dz + E)).sum() + 4e-6 * (weights * np.abs(r.row_loss)).sum()
    if gdt is None:
        return
    # D, in units of its largest row weight, then its rounding
    wmax = np.abs(r.coef).max()
    if wmax == 0:
        assert (f64(o.grad_hidden) == 0).all()
        return
    c = np.abs(r.coef)[:, None] / T
    least = 2.0 ** -25 / 2.0 ** 15 if dt == F16 else 0.0
    err = c * ((r.q + r.t) * (2 * dz[:, None] + E)) + half_step(dt) * np.abs(r.grad) + least * wmax / T * r.keep[:, None]
    size = np.abs(r.grad) + err
    u = half_step(gdt)
    for name, got, want, tol in (
            ("hidden", o.grad_hidden, gx, err @ np.abs(W) + (V / 16 + V / 1024 + 40) * 2.0 ** -23 * (size @ np.abs(W))),
            ("weight", o.grad_weight, gw, err.T @ np.abs(X) + (N / 16 + 40) * 2.0 ** -23 * (size.T @ np.abs(X)))):
        if name == "weight" and not weight:
            assert got is None
            continue
        d = np.abs(f64(got) - want)
        tol = tol + u * np.abs(want) + tiny(gdt)
        assert (d <= tol).all(), (name, (d / tol).max())


HEAD_CASES = [
    # N, V, H, dtype, grad dtype, T, k (0: cross entropy), reduction, weighted
    (1, 1, 8, BF16, BF16, 1.0, 0, "mean", False),
    (1, 300, 8, BF16, F32, 1.0, 0, "sum", False),
    (2, 257, 64, F16, F16, 0.7, 3, "sum", True),
    (7, 1000, 72, BF16, BF16, 1.0, 256, "mean", True),
    (127, 511, 136, BF16, F32, 1.7, 0, "mean", True),
    (129, 256, 64, F16, F32, 1.0, 5, "sum", False),
    (256, 2048, 256, BF16, BF16, 1.0, 0, "mean", False),
    (257, 2051, 264, F16, F16, 1.0, 0, "sum", True),
    (300, 5003, 712, BF16, BF16, 0.8, 20, "mean", True),
    (1000, 3001, 520, BF16, BF16, 1.0, 0, "mean", True),
    (33, 20011, 1024, BF16, F32, 1.0, 64, "mean", False),
    (9, 66001, 1024, BF16, BF16, 1.0, 0, "mean", True),   # a few rows, heads longer than the L2
    (5, 33001, 2056, F16, F16, 0.7, 7, "sum", True),
    (260, 60001, 1128, BF16, BF16, 1.0, 0, "mean", True),  # rows off a sector, two tiles of them
]


@pytest.mark.parametrize("N,V,H,dt,gdt,T,k,red,weighted", HEAD_CASES)
def test_head(ssv, N, V, H, dt, gdt, T, k, red, weighted):
    x, w, y, rw = head_inputs(N, V, H, dt, N + V + H)
    xd, wd, rd = x.to(DEV), w.to(DEV), rw.to(DEV) if weighted else None
    scale = 2.0 if dt == BF16 else 2.0 * 512
    kw = dict(row_weight=rd, reduction=red)
    if k == 0:
        if N > 4:
            y[::3] = -100
        target = dense_labels(y.numpy(), V, -100)
        a = (xd, wd, y.to(DEV), T)
        fwd, both = ssv.linear_cross_entropy, ssv.linear_cross_entropy_fwd_bwd
    else:
        full = f64(x) @ f64(w).T + np.random.Generator(np.random.PCG64(1)).normal(0, 0.5, (N, V))
        ids = np.argsort(-full, axis=1)[:, :k].astype(np.int32)
        tx = np.take_along_axis(full, ids, axis=1).astype(np.float32)
        if N > 4:
            ids[::3, k // 2:] = -1
            ids[1] = -1
        target = dense_teacher(ids, tx, T, V)
        a = (xd, wd, torch.from_numpy(ids).to(DEV), torch.from_numpy(tx).to(DEV), T)
        fwd, both = ssv.linear_topk_distill, ssv.linear_topk_distill_fwd_bwd
    f = fwd(*a, **kw)
    o = both(*a, scale, grad_dtype=gdt, **kw)
    h = both(*a, scale, grad_dtype=gdt, want_grad_weight=False, **kw)
    v = both(*a, scale, grad_dtype=gdt, want_grad_hidden=False, **kw)
    torch.cuda.synchronize()
    check_head(f, x, w, target, T, rw.numpy() if weighted else None, red, scale, None)
    check_head(o, x, w, target, T, rw.numpy() if weighted else None, red, scale, gdt)
    assert h.grad_weight is None and torch.equal(h.grad_hidden, o.grad_hidden)
    assert v.grad_hidden is None and torch.equal(v.grad_weight, o.grad_weight)
    for q in (f, h, v):
        assert torch.equal(q.loss, o.loss) and torch.equal(q.row_loss, o.row_loss) and torch.equal(q.lse, o.lse)
    assert int(o.status) == 0


@pytest.mark.parametrize("N", [70000, 170000, 520000])
def test_head_in_pieces(ssv, N):
    """Long batches, the last one long enough that its vocabulary is cut:
    against fp64 products on the GPU."""
    V, H = 4100, 64
    x, w, y, _ = head_inputs(N, V, H, BF16, 5)
    y[:N // 2] = -100
    xd, wd, yd = x.to(DEV), w.to(DEV), y.to(DEV)
    o = ssv.linear_cross_entropy_fwd_bwd(xd, wd, yd, 1.0, reduction="sum", grad_dtype=F32)
    torch.cuda.synchronize()
    X, W = xd.double(), wd.double()
    gw = torch.zeros_like(W)
    tw = torch.zeros_like(W)
    u = half_step(BF16)
    for r in range(0, N, 10000):
        z = X[r:r + 10000] @ W.T
        lse = torch.logsumexp(z, dim=1)
        dz = (H / 16 + 1) * 2.0 ** -23 * (X[r:r + 10000].abs() @ W.abs().T).amax(dim=1)
        assert ((o.lse[r:r + 10000].double() - lse).abs() <= dz + E + half_step(F32) * lse.abs()).all()
        keep = yd[r:r + 10000] >= 0
        q = torch.exp(z - lse[:, None]) * keep[:, None]
        t = torch.zeros_like(q)
        t[torch.nonzero(keep)[:, 0], yd[r:r + 10000][keep].long()] = 1.0
        d = q - t
        err = (q + t) * (2 * dz[:, None] + E) + u * d.abs()
        size = d.abs() + err
        gx = d @ W
        tol = err @ W.abs() + (V / 16 + V / 1024 + 40) * 2.0 ** -23 * (size @ W.abs()) + half_step(F32) * gx.abs()
        assert ((o.grad_hidden[r:r + 10000].double() - gx).abs() <= tol).all()
        gw += d.T @ X[r:r + 10000]
        tw += err.T @ X[r:r + 10000].abs() + (N / 16 + 40) * 2.0 ** -23 * (size.T @ X[r:r + 10000].abs())
    assert ((o.grad_weight.double() - gw).abs() <= tw + half_step(F32) * gw.abs()).all()


def test_head_rows_left_out_and_bad_rows(ssv):
    N, V, H = 20, 600, 64
    x, w, y, rw = head_inputs(N, V, H, BF16, 6)
    y[3] = 12345          # outside the vocabulary
    y[4] = -1
    y[5] = -100
    o = ssv.linear_cross_entropy_fwd_bwd(x.to(DEV), w.to(DEV), y.to(DEV), 1.0)
    torch.cuda.synchronize()
    assert int(o.status) == BAD_TOKEN
    check_head(o, x, w, dense_labels(y.numpy(), V, -100), 1.0, None, "mean", 1.0, BF16)
    assert (f64(o.grad_hidden)[3:6] == 0).all()
    # an ignore_index inside the vocabulary wins over the label that it is
    y2 = y.clone().clamp(0, V - 1)
    o = ssv.linear_cross_entropy_fwd_bwd(x.to(DEV), w.to(DEV), y2.to(DEV), 1.0, ignore_index=int(y2[0]))
    torch.cuda.synchronize()
    check_head(o, x, w, dense_labels(y2.numpy(), V, int(y2[0])), 1.0, None, "mean", 1.0, BF16)
    # NaN and infinite hidden states spoil their own rows and the head's gradient
    for bad in (float("nan"), float("inf")):
        xb = x.clone()
        xb[7, 3] = bad
        o = ssv.linear_cross_entropy_fwd_bwd(xb.to(DEV), w.to(DEV), y2.to(DEV), 1.0, reduction="sum")
        torch.cuda.synchronize()
        assert int(o.status) == BAD_LOGITS
        assert np.isnan(f64(o.row_loss)[7]) and np.isnan(f64(o.grad_hidden)[7]).all() and np.isnan(float(o.loss))
        rest = [i for i in range(N) if i != 7]
        assert np.isfinite(f64(o.row_loss)[rest]).all() and np.isfinite(f64(o.grad_hidden)[rest]).all()
    # nothing counts; no rows
    o = ssv.linear_cross_entropy_fwd_bwd(x.to(DEV), w.to(DEV), torch.full((N,), -100, dtype=torch.int32, device=DEV))
    assert float(o.loss) == 0 and (o.grad_hidden == 0).all() and (o.grad_weight == 0).all() and (o.row_loss == 0).all()
    o = ssv.linear_cross_entropy_fwd_bwd(x[:0].to(DEV), w.to(DEV), y[:0].to(DEV))
    assert float(o.loss) == 0 and (o.grad_weight == 0).all() and o.grad_hidden.shape == (0, H)


@pytest.mark.parametrize("N,kept", [(20, 3), (300, 64), (700, 129), (700, 0), (700, 700)])
@pytest.mark.parametrize("dt", [BF16, F16])
def test_head_left_out_rows_may_hold_anything(ssv, N, kept, dt):
    """Hidden states of rows that are left out reach no result but their own lse."""
    V, H = 900, 72
    x, w, y, rw = head_inputs(N, V, H, dt, N + kept)
    order = torch.randperm(N, generator=torch.Generator().manual_seed(3))
    y[order[kept:]] = -100
    clean = x.clone()
    clean[y < 0] = 0
    x[y < 0] = torch.tensor([float("nan"), float("inf"), -float("inf"), 7.0], dtype=dt).repeat(H // 4)
    kw = dict(row_weight=rw.to(DEV), reduction="sum", grad_dtype=F32)
    o = ssv.linear_cross_entropy_fwd_bwd(x.to(DEV), w.to(DEV), y.to(DEV), 1.0, 64.0, **kw)
    c = ssv.linear_cross_entropy_fwd_bwd(clean.to(DEV), w.to(DEV), y.to(DEV), 1.0, 64.0, **kw)
    torch.cuda.synchronize()
    assert int(o.status) == 0
    assert torch.equal(o.loss, c.loss) and torch.equal(o.row_loss, c.row_loss)
    assert torch.equal(o.grad_hidden, c.grad_hidden) and torch.equal(o.grad_weight, c.grad_weight)
    check_head(c, clean, w, dense_labels(y.numpy(), V, -100), 1.0, rw.numpy(), "sum", 64.0, F32)


def test_head_weights_of_either_sign(ssv):
    x, w, y, _ = head_inputs(40, 700, 128, BF16, 8)
    rw = torch.linspace(-2, 1, 40)
    o = ssv.linear_cross_entropy_fwd_bwd(x.to(DEV), w.to(DEV), y.to(DEV), 1.0, row_weight=rw.to(DEV), reduction="sum")
    torch.cuda.synchronize()
    check_head(o, x, w, dense_labels(y.numpy(), 700, -100), 1.0, rw.numpy(), "sum", 1.0, BF16)


def test_head_repeats_streams_and_graphs(ssv):
    x, w, y, rw = (t.to(DEV) for t in head_inputs(300, 5003, 200, BF16, 9))
    N, V, H = 300, 5003, 200
    a = ssv.linear_cross_entropy_fwd_bwd(x, w, y, 1.0, row_weight=rw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = ssv.linear_cross_entropy_fwd_bwd(x, w, y, 1.0, row_weight=rw, stream=s)
    torch.cuda.synchronize()
    ws = torch.full((ssv.lib().spec_linear_loss_workspace_bytes(ssv.SPEC_BF16, N, V, H, 1, 1, 1),), 255, dtype=torch.uint8, device=DEV)
    e = lambda *sh, dt=F32: torch.empty(sh, dtype=dt, device=DEV)  # noqa: E731
    out = ssv.LinearLossOutput(e(1), e(N), e(N), e(N, H, dt=BF16), e(V, H, dt=BF16),
                               torch.zeros(1, dtype=torch.int32, device=DEV))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ssv.linear_cross_entropy_fwd_bwd(x, w, y, 1.0, row_weight=rw, out=out, workspace=ws)
    for _ in range(2):
        out.grad_hidden.zero_()
        out.grad_weight.zero_()
        g.replay()
    torch.cuda.synchronize()
    for o in (b, out):
        assert torch.equal(a.loss, o.loss) and torch.equal(a.row_loss, o.row_loss) and torch.equal(a.lse, o.lse)
        assert torch.equal(a.grad_hidden, o.grad_hidden) and torch.equal(a.grad_weight, o.grad_weight)


@pytest.mark.parametrize("side", [False, True])
def test_captured_calls_own_their_memory(ssv, side):
    """Outputs and workspace of a captured call belong to the graph: eager calls
    of other sizes between the replays change nothing, also where the call runs
    on a stream that joined the capture."""
    x, w, y, rw = (t.to(DEV) for t in head_inputs(70, 3001, 136, BF16, 10))
    z, ids, tx, lse, kw = (t.to(DEV) for t in kd_inputs(20, 3001, 12, BF16, 14, 1.0, padded=True))

    def calls(stream=None):
        return (ssv.linear_cross_entropy_fwd_bwd(x, w, y, 1.0, row_weight=rw, stream=stream),
                ssv.topk_distill_fwd_bwd(z, ids, tx, 1.0, teacher_lse=lse, row_weight=kw, stream=stream))

    def values(pair):
        a, b = pair
        return [a.loss, a.row_loss, a.lse, a.grad_hidden, a.grad_weight, b.loss, b.row_loss, b.grad]

    want = values(calls())
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    with torch.cuda.graph(g):
        if side:
            s.wait_stream(torch.cuda.current_stream())
            pair = calls(s)
            torch.cuda.current_stream().wait_stream(s)
        else:
            pair = calls()
    bx, bw, by, _ = (t.to(DEV) for t in head_inputs(300, 5003, 200, BF16, 9))
    for _ in range(2):
        for t in values(pair):
            t.zero_()
        ssv.linear_cross_entropy_fwd_bwd(bx, bw, by, 1.0)
        g.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, values(pair)):
        assert torch.equal(a, b)
    assert int(pair[0].status.item()) == 0 and int(pair[1].status.item()) == 0


def test_python_refusals(ssv):
    x, w, y, rw = (t.to(DEV) for t in head_inputs(4, 64, 16, BF16, 9))
    ce = ssv.linear_cross_entropy_fwd_bwd
    ids, tl = torch.zeros(4, 2, dtype=torch.int32, device=DEV), torch.zeros(4, 2, device=DEV)
    with pytest.raises(TypeError):
        ce(x.float(), w.float(), y)
    with pytest.raises(TypeError):
        ce(x, w.half(), y)
    with pytest.raises(TypeError):
        ce(x, w, y.long())
    with pytest.raises(ValueError):
        ce(x, w[:, :8].contiguous(), y)
    with pytest.raises(ValueError):
        ce(x.t(), w, y)
    with pytest.raises(ValueError):
        ce(x, w, y, want_grad_hidden=False, want_grad_weight=False)
    with pytest.raises(TypeError):
        ce(x, w, y, grad_dtype=torch.float16)
    with pytest.raises(ValueError):
        ce(x, w, y, reduction="none")
    with pytest.raises(ValueError):
        ce(x, w, y, row_weight=rw[:3])
    with pytest.raises(ssv.SpecError):
        ce(x, w, y, 0.0)
    with pytest.raises(ssv.SpecError):
        ce(x, w, y, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    with pytest.raises(ssv.SpecError):
        ce(x[:, :12].contiguous(), w[:, :12].contiguous(), y)
    with pytest.raises(ValueError):
        ssv.linear_topk_distill(x, w, ids[:3], tl)
    with pytest.raises(TypeError):
        ssv.linear_topk_distill(x, w, ids, None)
    z = torch.zeros(4, 64, device=DEV)
    with pytest.raises(TypeError):
        ssv.topk_distill(z.double(), ids, tl)
    with pytest.raises(TypeError):
        ssv.topk_distill(z, ids, tl.half())
    with pytest.raises(TypeError):
        ssv.topk_distill_fwd_bwd(z, ids, tl, grad_dtype=BF16)
    with pytest.raises(ValueError):
        ssv.topk_distill(z.cpu(), ids, tl)
    with pytest.raises(ValueError):
        ssv.topk_distill(z, ids, tl, teacher_lse=torch.zeros(3, device=DEV))
    with pytest.raises(ssv.SpecError):
        ssv.topk_distill(z, torch.full((4, 300), -1, dtype=torch.int32, device=DEV), torch.zeros(4, 300, device=DEV))
