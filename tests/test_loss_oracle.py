"""Pins of the drafter-training losses' oracle: closed forms, the full KL as a
limit, and gradients against central differences (CPU)."""

import numpy as np
import pytest

from oracle import dense_labels, dense_teacher, head_loss, listed_loss


def _rows(N, V, k, seed, lse=False, T=1.0):
    rng = np.random.Generator(np.random.PCG64(seed))
    z = rng.normal(0, 2, (N, V))
    zt = z + rng.normal(0, 0.7, (N, V))
    ids = np.argsort(-zt, axis=1)[:, :k].astype(np.int32)
    x = np.take_along_axis(zt, ids, axis=1)
    full = np.log(np.exp(zt / T).sum(axis=1)) if lse else None
    return z, zt, ids, x, full


def test_uniform_logits_give_log_v():
    r = listed_loss(np.zeros((2, 7)), dense_labels([3, -100], 7, -100), 1.3)
    assert np.isclose(r.loss, np.log(7)) and r.row_loss[1] == 0 and (r.grad[1] == 0).all()
    np.testing.assert_allclose(r.grad[0], (np.full(7, 1 / 7) - np.eye(7)[3]) / 1.3)


def test_two_tokens_by_hand():
    # q = (1/4, 3/4); t = (1/2, 1/2): KL = 1/2 ln 2 + 1/2 ln(2/3)
    z = np.log(np.array([[1.0, 3.0]]))
    r = listed_loss(z, dense_teacher([[0, 1]], [[5.0, 5.0]], 1.0, 2), 1.0)
    assert np.isclose(r.loss, 0.5 * np.log(2) + 0.5 * np.log(2 / 3))
    np.testing.assert_allclose(r.grad, [[-0.25, 0.25]])


@pytest.mark.parametrize("T", [1.0, 0.6, 1.8])
def test_whole_vocabulary_is_the_full_kl(T):
    z, zt, ids, x, lse = _rows(3, 11, 11, 1, lse=True, T=T)
    p = np.exp(zt / T) / np.exp(zt / T).sum(axis=1, keepdims=True)
    q = np.exp(z / T) / np.exp(z / T).sum(axis=1, keepdims=True)
    kl = (p * np.log(p / q)).sum(axis=1)
    for full in (None, lse):
        r = listed_loss(z, dense_teacher(ids, x, T, 11, full), T, reduction="sum")
        np.testing.assert_allclose(r.row_loss, kl, rtol=1e-9)
        np.testing.assert_allclose(r.grad, (q - p) / T, rtol=1e-9, atol=1e-12)


def test_student_equal_to_teacher_is_the_minimum():
    z, _, ids, _, _ = _rows(3, 11, 4, 2)
    lse = np.log(np.exp(z).sum(axis=1))
    r = listed_loss(z, dense_teacher(ids, np.take_along_axis(z, ids, axis=1), 1.0, 11, lse), 1.0)
    np.testing.assert_allclose(r.row_loss, 0, atol=1e-12)
    np.testing.assert_allclose(r.grad, 0, atol=1e-12)


def test_the_bucket_is_a_merged_token():
    # merging the unlisted tokens on both sides gives the same KL over k + 1 outcomes
    z, zt, ids, x, lse = _rows(2, 9, 3, 3, lse=True)
    r = listed_loss(z, dense_teacher(ids, x, 1.0, 9, lse), 1.0)
    p, q = np.exp(zt - lse[:, None]), r.q
    for n in range(2):
        a = np.append(p[n, ids[n]], 1 - p[n, ids[n]].sum())
        b = np.append(q[n, ids[n]], 1 - q[n, ids[n]].sum())
        assert np.isclose(r.row_loss[n], (a * np.log(a / b)).sum())


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("T,reduction", [(1.0, "mean"), (0.7, "sum")])
def test_gradient_against_differences(tail, T, reduction):
    z, _, ids, x, lse = _rows(3, 8, 3, 4, lse=True, T=T)
    ids[1, 2] = -1
    ids[2] = -1  # left out
    target = dense_teacher(ids, x, T, 8, lse if tail else None)
    kw = dict(row_weight=[0.5, 2.0, 3.0], reduction=reduction)
    g = listed_loss(z, target, T, grad_scale=-1.5, **kw).grad
    h = 1e-5
    for n in range(3):
        for v in range(8):
            up, dn = z.copy(), z.copy()
            up[n, v] += h
            dn[n, v] -= h
            d = (listed_loss(up, target, T, **kw).loss - listed_loss(dn, target, T, **kw).loss) / (2 * h)
            assert abs(-1.5 * d - g[n, v]) < 1e-8
    assert (g[2] == 0).all()
    np.testing.assert_allclose(g.sum(axis=1), 0, atol=1e-12)  # softmax gradients sum to 0


def test_head_gradients_against_differences():
    rng = np.random.Generator(np.random.PCG64(5))
    x, w = rng.normal(0, 1, (4, 3)), rng.normal(0, 1, (6, 3))
    target = dense_labels([2, 0, 9, -100], 6, -100)  # the third label is out of range: left out
    f = lambda a, b: head_loss(a, b, target, 0.9)[0].loss  # noqa: E731
    _, gx, gw = head_loss(x, w, target, 0.9)
    h = 1e-5
    for a, g, wrt in ((x, gx, 0), (w, gw, 1)):
        for i in np.ndindex(a.shape):
            up, dn = a.copy(), a.copy()
            up[i] += h
            dn[i] -= h
            d = (f(up, w) - f(dn, w) if wrt == 0 else f(x, up) - f(x, dn)) / (2 * h)
            assert abs(d - g[i]) < 1e-8
    assert (gx[2:] == 0).all()


def test_rows_that_are_left_out():
    z = np.zeros((6, 5))
    ids = np.array([[-1, -1], [0, 5], [1, 1], [-2, 1], [0, 1], [2, -1]])
    x = np.array([[0, 0], [0, 0], [0, 0], [0, 0], [np.nan, 0], [0.5, 0]])
    t, listed, rest, keep = dense_teacher(ids, x, 1.0, 5)
    assert keep.tolist() == [False] * 5 + [True]
    assert t.sum() == 1.0 and listed.sum() == 1
    r = listed_loss(z, (t, listed, rest, keep), 1.0)
    assert np.isclose(r.loss, np.log(5))
