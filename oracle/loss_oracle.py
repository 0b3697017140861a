"""fp64 CPU oracle of the drafter-training losses (test infrastructure only).

A drafter is trained with cross entropy or a KL term (Bebop/DSpark blog,
section "Bebop 的解法"); only its own side is differentiated (SpecOPD summary,
method step (6)).  All losses are

    L_n = sum_i t_i (log t_i - log q_i) + t_r (log t_r - log q_r)

with q = softmax(z_n / T) over the vocabulary, t the teacher's probabilities
of the tokens that it lists, and t_r, q_r what the list leaves over on either
side (t_r = 0 unless the teacher's normaliser is given).  Cross entropy lists
the label with t = 1.
"""

from __future__ import annotations

from dataclasses import dataclass

import numpy as np

# A teacher remainder below this is the rounding of a sum in 32 bits: none.
REST_MIN = 1e-6


@dataclass
class LossResult:
    loss: float
    row_loss: np.ndarray   # [N], 0 where a row is left out
    lse: np.ndarray        # [N] log sum_v exp(z_v / T)
    keep: np.ndarray       # [N] the row counts
    coef: np.ndarray       # [N] factor of the row's loss in grad_scale * loss
    q: np.ndarray          # [N, V]
    t: np.ndarray          # [N, V] teacher probabilities, 0 off the list
    listed: np.ndarray     # [N, V] bool
    rest: np.ndarray       # [N] t_r
    grad: np.ndarray       # [N, V] gradient of grad_scale * loss in the logits


def logsumexp(a):
    with np.errstate(divide="ignore"):
        return np.log(np.exp(a).sum(axis=1))


def dense_teacher(ids, logits, temperature, V, lse=None):
    """(t [N, V], listed [N, V], rest [N], keep [N]) of the teacher's lists."""
    ids = np.asarray(ids)
    N, k = ids.shape
    t = np.zeros((N, V))
    listed = np.zeros((N, V), dtype=bool)
    rest = np.zeros(N)
    keep = np.zeros(N, dtype=bool)
    for n in range(N):
        used = ids[n] != -1
        i = ids[n][used]
        x = np.asarray(logits, dtype=np.float64)[n][used] / float(temperature)
        if not len(i) or i.min() < 0 or i.max() >= V or len(set(i.tolist())) != len(i):
            continue
        if np.isnan(x).any() or np.isposinf(x).any():
            continue
        if lse is None:
            if np.isneginf(x).all():
                continue
            e = np.exp(x - x.max())
            p = e / e.sum()
        else:
            if not np.isfinite(lse[n]):
                continue
            p = np.exp(x - float(lse[n]))
            r = 1.0 - p.sum()
            rest[n] = r if r > REST_MIN else 0.0
        keep[n] = True
        listed[n, i] = True
        t[n, i] = p
    return t, listed, rest, keep


def dense_labels(labels, V, ignore_index):
    labels = np.asarray(labels)
    N = len(labels)
    t = np.zeros((N, V))
    keep = (labels != ignore_index) & (labels >= 0) & (labels < V)
    t[np.nonzero(keep)[0], labels[keep]] = 1.0
    return t, t > 0, np.zeros(N), keep


def listed_loss(z, target, temperature, *, row_weight=None, reduction="mean", grad_scale=1.0):
    """The loss of logits z [N, V] against ``target`` = dense_teacher(...) or
    dense_labels(...), and its gradient with respect to z:

      dL/dz_v = (M q_v - t_v) / T            v listed, M = sum_i t_i + t_r
              = q_v (M - t_r / q_r) / T      otherwise
    """
    t, listed, rest, keep = target
    a = np.asarray(z, dtype=np.float64) / float(temperature)
    N, V = a.shape
    # each row's maximum comes off first: beside the lowest value of a type the
    # logarithm of a sum would be lost
    top = np.max(a, axis=1) if N else np.zeros(0)
    top = np.where(np.isneginf(top), 0.0, top)
    a = a - top[:, None]
    lse = logsumexp(a) if N else np.zeros(0)
    with np.errstate(divide="ignore", invalid="ignore"):
        logq = a - lse[:, None]
        q = np.exp(logq)
        row = np.where(t > 0, t * (np.log(t) - logq), 0.0).sum(axis=1)
        lse_rest = logsumexp(np.where(listed, -np.inf, a)) if N else np.zeros(0)
        row = row + np.where(rest > 0, rest * (np.log(rest) - (lse_rest - lse)), 0.0)
        ratio = np.where(rest > 0, rest / np.exp(lse_rest - lse), 0.0)
    row = np.where(keep, row, 0.0)
    w = np.ones(N) if row_weight is None else np.asarray(row_weight, dtype=np.float64)
    w = np.where(keep, w, 0.0)
    den = max(int(keep.sum()), 1) if reduction == "mean" else 1
    mass = (t.sum(axis=1) + rest)[:, None]
    coef = grad_scale * w / den
    with np.errstate(invalid="ignore"):
        g = np.where(listed, mass * q - t, q * (mass - ratio[:, None]))
        g = np.where(keep[:, None], g * (coef / float(temperature))[:, None], 0.0)
    return LossResult(float((w * row)[keep].sum() / den), row, top + lse, keep, coef, q, t, listed, rest, g)


def head_loss(hidden, weight, target, temperature, **kw):
    """listed_loss of the head's logits hidden @ weight.T, with the gradients
    of hidden and weight: (LossResult, grad_hidden [N, H], grad_weight [V, H])."""
    x = np.asarray(hidden, dtype=np.float64)
    w = np.asarray(weight, dtype=np.float64)
    r = listed_loss(x @ w.T, target, temperature, **kw)
    return r, r.grad @ w, r.grad.T @ x
