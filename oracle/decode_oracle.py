"""fp64 CPU oracle of the decoding step around the verify (test infrastructure only).

Attention of a pass's rows over cached tokens and the rows that a mask names
(SpecOPD summary, section on tree attention: a node sees the prefix, itself and its
ancestors), the page allocator, the commit of an accepted path, and the rules on
logits.  Everything is written request by request and token by token.
"""

from __future__ import annotations

from dataclasses import dataclass

import numpy as np


@dataclass
class AttentionResult:
    out: np.ndarray   # [rows, Hq, D]
    lse: np.ndarray   # [rows, Hq]
    mass: np.ndarray  # [rows, Hq, D] sum of weight times |v|, the scale of a weight's rounding
    spread: np.ndarray  # [rows, Hq] largest sum of |q k| scale over the row's keys


def tree_attention(q, k_new, v_new, k_cache, v_cache, table, lens, offsets, mask, scale):
    """q [rows, Hq, D], k_new and v_new [rows, Hkv, D], caches [pages, page, Hkv, D], all float64;
    offsets [B + 1]; mask [B, T, T] or None (a chain)."""
    rows, Hq, D = q.shape
    Hkv, page = k_new.shape[1], k_cache.shape[1]
    out, mass = np.zeros((rows, Hq, D)), np.zeros((rows, Hq, D))
    lse, spread = np.full((rows, Hq), -np.inf), np.zeros((rows, Hq))
    for b in range(len(lens)):
        r0, r1 = offsets[b], offsets[b + 1]
        n = int(lens[b])
        at = np.arange(n)
        ids, place = np.asarray(table[b])[at // page].astype(int) if n else at, at % page
        good = (ids >= 0) & (ids < len(k_cache)) if n else np.zeros(0, dtype=bool)
        for h in range(Hq):
            kh = h // (Hq // Hkv)
            k, v = np.zeros((n, D)), np.zeros((n, D))  # a page outside the cache reads as zeros
            k[good], v[good] = k_cache[ids[good], place[good], kh], v_cache[ids[good], place[good], kh]
            for i in range(r1 - r0):
                sees = np.arange(r1 - r0) <= i if mask is None else np.asarray(mask[b, i, :r1 - r0]) != 0
                ki = np.concatenate([k, k_new[r0:r1, kh][sees]])
                vi = np.concatenate([v, v_new[r0:r1, kh][sees]])
                with np.errstate(invalid="ignore"):
                    s = scale * (ki @ q[r0 + i, h])
                spread[r0 + i, h] = (np.abs(ki) @ np.abs(q[r0 + i, h])).max(initial=0.0) * abs(scale)
                m = s.max(initial=-np.inf)
                if m == -np.inf:
                    continue
                with np.errstate(invalid="ignore"):
                    p = np.exp(s - m)
                    total = p.sum()
                    out[r0 + i, h] = p @ vi / total
                    mass[r0 + i, h] = p @ np.abs(vi) / total
                    lse[r0 + i, h] = m + np.log(total)
    return AttentionResult(out, lse, mass, spread)


@dataclass
class PlanResult:
    table: np.ndarray
    free: np.ndarray
    count: int
    lens: np.ndarray
    slots: np.ndarray
    bad: bool
    short: bool  # too few pages


def plan_cache(lens, new, table, free, count, page, T):
    lens, new = [int(x) for x in lens], [int(x) for x in new]
    table, stack, count = np.array(table), np.array(free), int(count)
    B, width = table.shape
    pages = lambda n: -(-n // page)  # noqa: E731
    slots = np.full((B, T), -1, dtype=np.int32)
    ok = [0 <= n <= width * page and 0 <= n + a <= width * page and a <= T for n, a in zip(lens, new)]
    bad = not all(ok)
    back = sum(max(pages(n) - pages(n + a), 0) for n, a, o in zip(lens, new, ok) if o)
    if count < 0 or count + back > len(stack):
        return PlanResult(table, stack, count, np.array(lens, dtype=np.int32), slots, True, False)
    for b in range(B):
        if ok[b]:
            for j in range(pages(lens[b] + new[b]), pages(lens[b])):
                stack[count] = table[b, j]
                count += 1
    short = False
    for b in range(B):
        if not ok[b]:
            continue
        first, last = pages(lens[b]), pages(lens[b] + new[b])
        if last > first and (short or last - first > count):
            short = True
            continue
        for j in range(first, last):
            count -= 1
            table[b, j] = stack[count]
        for i in range(max(new[b], 0)):
            slots[b, i] = table[b, (lens[b] + i) // page] * page + (lens[b] + i) % page
        lens[b] += new[b]
    return PlanResult(table, stack, count, np.array(lens, dtype=np.int32), slots, bad, short)


def adjust_logits(z, tokens, offsets, mask, history, lens, prompts=None, repetition=None, frequency=None,
                  presence=None, bias_ids=None, bias=None, allowed=None):
    """z [rows, V] float64, tokens [rows], allowed [rows, words] uint32."""
    z = np.array(z, dtype=np.float64)
    V = z.shape[1]
    valid = lambda t: t[(t >= 0) & (t < V)]  # noqa: E731
    for b in range(len(lens)):
        r0, r1 = offsets[b], offsets[b + 1]
        n = int(min(max(lens[b], 0), history.shape[1]))
        start = 0 if prompts is None else int(prompts[b])
        seen = np.zeros(V, dtype=bool)
        seen[valid(history[b, :n][:max(start, 0)])] = True
        made = np.bincount(valid(history[b, :n][max(start, 0):]), minlength=V)
        for r in range(r0, r1):
            see = np.arange(r1 - r0) <= r - r0 if mask is None else np.asarray(mask[b, r - r0, :r1 - r0]) != 0
            c = made + np.bincount(valid(tokens[r0:r1][see]), minlength=V)
            x = z[r]
            hit = seen | (c > 0)
            with np.errstate(invalid="ignore", over="ignore"):
                if repetition is not None:
                    rep = float(repetition[b])
                    x[hit] = np.where(x[hit] > 0, x[hit] / rep, x[hit] * rep)
                drop = np.zeros(V)
                if frequency is not None:
                    drop += float(frequency[b]) * c
                if presence is not None:
                    drop += float(presence[b]) * (c > 0)
                x[c > 0] -= drop[c > 0]
                if bias is not None:
                    for t, v in zip(bias_ids[b], bias[b]):
                        if 0 <= t < V:
                            x[t] += float(v)
            if allowed is not None:
                bits = np.unpackbits(np.ascontiguousarray(allowed[r]).view(np.uint8), bitorder="little")[:V]
                x[bits == 0] = -np.inf
    return z
