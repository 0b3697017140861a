"""Pins of the decoding step's oracle (CPU): hand examples and closed forms."""

import numpy as np

from oracle import decode


def pass_of(rows, Hq, Hkv, D, seed=0):
    g = np.random.default_rng(seed)
    return g.normal(size=(rows, Hq, D)), g.normal(size=(rows, Hkv, D)), g.normal(size=(rows, Hkv, D))


def test_equal_scores_average_the_values_that_are_seen():
    q, k, v = pass_of(3, 2, 1, 4)
    cache = np.random.default_rng(1).normal(size=(2, 3, 1, 4))
    mask = np.array([[[1, 0, 0], [1, 1, 0], [1, 0, 1]]])
    r = decode.tree_attention(q * 0, k, v, cache, cache, [[1, 0]], [4], [0, 3], mask, 1.0)
    old = np.concatenate([cache[1, :, 0], cache[0, :1, 0]])
    for i, seen in enumerate(([0], [0, 1], [0, 2])):
        want = np.concatenate([old, v[seen, 0]]).mean(axis=0)
        assert np.allclose(r.out[i], want[None]) and np.allclose(r.lse[i], np.log(4 + len(seen)))


def test_one_key_is_copied_and_nothing_seen_is_zero():
    q, k, v = pass_of(2, 1, 1, 8)
    mask = np.array([[[1, 0], [0, 0]]])
    none = np.zeros((0, 16, 1, 8))
    r = decode.tree_attention(q, k, v, none, none, np.zeros((1, 0), int), [0], [0, 2], mask, 0.3)
    assert np.allclose(r.out[0, 0], v[0, 0]) and np.isclose(r.lse[0, 0], 0.3 * q[0, 0] @ k[0, 0])
    assert not r.out[1].any() and r.lse[1, 0] == -np.inf


def test_plan_hand_example():
    # pages of 4: request 0 grows from 3 to 6 (one page more), 1 is done (two pages back),
    # 2 grows from 4 to 5; the stack [7, 8] becomes [7, 8, 3, 2], then 2 and 3 are popped
    table = [[5, -1, -1], [3, 2, -1], [6, -1, -1]]
    r = decode.plan_cache([3, 8, 4], [3, -8, 1], table, [7, 8, -1, -1], 2, 4, 4)
    assert r.table.tolist() == [[5, 2, -1], [3, 2, -1], [6, 3, -1]]
    assert r.count == 2 and r.free.tolist() == [7, 8, 3, 2] and r.lens.tolist() == [6, 0, 5]
    assert r.slots.tolist() == [[23, 8, 9, -1], [-1] * 4, [12, -1, -1, -1]]
    assert not r.bad and not r.short
    r = decode.plan_cache([3, 8, 4], [3, 4, 1], table, [7, -1], 1, 4, 4)  # one page for three requests
    assert r.short and r.lens.tolist() == [6, 8, 4] and r.count == 0 and r.slots[0, 0] == 23
    assert decode.plan_cache([13], [0], [[1, 2, 3]], [0], 1, 4, 4).bad


def test_rules_hand_example():
    z = np.array([[2.0, -2.0, 1.0, 0.5, 4.0], [2.0, -2.0, 1.0, 0.5, 4.0]])
    words = np.array([[0b11110], [0b11111]], dtype=np.uint32)
    out = decode.adjust_logits(z, np.array([2, 4]), [0, 2], None, np.array([[1, 1, 3, 0]]), [3], [1],
                               repetition=[2.0], frequency=[0.25], presence=[1.0], bias_ids=np.array([[2, 2, -1]]),
                               bias=np.array([[0.5, 0.25, 9.0]]), allowed=words)
    # token 1: in the prompt and generated once; 3 generated; 2 drafted in both rows, 4 in the second
    assert np.allclose(out[0], [-np.inf, -5.25, 0.5 - 1.25 + 0.75, 0.25 - 1.25, 4.0])
    assert np.allclose(out[1], [2.0, -5.25, 0.5 - 1.25 + 0.75, 0.25 - 1.25, 2.0 - 1.25])
