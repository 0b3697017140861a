"""Cache plan and commit against the oracle, bit by bit."""

import numpy as np
import pytest
import torch

from oracle import decode

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def ssv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sampling_spec_verify_gb300 as m
    m.lib()
    return m


def put(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def plan_case(seed, B, width, page, T, spare, used=0.6):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, max(1, int(width * page * used)) + 1, size=B)
    new = rng.integers(0, T + 1, size=B)
    kind = rng.uniform(size=B)
    new = np.where(kind < 0.2, -lens, np.where(kind < 0.4, -np.minimum(lens, rng.integers(0, 2 * page + 1, size=B)), new))
    held = -(-lens // page)
    total = int(held.sum()) + spare
    ids = rng.permutation(total)
    table = np.full((B, width), -7, dtype=np.int32)
    n = 0
    for b in range(B):
        table[b, :held[b]] = ids[n:n + held[b]]
        n += held[b]
    free = np.full(total, -9, dtype=np.int32)
    free[:spare] = ids[n:]
    return lens, new, table, free, spare, page, T


def run(ssv, lens, new, table, free, count, page, T, in_place=False):
    t, f = put(table), put(free)
    kw = {}
    if in_place:
        B = len(lens)
        e = lambda *s: torch.empty(*s, dtype=torch.int32, device=DEV)  # noqa: E731
        kw["out"] = ssv.CachePlan(t, f, e(1), e(B), e(B, T), torch.zeros(1, dtype=torch.int32, device=DEV))
    o = ssv.plan_cache(put(lens), put(new), t, f, put([count]), page, T, **kw)
    torch.cuda.synchronize()
    return o


def compare(ssv, case):
    r = decode.plan_cache(*case[:5], case[5], case[6])
    for in_place in (False, True):
        o = run(ssv, *case, in_place=in_place)
        for got, want in ((o.block_table, r.table), (o.free_pages, r.free), (o.free_count, [r.count]),
                          (o.context_lens, r.lens), (o.slots, r.slots)):
            assert got.cpu().numpy().tolist() == np.asarray(want).tolist()
        st = int(o.status.item())
        assert st == (ssv.DEV_BAD_OFFSETS if r.bad else 0) | (ssv.DEV_NO_PAGES if r.short else 0)
    return r


@pytest.mark.parametrize("B,width,page,T,spare", [
    (1, 1, 1, 1, 1), (3, 4, 16, 5, 20), (8, 40, 16, 8, 0), (255, 9, 8, 64, 700), (256, 30, 24, 3, 4),
    (257, 17, 7, 33, 60), (1500, 12, 16, 9, 200), (5000, 5, 3, 4, 40), (2, 3000, 64, 1, 2), (5, 6, 16, 0, 3)])
def test_plan_against_oracle(ssv, B, width, page, T, spare):
    for seed in range(4):
        compare(ssv, plan_case(seed + 10 * B, B, width, page, T, spare))


def test_plan_edges(ssv):
    # a bad length, one that does not fit, too many new ones, all beside good ones
    table = np.array([[0, 1], [2, 3], [4, -1], [5, 6], [7, -1]])
    free = [8, 9, 10, -1]
    for lens, new in (([8, 8, -1, 8, 3], [0, 1, 2, -8, 1]), ([9, 2, 3, 8, 3], [0, 7, 5, -9, 2]),
                      ([8, 8, 3, 8, 3], [2 ** 31 - 1, -2 ** 31, 5, -8, 5]), ([2 ** 31 - 1, -2 ** 31, 0, 0, 0], [1, -1, 0, 0, 4])):
        compare(ssv, (np.array(lens), np.array(new), table, np.array(free), 3, 4, 5))
    # a stack count that cannot be, and more given back than the stack holds: nothing changes
    for count in (-1, 5, 4, 3):
        compare(ssv, (np.array([8, 8, 3, 8, 3]), np.array([0, -8, 5, -8, 5]), table, np.array(free), count, 4, 5))


def test_plan_empty(ssv):
    e = torch.empty(0, dtype=torch.int32, device=DEV)
    o = ssv.plan_cache(e, e, torch.empty(0, 4, dtype=torch.int32, device=DEV), put([3, 2, -1]), put([2]), 16, 4)
    torch.cuda.synchronize()
    assert o.free_count.item() == 2 and o.free_pages.tolist() == [3, 2, -1] and o.slots.shape == (0, 4)


@pytest.mark.parametrize("layers", [0, 1, 5])
@pytest.mark.parametrize("dtype,D,Hkv,page,ragged,tree", [
    (torch.bfloat16, 128, 8, 16, False, False), (torch.float16, 8, 1, 1, True, False),
    (torch.bfloat16, 80, 2, 24, True, True), (torch.float16, 64, 3, 64, False, True)])
def test_commit(ssv, layers, dtype, D, Hkv, page, ragged, tree):
    """layers 0: tensors without that dimension."""
    rng = np.random.default_rng(D)
    B, T, L = 6, 7, max(layers, 1)
    rows = rng.integers(1, T + 1, size=B) if ragged else np.full(B, T)
    off = np.concatenate([[0], np.cumsum(rows)])
    kept = np.array([rng.integers(0, n + 1) for n in rows])
    pages = -(-B * T * 2 // page)
    free = rng.permutation(pages * page)[:B * T].reshape(B, T)
    slots = np.where(np.arange(T) < kept[:, None], free, -1)
    path = np.full((B, T), -1)
    for b in range(B):
        if kept[b] > 1:
            path[b, :kept[b] - 1] = np.sort(rng.choice(rows[b] - 1, kept[b] - 1, replace=False))
    g = torch.Generator(device=DEV).manual_seed(1)
    f = lambda *s: torch.randn(*s, generator=g, device=DEV).to(dtype)  # noqa: E731
    R = int(off[-1])
    qkv = f(L, R, 3 * Hkv * D)  # keys and values as slices of one projection
    kn, vn = (qkv[..., i * Hkv * D:(i + 1) * Hkv * D].view(L, R, Hkv, D) for i in (1, 2))
    kc = f(L, pages, Hkv, page, D).transpose(2, 3)
    vc = f(L, pages, page, Hkv, D)
    want_k, want_v = kc.clone(), vc.clone()
    for b in range(B):
        for i in range(kept[b]):
            r = off[b] + (i if not tree or i == 0 else path[b, i - 1] + 1)
            p, s = divmod(int(slots[b, i]), page)
            want_k[:, p, s], want_v[:, p, s] = kn[:, r], vn[:, r]
    if not ragged:
        kn, vn = (t.unflatten(1, (B, T)) for t in (kn, vn))
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    a = [t if layers else t[0] for t in (kn, vn, kc, vc)]
    ssv.commit_cache(*a, put(slots), path=put(path) if tree else None, row_offsets=put(off) if ragged else None,
                     status=st)
    torch.cuda.synchronize()
    assert torch.equal(kc, want_k) and torch.equal(vc, want_v) and st.item() == 0


def test_commit_skips_what_cannot_be(ssv):
    B, T, D = 3, 4, 16
    kn, vn = (torch.randn(B * T, 2, D, device=DEV).bfloat16() for _ in range(2))
    kc, vc = (torch.zeros(2, 8, 2, D, device=DEV).bfloat16() for _ in range(2))
    for slots, path, off, bits in (
            ([[16, -1], [2 ** 31 - 1, 1], [3, -5]], None, None, ssv.DEV_BAD_PAGE),
            ([[0, 1], [2, 3], [4, 5]], [[3], [-1], [0]], None, ssv.DEV_BAD_OFFSETS),
            ([[0, 1], [2, 3], [4, 5]], [[3], [2 ** 31 - 1], [-2 ** 31]], None, ssv.DEV_BAD_OFFSETS),
            ([[0, 1], [2, 3], [4, 5]], None, [0, 4, 3, 13], ssv.DEV_BAD_OFFSETS),
            ([[0, 1], [2, 3], [4, 5]], None, [0, 1, 2, 4], ssv.DEV_BAD_OFFSETS)):
        kc.zero_(), vc.zero_()
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        a = (kn, vn) if off else (kn.view(B, T, 2, D), vn.view(B, T, 2, D))
        ssv.commit_cache(*a, kc, vc, put(slots), path=None if path is None else put(path),
                         row_offsets=None if off is None else put(off), status=st)
        torch.cuda.synchronize()
        assert st.item() == bits
        want = torch.zeros_like(kc).view(16, 2, D)
        for b in range(B):
            r0, r1 = (off[b], off[b + 1]) if off else (b * T, (b + 1) * T)
            for i in range(2):
                node = -1 if path is None or i == 0 else path[b][i - 1]
                row = i if path is None or i == 0 else node + 1 if node >= 0 else -1  # below 0: no node
                if 0 <= slots[b][i] < 16 and 0 <= r0 <= r1 <= B * T and 0 <= row < r1 - r0:
                    want[slots[b][i]] = kn[r0 + row]
        assert torch.equal(kc.view(16, 2, D), want)


def test_pages_that_no_slot_can_name(ssv):
    """Ids below 0, or whose slots pass 2^31 - 1, in a table's last page and on the stack: the tokens get a
    slot that a commit refuses, not one of another page (2^28 * 16 wraps to 0) and not -1."""
    big = 2 ** 31 - 1
    for page_id in (-1, -2 ** 31, 2 ** 28, 2 ** 28 + 1, 2 ** 27, big):
        table = np.array([[3, page_id, -1], [5, -1, -1], [6, 7, -1]])
        free = [9, page_id, -1, -1]
        for in_place in (False, True):
            # request 0 goes on in its last page, 1 takes the stack's top, 2 stays
            o = run(ssv, [20, 14, 18], [2, 4, 0], table, free, 2, 16, 5, in_place)
            assert int(o.status.item()) == ssv.DEV_BAD_PAGE
            assert o.slots.tolist() == [[big, big, -1, -1, -1], [5 * 16 + 14, 5 * 16 + 15, big, big, -1], [-1] * 5]
            assert o.context_lens.tolist() == [22, 18, 18] and o.free_count.item() == 1
            assert o.block_table[1].tolist() == [5, page_id, -1]
            kn, vn = (torch.randn(3, 5, 1, 8, device=DEV).bfloat16() for _ in range(2))
            kc, vc = (torch.zeros(8, 16, 1, 8, device=DEV).bfloat16() for _ in range(2))
            st = torch.zeros(1, dtype=torch.int32, device=DEV)
            ssv.commit_cache(kn, vn, kc, vc, o.slots, status=st)
            torch.cuda.synchronize()
            assert st.item() == ssv.DEV_BAD_PAGE
            want = torch.zeros_like(kc).view(128, 1, 8)
            want[94:96] = kn[1, :2]
            assert torch.equal(kc.view(128, 1, 8), want)
    # the last slots that 32 bits hold
    o = run(ssv, [14], [2], np.array([[2 ** 27 - 1]]), [-1], 0, 16, 2)
    assert o.slots.tolist() == [[2 ** 31 - 2, 2 ** 31 - 1]] and int(o.status.item()) == 0
    # given back, they name no slot
    o = run(ssv, [20], [-10], np.array([[3, -5]]), [-1], 0, 16, 2)
    assert o.free_pages.tolist() == [-5] and int(o.status.item()) == 0
