"""Attention over the paged cache against the fp64 oracle."""

import numpy as np
import pytest
import torch

from decode_cases import attention_bounds, attention_case, attention_oracle, on_gpu

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def ssv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sampling_spec_verify_gb300 as m
    m.lib()
    return m


def check(ssv, c, dtype, **kw):
    args, more = on_gpu(c)
    o = ssv.tree_attention(*args, want_lse=True, **more, **kw)
    torch.cuda.synchronize()
    r = attention_oracle(c)
    n = c["offsets"][-1]
    got = o.out.reshape(-1, *o.out.shape[-2:]).double().cpu().numpy()[:n]
    lse = o.lse.reshape(-1, o.lse.shape[-1]).double().cpu().numpy()[:n]
    tol, tol_lse = attention_bounds(c, r, dtype)
    off = np.abs(got - r.out[:n]) / tol[:n]
    assert np.isfinite(got).all() and off.max(initial=0.0) <= 1.0, off.max()
    same = np.where(np.isinf(r.lse[:n]), lse == r.lse[:n], np.abs(lse - r.lse[:n]) <= tol_lse[:n])
    assert same.all()
    assert int(o.status.item()) == 0
    return o


CASES = [
    # rows, contexts, Hq, Hkv, D, page, dtype, options
    ([1], [0], 1, 1, 64, 16, BF, {}),
    ([1], [1], 4, 2, 128, 16, BF, {}),
    ([1, 1, 1], [7, 128, 129], 8, 1, 128, 16, HF, {}),
    ([5], [1000], 32, 8, 128, 16, BF, {}),
    ([5, 5], [127, 300], 10, 2, 80, 24, HF, dict(tree=True)),
    ([3, 3, 3], [64, 0, 63], 4, 4, 8, 8, BF, dict(tree=True)),
    ([2, 2], [511, 1100], 6, 2, 256, 32, BF, dict(tree=True)),
    ([2], [90], 2, 2, 248, 8, HF, {}),
    ([33, 33], [700, 90], 8, 2, 128, 64, BF, dict(tree=True)),
    ([65], [257], 8, 1, 64, 128, HF, dict(tree=True)),
    ([40], [130], 16, 2, 128, 16, BF, {}),
    ([150], [40], 2, 1, 64, 16, BF, dict(tree=True)),
    ([300], [0], 3, 1, 72, 40, HF, {}),
    ([1, 7, 3, 0, 5], [100, 0, 333, 50, 16], 6, 2, 128, 16, BF, dict(ragged=True, tree=True, spare_rows=3)),
    ([0, 4, 0], [9, 700, 9], 4, 2, 96, 48, HF, dict(ragged=True, T=9, spare_rows=130)),
    ([4, 4], [200, 500], 8, 2, 128, 16, BF, dict(layout="hnd")),
    ([4, 4], [200, 500], 8, 2, 64, 16, HF, dict(layout="joint", strided=True, tree=True)),
    ([4, 4], [200, 500], 8, 2, 128, 16, HF, dict(layout="joint", strided=True)),
    ([3, 3], [333, 70], 8, 2, 128, 32, BF, dict(layout="mixed", tree=True)),
    ([3, 3], [333, 70], 8, 2, 256, 32, BF, dict(layout="hnd")),
    ([3, 3], [333, 70], 8, 2, 192, 64, HF, dict(layout="joint", tree=True)),
    ([3, 3], [333, 470], 8, 2, 128, 64, BF, dict(layout="apart", tree=True)),
    ([70, 70], [333, 470], 4, 2, 128, 128, BF, dict(layout="hnd", tree=True)),
    ([3], [200], 128, 1, 128, 16, BF, dict(tree=True)),
    ([2, 2], [150, 64], 100, 1, 64, 16, HF, {}),
    ([5], [300], 96, 2, 256, 16, BF, dict(tree=True)),
    ([1024], [70], 1, 1, 16, 8, BF, {}),
    ([500, 500], [0, 130], 2, 1, 64, 64, HF, dict(tree=True)),
    ([i % 4 for i in range(450)], [7 * (i % 40) for i in range(450)], 4, 2, 64, 16, BF, dict(ragged=True, tree=True)),
    ([3, 1], [5000, 9000], 8, 4, 128, 4096, BF, dict(ragged=True)),
    ([7], [1], 5, 1, 104, 16, HF, dict(tree=True)),
    ([130], [121], 1, 1, 128, 16, BF, dict(tree=True)),
    ([9] * 40, list(range(0, 400, 10)), 4, 2, 64, 8, BF, dict(tree=True)),
    ([2], [6000], 4, 1, 128, 160, BF, {}),
    ([20, 20], [300, 170], 30, 2, 192, 16, BF, dict(tree=True)),
    ([6], [2000], 8, 2, 128, 16, BF, dict(spread=4000.0)),
    ([6], [400], 8, 2, 128, 16, HF, dict(spread=40.0)),  # one key takes nearly all of the weight
]


@pytest.mark.parametrize("rows,ctx,Hq,Hkv,D,page,dtype,more", CASES)
def test_against_oracle(ssv, rows, ctx, Hq, Hkv, D, page, dtype, more):
    check(ssv, attention_case(len(rows) * 1000 + ctx[0] + D, rows, ctx, Hq, Hkv, D, page, dtype, **more), dtype)


def test_rows_that_see_nothing(ssv):
    c = attention_case(3, [4, 4], [0, 20], 4, 2, 64, 16, BF, tree=True)
    c["mask"][0, 1] = 0
    c["mask"][1, 2] = 0  # sees the cache alone
    o = check(ssv, c, BF)
    assert not o.out[0, 1].any() and bool((o.lse[0, 1] == float("-inf")).all())


def test_garbage_that_is_not_seen_does_not_enter(ssv):
    c = attention_case(4, [6, 6], [40, 130], 4, 2, 128, 16, BF, tree=True)
    c["mask"][:] = 0
    for i in range(6):
        c["mask"][:, i, 0] = 1
        c["mask"][:, i, i] = 1
    clean = {k: c[k].clone() for k in ("k_new", "v_new")}
    want = check(ssv, c, BF)
    for bad in (float("nan"), float("inf"), float("-inf"), torch.finfo(BF).min):
        for k in ("k_new", "v_new"):
            c[k] = clean[k].clone()
            c[k].view(2, 6, 2, 128)[:, 3, :, 5:9] = bad
        args, kw = on_gpu(c)
        o = ssv.tree_attention(*args, want_lse=True, **kw)
        torch.cuda.synchronize()
        keep = [0, 1, 2, 4, 5]
        assert torch.equal(o.out[:, keep], want.out[:, keep]) and torch.equal(o.lse[:, keep], want.lse[:, keep])
    c["k_new"] = clean["k_new"]  # a value that is seen passes on
    for bad in (float("nan"), float("inf"), float("-inf")):
        c["v_new"] = clean["v_new"].clone()
        c["v_new"].view(2, 6, 2, 128)[:, 3, :, 5:9] = bad
        args, kw = on_gpu(c)
        o = ssv.tree_attention(*args, **kw)
        torch.cuda.synchronize()
        got = o.out[:, 3, :, 5:9].float()
        assert bool(torch.isnan(got).all()) if bad != bad else bool((got == bad).all())
        assert torch.equal(o.out[:, 3, :, 9:], want.out[:, 3, :, 9:])
        assert torch.equal(o.out[:, keep], want.out[:, keep])


def test_values_that_are_not_finite_over_many_units_a_cta(ssv):
    """Units of two row tiles and of one in turn, some with such a value that rows from 5 on see."""
    rows = [40 if i % 3 == 0 else 3 + 30 * (i % 2) for i in range(1500)]
    c = attention_case(9, rows, [i % 21 for i in range(1500)], 4, 1, 64, 16, BF, ragged=True)
    args, kw = on_gpu(c)
    want = ssv.tree_attention(*args, **kw).out
    hit = torch.zeros(sum(rows), dtype=torch.bool)
    at = []
    for b, n in enumerate(rows):
        if b % 5 in (0, 3) and n > 5:
            r = int(c["offsets"][b])
            at.append(r + 5)
            hit[r + 5:r + n] = True
    args[2][torch.tensor(at).cuda(), 0, 17] = float("inf")
    for _ in range(5):
        got = ssv.tree_attention(*args, **kw).out
        torch.cuda.synchronize()
        assert bool((got[hit.cuda(), :, 17] == float("inf")).all())
        back = got.clone()
        back[hit.cuda(), :, 17] = want[hit.cuda(), :, 17]
        assert torch.equal(back, want)


def test_nan_query_stays_in_its_row(ssv):
    c = attention_case(5, [3, 3], [50, 60], 4, 2, 64, 16, HF)
    want = check(ssv, c, HF)
    c["q"][4, 1, 7] = float("nan")
    args, kw = on_gpu(c)
    o = ssv.tree_attention(*args, **kw)
    torch.cuda.synchronize()
    nan = torch.isnan(o.out)
    assert bool(nan[1, 1, 1].all()) and int(nan.sum()) == 64
    assert torch.equal(o.out[~nan], want.out[~nan])


def test_rows_of_nobody_stay(ssv):
    c = attention_case(6, [2, 3], [30, 9], 4, 2, 64, 16, BF, ragged=True, T=4, spare_rows=5)
    args, kw = on_gpu(c)
    out = ssv.AttentionOutput(torch.full_like(args[0], 7.0), torch.full(args[0].shape[:2], 7.0, device="cuda"),
                              torch.zeros(1, dtype=torch.int32, device="cuda"))
    ssv.tree_attention(*args, out=out, want_lse=True, **kw)
    torch.cuda.synchronize()
    assert bool((out.out[5:] == 7).all()) and bool((out.lse[5:] == 7).all()) and not bool((out.out[:5] == 7).all())


def test_bad_lengths_offsets_and_pages(ssv):
    c = attention_case(7, [2, 2, 2], [30, 9, 40], 4, 2, 64, 16, BF, ragged=True, T=3)
    good = check(ssv, c, BF)
    args, kw = on_gpu(c)

    def run(ctx=None, offsets=None, table=None):
        a, k = list(args), dict(kw)
        if ctx is not None:
            a[6] = torch.tensor(ctx, dtype=torch.int32, device="cuda")
        if offsets is not None:
            k["row_offsets"] = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        if table is not None:
            a[5] = torch.from_numpy(table).cuda()
        out = ssv.AttentionOutput(torch.full_like(args[0], 7.0), None, torch.zeros(1, dtype=torch.int32, device="cuda"))
        ssv.tree_attention(*a, out=out, **k)
        torch.cuda.synchronize()
        return out.out, int(out.status.item())

    o, st = run(ctx=[30, -4, 40])  # counts as 0
    o0, st0 = run(ctx=[30, 0, 40])
    assert st == ssv.DEV_BAD_OFFSETS and st0 == 0 and torch.equal(o, o0)
    _, st = run(ctx=[30, 10 ** 6, 40])
    assert st & ssv.DEV_BAD_OFFSETS
    for offsets in ([0, 2, 4, 7], [0, 2, 1, 6], [-1, 2, 4, 6], [0, 2, 6, 6]):
        o, st = run(offsets=offsets)
        assert st == ssv.DEV_BAD_OFFSETS
        assert torch.equal(o[:2], good.out[:2]) or offsets[0] == -1
    assert bool((run(offsets=[0, 2, 6, 6])[0][2:] == 7).all())
    # pages outside the cache read as zeros
    for page in (-1, -2 ** 31, 10 ** 9, int(args[3].shape[0])):
        t = c["table"].copy()
        t[2, 1] = page
        o, st = run(table=t)
        assert st == ssv.DEV_BAD_PAGE and torch.equal(o[:4], good.out[:4])
        d = dict(c, table=t)
        r = attention_oracle(d)
        assert (np.abs(o[4:6].double().cpu().numpy() - r.out[4:6]) <= attention_bounds(d, r, BF)[0][4:6]).all()


def test_no_cache_at_all(ssv):
    c = attention_case(8, [3], [0], 2, 1, 64, 16, BF)
    args, kw = on_gpu(c)
    want = ssv.tree_attention(*args, **kw).out
    args[3] = args[4] = torch.empty(0, 16, 1, 64, dtype=BF, device="cuda")
    args[5] = torch.empty(1, 0, dtype=torch.int32, device="cuda")
    assert torch.equal(ssv.tree_attention(*args, **kw).out, want)
    e = ssv.tree_attention(args[0][:0], args[1][:0], args[2][:0], args[3], args[4], args[5][:0], args[6][:0])
    assert e.out.shape[0] == 0


def test_pages_of_an_empty_cache_read_as_zeros(ssv):
    c = attention_case(12, [3], [20], 2, 1, 64, 16, BF, poison=False)
    c["table"][:] = 0
    c["k_cache"], c["v_cache"] = c["k_cache"][:0], c["v_cache"][:0]
    args, kw = on_gpu(c)
    o = ssv.tree_attention(*args, **kw)
    torch.cuda.synchronize()
    r = attention_oracle(dict(c, k_cache=torch.zeros(1, 16, 1, 64, dtype=BF), v_cache=torch.zeros(1, 16, 1, 64, dtype=BF)))
    c["v_cache"] = torch.zeros(1, 16, 1, 64, dtype=BF)
    tol = attention_bounds(c, r, BF)[0]
    assert int(o.status.item()) == ssv.DEV_BAD_PAGE
    assert (np.abs(o.out[0].double().cpu().numpy() - r.out) <= tol).all()


@pytest.mark.parametrize("B,T,Hq,Hkv,D,page,tree", [(128, 1, 16, 4, 128, 16, False), (48, 33, 8, 2, 128, 32, True),
                                                    (64, 5, 8, 4, 192, 16, True), (96, 9, 4, 4, 64, 64, False)])
def test_many_units_a_cta_give_the_same_bits(ssv, B, T, Hq, Hkv, D, page, tree):
    """Units that follow each other in a CTA and go on in the next: their products, results and
    maxima may not run into each other (a result read before its last product was such a fault)."""
    ctx = [(37 * i) % 2100 for i in range(B)]
    c = attention_case(13, [T] * B, ctx, Hq, Hkv, D, page, BF, tree=tree)
    args, kw = on_gpu(c)
    first = ssv.tree_attention(*args, want_lse=True, **kw)
    q, kn, vn, kc, vc, table, lens = args
    for b in range(0, B, 5):  # against 64 bits
        n = int(lens[b])
        ids = table[b, :-(-n // page)].long()
        old = lambda t: t[ids].flatten(0, 1)[:n].double()  # noqa: E731
        k, v = torch.cat([old(kc), kn[b].double()]), torch.cat([old(vc), vn[b].double()])
        sees = torch.ones(T, n + T, dtype=torch.bool, device="cuda")
        sees[:, n:] = kw["mask"][b] != 0 if tree else torch.ones(T, T, device="cuda").tril() != 0
        k, v = (t.repeat_interleave(Hq // Hkv, dim=1) for t in (k, v))
        s = torch.einsum("thd,nhd->htn", q[b].double(), k) * c["scale"]
        p = torch.softmax(s.masked_fill(~sees, float("-inf")), dim=2)
        want, mass = torch.einsum("htn,nhd->thd", p, v), torch.einsum("htn,nhd->thd", p, v.abs())
        # a rounding of every weight and one of the result; scores within 2^-10 of themselves
        assert bool(((first.out[b].double() - want).abs() <= 2.0 ** -8 * 1.01 * (mass + want.abs()) + 2.0 ** -8 * mass / 8).all())
    for _ in range(30):
        o = ssv.tree_attention(*args, want_lse=True, **kw)
        assert torch.equal(o.out, first.out) and torch.equal(o.lse, first.lse)


def test_same_bits_again_on_a_stream_and_in_a_graph(ssv):
    c = attention_case(9, [8, 8], [3000, 500], 8, 2, 128, 16, BF, tree=True)
    args, kw = on_gpu(c)
    first = ssv.tree_attention(*args, want_lse=True, **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = ssv.tree_attention(*args, want_lse=True, stream=s, **kw)
    s.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(ssv.tree_attention(*args, want_lse=True, **kw))
        graphs.append(g)
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    for o in (other, *outs):
        assert torch.equal(o.out, first.out) and torch.equal(o.lse, first.lse)
    # other lengths in the same graph
    args[6].copy_(torch.tensor([17, 2900], dtype=torch.int32))
    args[5].copy_(args[5].flip(0))
    want = ssv.tree_attention(*args, want_lse=True, **kw)
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0].out, want.out)


def test_cache_beyond_32_bits(ssv):
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    page, Hkv, D = 64, 8, 128
    pages = (5 << 30) // (page * Hkv * D)  # 5 Gi elements
    c = attention_case(10, [4], [190], 8, Hkv, D, page, BF, poison=False)
    args, kw = on_gpu(c)
    want = ssv.tree_attention(*args, **kw)
    kc, vc = (torch.empty(pages, page, Hkv, D, dtype=BF, device="cuda") for _ in range(2))
    t = args[5].clone()
    n = t[0, :3].long()
    far = torch.tensor([pages - 1, pages // 2 + 1, pages - 7], device="cuda")
    kc[far], vc[far] = args[3][n], args[4][n]
    t[0, :3] = far.int()
    o = ssv.tree_attention(*args[:3], kc, vc, t, args[6], **kw)
    torch.cuda.synchronize()
    assert torch.equal(o.out, want.out)


def test_given_scale(ssv):
    c = attention_case(11, [3, 3], [100, 20], 4, 2, 64, 16, BF)
    c["scale"] = 0.37
    check(ssv, c, BF, scale=0.37)
    c["scale"] = 0.0  # the mean of what is seen
    check(ssv, c, BF, scale=0.0)
    c["scale"] = -0.2
    check(ssv, c, BF, scale=-0.2)


def test_calls_at_once_on_streams_and_threads(ssv):
    import threading

    cases = [on_gpu(attention_case(20 + i, [4 + i] * 6, [500 * i + 90 * j for j in range(6)], 8, 2, 128, 16, BF, tree=True))
             for i in range(4)]
    want = [ssv.tree_attention(*a, **kw).out for a, kw in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[] for _ in cases]
    for _ in range(10):
        for i, (a, kw) in enumerate(cases):
            got[i].append(ssv.tree_attention(*a, stream=streams[i], **kw).out)

    def work(i):  # all threads on the default stream, whose workspace they share
        a, kw = cases[i]
        for _ in range(10):
            got[i].append(ssv.tree_attention(*a, **kw).out)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    for w, outs in zip(want, got):
        assert len(outs) == 20 and all(torch.equal(w, o) for o in outs)


def two_kinds_of_keys(T, ctx, D, page, dtype, top, rest, value_top, value_rest):
    """One request and head whose queries are 1 in component 0 and 0 elsewhere: the first cached key holds top
    there, all others rest, and their values are value_top and value_rest throughout."""
    c = attention_case(3, [T], [ctx], 1, 1, D, page, dtype, poison=False)
    for k in ("q", "k_new", "k_cache"):
        c[k].zero_()
    c["q"][:, 0, 0] = 1.0
    at = torch.arange(ctx)
    ids, place = torch.from_numpy(c["table"])[0].long()[at // page], at % page
    c["k_cache"][ids, place, 0, 0] = torch.where(at < 1, float(top), float(rest)).to(dtype)
    c["k_new"][:, 0, 0] = float(rest)
    c["v_cache"][ids, place] = torch.where(at[:, None, None] < 1, float(value_top), float(value_rest)).to(dtype)
    c["v_new"].fill_(float(value_rest))
    return c


@pytest.mark.parametrize("dtype,exponents", [(BF, (8, 20, 27, 34, 60)), (HF, (8, 20, 26, 29))])
@pytest.mark.parametrize("T,ctx,D", [(1, 300, 64), (2, 20000, 128), (130, 700, 128), (3, 500, 192)])
def test_scores_of_any_size(ssv, dtype, exponents, T, ctx, D):
    """Scores that fp32 holds exactly, of which the largest occurs several times and the next is
    half of it: the result is those keys' mean, however large they are."""
    for e in exponents:
        for m in (1.0, 1.125, 1.375, 1.75):
            c = two_kinds_of_keys(T, ctx, D, 16, dtype, 0.0, 0.0, 0.0, 1.0)
            hi, lo = e // 2, e - e // 2
            c["q"][:, 0, 0] = m * 2.0 ** hi
            at = torch.arange(ctx)
            ids, place = torch.from_numpy(c["table"])[0].long()[at // 16], at % 16
            top = at % 97 == 5
            c["k_cache"][ids, place, 0, 0] = torch.where(top, 1.25 * 2.0 ** lo, 1.25 * 2.0 ** (lo - 1)).to(dtype)
            c["v_cache"][ids, place] = torch.where(top, (at % 7).float(), 100.0)[:, None, None].to(dtype)
            args, kw = on_gpu(c)
            o = ssv.tree_attention(*args, scale=1.0, want_lse=True, **kw)
            torch.cuda.synchronize()
            score = m * 1.25 * 2.0 ** e
            w = np.where(top.numpy(), 1.0, np.exp(-score / 2))  # below 2^-126 from 2^8 on
            want = float((w * np.where(top.numpy(), at.numpy() % 7, 100.0)).sum() / w.sum())
            got = o.out.double().cpu().numpy()
            # weights of one size round alike; the result's own rounding, sums in fp32
            assert (np.abs(got - want) <= want * (torch.finfo(dtype).eps / 2 * 1.01 + 2.0 ** -18)).all(), (e, m, want)
            lse = score + np.log(w.sum())
            assert (np.abs(o.lse.double().cpu().numpy() - lse) <= 2.0 ** -16 + 2.0 ** -22 * lse).all(), (e, m)


@pytest.mark.parametrize("gap", [16.5, 20.5, 24.5, 25.5, 28.25, 30.5])
@pytest.mark.parametrize("T,D", [(1, 64), (130, 128), (1, 192)])
def test_many_small_weights_in_fp16(ssv, gap, T, D):
    """20000 keys of a weight 2^-gap of the largest one, which among fp16's steps of 2^-24 would be off by
    up to half of itself or gone: weights are rounded at 2^11 times their size, so each is off by 2^-11 of
    itself or, below the normal range, by 2^-36 of the largest one.  Enough requests that a
    unit's keys meet in one CTA (over the same pages)."""
    B, n_cached = 300, 20000
    c = two_kinds_of_keys(T, n_cached, D, 64, HF, gap, 0.0, 0.0, 1.0)
    scale = float(np.log(2.0))
    args, kw = on_gpu(c)
    for i in (0, 1, 2, 5, 6):
        args[i] = args[i].repeat(B, *[1] * (args[i].dim() - 1))
    o = ssv.tree_attention(*args, scale=scale, want_lse=True)
    torch.cuda.synchronize()
    n = n_cached + np.arange(T)[:, None, None]  # small weights, the pass's own keys among them
    w = 2.0 ** -gap
    want = n * w / (1.0 + n * w)
    # the weights' rounding and the result's, and n sums in fp32; then what is below the normal ranges
    tol = (2 * 2.0 ** -11 + n * 2.0 ** -24) * want + n * 2.0 ** -36 + 2.0 ** -25
    off = np.abs(o.out.double().cpu().numpy() - want) / tol
    assert off.max() <= 1.0, off.max()
    lse = gap * np.log(2.0) + np.log1p(n[..., 0] * w)
    assert (np.abs(o.lse.double().cpu().numpy() - lse) <= n[..., 0] * 2.0 ** -24 + 2.0 ** -22 * lse).all()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("T,ctx,D", [(1, 100, 64), (2, 30000, 128), (130, 300, 128), (3, 500, 192), (2, 9000, 256)])
@pytest.mark.parametrize("value", [float("inf"), float("nan"), 1.0])
def test_only_scores_of_minus_infinity(ssv, dtype, T, ctx, D, value):
    """Such a row gets zeros and -inf, whatever the values hold."""
    c = two_kinds_of_keys(T, ctx, D, 16, dtype, float("-inf"), float("-inf"), value, value)
    args, kw = on_gpu(c)
    o = ssv.tree_attention(*args, scale=1.0, want_lse=True, **kw)
    torch.cuda.synchronize()
    assert not o.out.any() and bool((o.lse == float("-inf")).all()) and int(o.status.item()) == 0


@pytest.mark.parametrize("rows,Hq,Hkv,D", [([3], 2, 1, 64), ([40], 8, 2, 128), ([5], 2, 1, 192), ([2, 2], 2, 2, 80)])
def test_no_cache_at_all_raises_nothing(ssv, rows, Hq, Hkv, D):
    c = attention_case(8, rows, [0] * len(rows), Hq, Hkv, D, 16, BF)
    args, kw = on_gpu(c)
    want = ssv.tree_attention(*args, **kw)
    args[3] = args[4] = torch.empty(0, 16, Hkv, D, dtype=BF, device="cuda")
    args[5] = torch.empty(len(rows), 0, dtype=torch.int32, device="cuda")
    o = ssv.tree_attention(*args, **kw)
    assert torch.equal(o.out, want.out) and int(o.status.item()) == 0 and int(want.status.item()) == 0
