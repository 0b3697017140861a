"""Rules on a pass's logits against the fp64 oracle."""

import numpy as np
import pytest
import torch

from decode_cases import tree_masks
from oracle import decode

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ssv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sampling_spec_verify_gb300 as m
    m.lib()
    return m


def case(seed, rows, V, H, dtype, biases=0, grammar=False, tree=False, prompts=True, T=None, spare=0):
    rng = np.random.default_rng(seed)
    B, T, R = len(rows), T or max(rows), sum(rows) + spare
    few = max(1, min(V, 40))  # repeats
    tok = lambda *s: np.where(rng.uniform(size=s) < 0.5, rng.integers(0, few, size=s), rng.integers(0, V, size=s))  # noqa: E731
    lens = rng.integers(0, H + 1, size=B)
    c = dict(z=torch.from_numpy((2.5 * rng.normal(size=(R, V))).astype(np.float32)).to(dtype), tokens=tok(R),
             history=tok(B, H), lens=lens, prompts=rng.integers(0, lens + 1) if prompts else None,
             repetition=rng.uniform(0.8, 1.6, size=B).astype(np.float32),
             frequency=rng.uniform(-0.1, 0.5, size=B).astype(np.float32),
             presence=rng.uniform(-0.5, 1.0, size=B).astype(np.float32), bias_ids=None, bias=None, allowed=None,
             mask=tree_masks(rng, B, T) if tree else None, offsets=np.concatenate([[0], np.cumsum(rows)]), T=T)
    if biases:
        c["bias_ids"] = np.where(rng.uniform(size=(B, biases)) < 0.2, -1, tok(B, biases))
        c["bias"] = (3 * rng.normal(size=(B, biases))).astype(np.float32)
    if grammar:
        c["allowed"] = rng.integers(0, 2 ** 32, size=(R, -(-V // 32)), dtype=np.uint32)
        c["allowed"][0] = 0  # nothing is allowed
    return c


def call(ssv, c, ragged, z=None, **kw):
    B, T = len(c["lens"]), c["T"]
    i32 = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a).astype(np.int64).astype(np.uint32).view(np.int32) if a.dtype == np.uint32 else np.ascontiguousarray(a, dtype=np.int32)).to(DEV)  # noqa: E731
    f32 = lambda a: None if a is None else torch.from_numpy(a).to(DEV)  # noqa: E731
    z = c["z"].to(DEV) if z is None else z
    fit = (lambda t: t) if ragged else (lambda t: None if t is None else t.view(B, T, *t.shape[1:]))
    if ragged:
        kw.update(row_offsets=i32(c["offsets"]), max_rows=T)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = ssv.adjust_logits(fit(z), fit(i32(c["tokens"])), i32(c["history"]), i32(c["lens"]),
                            prompt_lens=i32(c["prompts"]), repetition=f32(c["repetition"]),
                            frequency=f32(c["frequency"]), presence=f32(c["presence"]), bias_ids=i32(c["bias_ids"]),
                            bias=f32(c["bias"]), allowed=fit(i32(c["allowed"])),
                            mask=None if c["mask"] is None else torch.from_numpy(c["mask"]).to(DEV), status=st, **kw)
    torch.cuda.synchronize()
    return out.reshape(-1, out.shape[-1]), int(st.item())


def want_of(c):
    return decode.adjust_logits(c["z"].double().numpy(), c["tokens"], c["offsets"], c["mask"], c["history"], c["lens"],
                                c["prompts"], c["repetition"], c["frequency"], c["presence"], c["bias_ids"], c["bias"],
                                c["allowed"])


def agree(c, got, dtype):
    """At most eight fp32 roundings of values no larger than the sum of what enters, then one to dtype."""
    want = want_of(c)
    n = c["offsets"][-1]
    got, want = got.double().cpu().numpy()[:n], want[:n]
    scale = np.abs(c["z"].double().numpy()[:n]) * 2 + 2.0
    if c["frequency"] is not None:
        scale = scale + 0.5 * (c["history"].shape[1] + c["T"])
    if c["bias"] is not None:
        scale = scale + np.abs(c["bias"]).sum(axis=1).max()
    fin = np.isfinite(want)
    assert (got[~fin] == want[~fin]).all()
    u = torch.finfo(dtype).eps / 2 if dtype != F else 0.0
    assert (np.abs(got - want)[fin] <= (u * np.abs(want) + 8 * 2.0 ** -24 * scale)[fin]).all()


@pytest.mark.parametrize("rows,V,H,dtype,biases,grammar,tree,ragged", [
    ([1], 1, 1, F, 0, False, False, False), ([3], 31, 5, F, 4, True, False, False),
    ([5], 1000, 700, BF, 0, False, False, False), ([2, 2], 4097, 300, BF, 20, True, True, False),
    ([7, 1, 0, 4], 5003, 100, F, 8, True, True, True), ([9] * 3, 50257, 2000, BF, 64, True, True, False),
    ([17] * 2, 50257, 2000, F, 64, True, True, False), ([8] * 20, 32000, 900, BF, 300, True, False, False),
    ([4, 3], 151936, 4000, BF, 1024, True, False, True), ([2], 129280, 3, F, 0, True, False, False),
    ([40], 777, 0, BF, 3, False, True, False), ([70], 3001, 60, F, 9, True, True, False),
    ([100, 65], 4096, 500, BF, 0, True, False, True), ([1] * 50, 20000, 9000, BF, 5, True, False, False),
    ([1] * 50, 9001, 9000, F, 5, False, False, False)])
def test_against_oracle(ssv, rows, V, H, dtype, biases, grammar, tree, ragged):
    c = case(V + len(rows), rows, V, H, dtype, biases, grammar, tree, spare=2 if ragged else 0)
    got, st = call(ssv, c, ragged)
    agree(c, got, dtype)
    assert st == 0
    z = c["z"].to(DEV)  # in place
    there, _ = call(ssv, c, ragged, z=z, out=z if ragged else z.view(len(rows), c["T"], V))
    n = c["offsets"][-1]
    assert torch.equal(there[:n], got[:n]) and there.data_ptr() == z.data_ptr()
    assert torch.equal(z[n:].cpu(), c["z"][n:])  # rows of nobody


def test_untouched_rows_are_copied_bit_by_bit(ssv):
    c = case(1, [2], 4099, 0, BF, prompts=False)
    c.update(tokens=np.array([-1, -1]), repetition=None, frequency=None, presence=None)
    bits = torch.randint(-2 ** 15, 2 ** 15, (2, 4099), dtype=torch.int16, generator=torch.Generator().manual_seed(2))
    got, st = call(ssv, c, False, z=bits.view(BF).to(DEV))
    assert torch.equal(got.view(torch.int16).cpu(), bits) and st == 0


@pytest.mark.parametrize("dtype,V,shift_in,shift_out", [(BF, 4096, 1, 1), (BF, 5001, 0, 3), (F, 4096, 1, 0), (F, 777, 2, 2)])
def test_memory_off_16_bytes(ssv, dtype, V, shift_in, shift_out):
    c = case(7, [3, 3], V, 200, dtype, 12, True, True)
    want, _ = call(ssv, c, False)
    big = torch.zeros(6 * V + 8, dtype=dtype, device=DEV)
    z = big[shift_in:shift_in + 6 * V].view(6, V).copy_(c["z"])
    out = torch.full((6 * V + 16,), 7.0, dtype=dtype, device=DEV)
    got, st = call(ssv, c, False, z=z, out=out[8 + shift_out:8 + shift_out + 6 * V].view(2, 3, V))
    assert torch.equal(got, want) and st == 0
    assert bool((out[:8 + shift_out] == 7).all()) and bool((out[8 + shift_out + 6 * V:] == 7).all())


def test_special_values(ssv):
    low, inf, nan = torch.finfo(BF).min, float("inf"), float("nan")
    c = case(3, [1], 64, 8, BF, prompts=False)
    c["z"][0, :8] = torch.tensor([low, inf, -inf, nan, 0.0, -0.0, 1.0, low])
    c.update(history=np.arange(8)[None], lens=np.array([7]), tokens=np.array([-1]))
    c.update(repetition=np.array([2.0], dtype=np.float32), frequency=None, presence=None)
    got, st = call(ssv, c, False)
    assert st == 0
    assert got[0, :8].tolist()[:3] == [-inf, inf, -inf] and bool(torch.isnan(got[0, 3]))
    assert got[0, 4:8].tolist() == [0.0, 0.0, 0.5, torch.tensor(low).to(BF).item()]


def test_what_is_outside_counts_for_nothing(ssv):
    base = case(4, [3, 3], 500, 20, F, biases=6, prompts=True)
    good, st = call(ssv, base, False)
    assert st == 0
    c = dict(base, history=np.concatenate([base["history"], np.full((2, 1), 3)], axis=1))
    for key, at, value in (("history", (0, 0), 500), ("history", (0, 0), -1), ("tokens", (1,), 500),
                           ("tokens", (1,), -2), ("bias_ids", (1, 2), 2 ** 31 - 1), ("bias_ids", (1, 2), -3)):
        c = {k: v.copy() if isinstance(v, np.ndarray) else v for k, v in base.items()}
        c["lens"][0], c["prompts"][0] = 20, 1
        c[key][at] = value
        got, st = call(ssv, c, False)
        assert st == ssv.DEV_BAD_TOKEN
        agree(c, got, F)
    for lens, prompts in (([21, 4], [1, 2]), ([-1, 4], [0, 2]), ([5, 4], [6, 2]), ([5, 4], [-1, 2])):
        c = dict(base, lens=np.array(lens), prompts=np.array(prompts))
        got, st = call(ssv, c, False)
        assert st == ssv.DEV_BAD_OFFSETS
        agree(c, got, F)
    c = dict(base, offsets=np.array([0, 4, 3]))
    got, st = call(ssv, c, True, out=base["z"].to(DEV).clone().zero_())
    assert st == ssv.DEV_BAD_OFFSETS and not got.any()


def test_same_bits_in_a_graph_and_on_a_stream(ssv):
    c = case(6, [4] * 8, 32000, 500, BF, 30, True, True)
    want, _ = call(ssv, c, False)
    s = torch.cuda.Stream()
    got, _ = call(ssv, c, False, stream=s)
    assert torch.equal(got, want)
    z = c["z"].to(DEV).view(8, 4, 32000)
    t = torch.from_numpy(c["tokens"].astype(np.int32)).to(DEV).view(8, 4)
    h = torch.from_numpy(c["history"].astype(np.int32)).to(DEV)
    n = torch.from_numpy(c["lens"].astype(np.int32)).to(DEV)
    r = torch.from_numpy(c["repetition"]).to(DEV)
    eager = ssv.adjust_logits(z, t, h, n, repetition=r)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o = ssv.adjust_logits(z, t, h, n, repetition=r)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, eager)


def bits_of(t):
    return t.contiguous().view(torch.int32).cpu()


def test_a_bias_alone_is_added_whole(ssv):
    """z = 0: the result is the bias, to its last bit, in a long slice's list as in a short one."""
    for V, n in ((50, 40), (20000, 1000), (3000, 1024)):
        c = case(11, [1, 1], V, 1, F, prompts=False)
        rng = np.random.default_rng(V)
        c["z"].zero_()
        word = rng.integers(0, 2 ** 32, size=(2, n), dtype=np.uint64).astype(np.uint32)
        word[:, :6] = [1, 0x3DCCCCCD, 0x7F800001, 0x80000001, 0x7FC00001, 0xFF800000]
        c.update(tokens=np.array([-1, -1]), lens=np.array([0, 0]), repetition=None, frequency=None, presence=None,
                 bias_ids=np.stack([rng.permutation(V)[:n] for _ in range(2)]), bias=word.view(np.float32))
        got, st = call(ssv, c, False)
        got, want = bits_of(got).numpy().view(np.uint32), word
        for b in range(2):
            have = got[b][c["bias_ids"][b]]
            nan = np.isnan(want[b].view(np.float32))
            zero = want[b] == 0x80000000  # 0 + -0
            assert (np.isnan(have.view(np.float32)) == nan).all()
            assert (have == want[b])[~nan & ~zero].all() and st == 0


def test_a_row_that_is_not_seen_changes_no_bit(ssv):
    """Row 0 of a tree with and without a sibling, which it does not see, that drafts the tokens that have biases,
    penalties and a place in the history."""
    for V, rows in ((3000, 70), (5001, 9), (40000, 33)):
        c = case(12, [rows, rows], V, 500, F, biases=200, tree=True)
        c["mask"][:] = np.eye(rows, dtype=np.uint8)
        rng = np.random.default_rng(rows)
        c["tokens"] = np.where(rng.uniform(size=2 * rows) < 0.5, c["history"].ravel()[:2 * rows], c["bias_ids"].ravel()[:2 * rows])
        alone = dict(c, tokens=c["tokens"].copy())
        keep = [0, rows]
        alone["tokens"][[i for i in range(2 * rows) if i not in keep]] = -1
        got, want = call(ssv, c, False)[0], call(ssv, alone, False)[0]
        assert torch.equal(bits_of(got)[keep], bits_of(want)[keep])


@pytest.mark.parametrize("rep", [1.1, 1.3, 3.0, 0.7, 7e-40, 3e38, 1e-42])
def test_the_repetition_penalty_divides(ssv, rep):
    """Bit by bit z / r above zero and z r elsewhere, for tokens of the history, drafted ones and those
    in no vector."""
    V = 1003
    c = case(13, [2, 1], V, 900, F, T=2)
    c = dict(c, repetition=np.full(2, rep, dtype=np.float32), frequency=None, presence=None)
    c["z"].mul_(1e-3 if rep > 1e-30 else 1e-39)
    got, st = call(ssv, c, True)
    r = torch.tensor(rep, dtype=torch.float32)
    for b, at in ((0, 0), (0, 1), (1, 2)):
        seen = torch.zeros(V, dtype=torch.bool)
        seen[torch.from_numpy(c["history"][b, :c["lens"][b]]).long()] = True
        seen[torch.from_numpy(c["tokens"][c["offsets"][b]:at + 1]).long()] = True
        z = c["z"][at]
        want = torch.where(seen, torch.where(z > 0, z / r, z * r), z)
        assert torch.equal(got[at].cpu(), want) and st == 0
