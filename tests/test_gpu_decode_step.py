"""A decoding loop of trees: cache plan, attention over the paged cache, rules on the
logits, greedy tree verify, plan and commit, against decoding one token after the
other in 64 bits."""

import numpy as np
import pytest
import torch

from decode_cases import random_parents

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def ssv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sampling_spec_verify_gb300 as m
    m.lib()
    return m


class Model:
    """One attention layer over token embeddings, and a head."""

    V, Hq, Hkv, D = 97, 4, 2, 64

    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        f = lambda *s: torch.randn(*s, generator=g).bfloat16()  # noqa: E731
        self.q, self.k, self.v = f(self.V, self.Hq, self.D), f(self.V, self.Hkv, self.D), f(self.V, self.Hkv, self.D)
        self.head = 4 * torch.randn(self.Hq * self.D, self.V, generator=g)

    def on(self, dev):
        c = Model.__new__(Model)
        c.__dict__ = {k: v.to(dev) for k, v in self.__dict__.items()}
        return c

    def logits(self, tokens, prompt, rep, freq, pres):
        """The logits after `tokens` in 64 bits, and how far bf16 attention may be off them: a rounding of
        every weight (2^-8 of the mass) and of the result, an eighth more for the fp32 sums, through the head
        and the repetition penalty."""
        t = torch.tensor(tokens)
        q, k, v = self.q[t[-1]].double(), self.k[t].double(), self.v[t].double()
        k, v = (x.repeat_interleave(self.Hq // self.Hkv, dim=1) for x in (k, v))
        p = torch.softmax(torch.einsum("hd,nhd->hn", q, k) / self.D ** 0.5, dim=1)
        out = torch.einsum("hn,nhd->hd", p, v).reshape(-1)
        mass = torch.einsum("hn,nhd->hd", p, v.abs()).reshape(-1)
        off = 2.0 ** -8 * 1.125 * (mass + out.abs()) @ self.head.double().abs() * rep
        z = out @ self.head.double()
        made = np.bincount(tokens[prompt:], minlength=self.V)
        for x in range(self.V):
            if made[x] or x in tokens[:prompt]:
                z[x] = z[x] / rep if z[x] > 0 else z[x] * rep
            z[x] -= freq * made[x] + pres * (made[x] > 0)
        return z, off


@pytest.mark.parametrize("seed,page", [(1, 16), (2, 8)])
def test_trees_decode_what_single_tokens_do(ssv, seed, page):
    rng = np.random.default_rng(seed)
    cpu, B, N, steps = Model(seed), 5, 7, 9
    m = cpu.on(DEV)
    rep, freq, pres = 1.2, 0.3, 0.4
    prompts = [rng.integers(0, m.V, size=n).tolist() for n in (3, 40, 17, 129, 64)]
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    width, T = 24, N + 1
    pages = B * width
    plan = ssv.CachePlan(torch.full((B, width), -1, dtype=torch.int32, device=DEV),
                         i32(rng.permutation(pages).tolist()), i32([pages]), torch.zeros(B, dtype=torch.int32, device=DEV),
                         None, None)
    cache = [torch.full((pages, page, m.Hkv, m.D), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2)]

    def commit(plan, new, k, v, most, path=None, **kw):
        out = ssv.plan_cache(plan.context_lens, new, plan.block_table, plan.free_pages, plan.free_count, page, most)
        ssv.commit_cache(k, v, *cache, out.slots, path=path, **kw)
        return out

    # the prompts but for their last token, as one ragged pass
    rows = [p[:-1] for p in prompts]
    flat = i32(sum(rows, []))
    offsets = i32(np.cumsum([0] + [len(r) for r in rows]).tolist())
    plan = commit(plan, i32([len(r) for r in rows]), m.k[flat.long()], m.v[flat.long()], 130, row_offsets=offsets)
    tokens = [list(p) for p in prompts]
    for step in range(steps):
        parent = np.stack([random_parents(rng, T) for _ in range(B)])
        drafted = np.zeros((B, T), dtype=np.int32)
        for b in range(B):  # the root is the last committed token; nodes often guess right
            drafted[b, 0] = tokens[b][-1]
            depth, ahead = np.zeros(T, dtype=int), list(tokens[b])
            for _ in range(T):
                ahead.append(int(cpu.logits(ahead, len(prompts[b]), rep, freq, pres)[0].argmax()))
            for i in range(1, T):
                depth[i] = depth[parent[b, i]] + 1
                drafted[b, i] = ahead[len(tokens[b]) - 1 + depth[i]] if rng.uniform() < 0.6 else rng.integers(0, m.V)
        ids = torch.from_numpy(drafted).to(DEV)
        mask, _ = ssv.tree_mask(torch.from_numpy(parent).to(DEV))
        q, k, v = m.q[ids.long()], m.k[ids.long()], m.v[ids.long()]
        o = ssv.tree_attention(q, k, v, *cache, plan.block_table, plan.context_lens, mask=mask)
        logits = (o.out.float().reshape(B, T, -1) @ m.head).contiguous()
        # all committed tokens are history, the root among them: its row's token is not counted again
        most = max(len(t) for t in tokens)
        hist = i32([t + [0] * (most - len(t)) for t in tokens])
        f = lambda x: torch.full((B,), x, device=DEV)  # noqa: E731
        counted = torch.cat([torch.full_like(ids[:, :1], -1), ids[:, 1:]], 1)
        logits = ssv.adjust_logits(logits, counted, hist, i32([len(t) for t in tokens]),
                                   prompt_lens=i32([len(p) for p in prompts]), repetition=f(rep), frequency=f(freq),
                                   presence=f(pres), mask=mask)
        verdict = ssv.tree_verify_greedy(logits, torch.from_numpy(parent[:, 1:] - 1).to(DEV).contiguous(),
                                         ids[:, 1:].contiguous())
        plan = commit(plan, verdict.n_accepted + 1, k, v, T, path=verdict.path)
        torch.cuda.synchronize()
        for b, n in enumerate(verdict.n_accepted.tolist()):
            for x in verdict.tokens[b, :n + 1].tolist():
                z, off = cpu.logits(tokens[b], len(prompts[b]), rep, freq, pres)
                assert bool((z[x] + off[x] >= z - off).all()), (step, b, n)
                tokens[b].append(x)
        assert plan.context_lens.tolist() == [len(t) - 1 for t in tokens] and int(plan.status.item()) == 0
    assert max(len(t) - len(p) for t, p in zip(tokens, prompts)) > steps  # trees were accepted
    # all requests done: their pages come back, each once
    plan = ssv.plan_cache(plan.context_lens, -plan.context_lens, plan.block_table, plan.free_pages, plan.free_count, page, 1)
    torch.cuda.synchronize()
    assert int(plan.free_count) == pages and sorted(plan.free_pages.tolist()) == list(range(pages))
