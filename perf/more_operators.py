"""The operators of a decoding step around the verify, as measured workloads.

* ``attn``   -- attention of a pass's rows (a chain or a tree of drafted tokens, one
  token in plain decoding) over a paged cache and the pass's own keys and values;
* ``plan``   -- block tables, free pages and slot maps from request lengths;
* ``commit`` -- keys and values of the accepted rows into their slots of the cache;
* ``adjust`` -- penalties, biases and grammar masks on the pass's logits.

``run`` makes the library's calls where ``own`` is true and computes the same in
elementary torch operations otherwise; ``exact`` gives the 64-bit answer.
"""

import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}

# exact() computes products in fp64; beyond this many operations it would take too long
EXACT_FLOPS = 4e12

# drawn cases stay within the largest listed ones
MAX_KEY_HEADS = 2 * 131072 * 8    # cached tokens of the batch x key heads
MAX_ATTN_FLOPS = 3e11
MAX_LOGITS = 128 * 8 * 129280


def listed():
    return [
        # one request, a chain of 4 drafted tokens after the last committed one: latency
        dict(name="attn_b1_t5_c1000", op="attn", B=1, T=5, lo=1000, hi=1000, Hq=32, Hkv=8, D=128, page=16,
             dtype="bf16", tree=False, ragged=False, lse=False),
        # plain decoding of a full batch, one token a request
        dict(name="attn_b128_t1_c2048", op="attn", B=128, T=1, lo=64, hi=4096, Hq=32, Hkv=8, D=128, page=16,
             dtype="bf16", tree=False, ragged=False, lse=False),
        # a batch of candidate trees of 32 nodes
        dict(name="attn_b32_t33_c4096_tree", op="attn", B=32, T=33, lo=512, hi=8192, Hq=32, Hkv=8, D=128, page=64,
             dtype="bf16", tree=True, ragged=False, lse=False),
        # two long documents, 7 drafted positions, wide groups: the most keys
        dict(name="attn_b2_t8_c131072", op="attn", B=2, T=8, lo=131072, hi=131072, Hq=64, Hkv=8, D=128, page=64,
             dtype="bf16", tree=False, ragged=False, lse=True),
        # verify lengths of their own, an odd head size and page, requests that have nothing cached yet
        dict(name="attn_b13_c3001_d80_ragged", op="attn", B=13, T=7, lo=0, hi=3001, Hq=10, Hkv=2, D=80, page=24,
             dtype="fp16", tree=True, ragged=True, lse=True),
        # a few requests' pages
        dict(name="plan_b8_page16", op="plan", B=8, page=16, table=512, T=8, used=0.4, tight=False),
        # a large batch with wide tables, some requests done, some taken back
        dict(name="plan_b1024_page16", op="plan", B=1024, page=16, table=2048, T=16, used=0.5, tight=True),
        # the accepted rows of a few chains, one layer
        dict(name="commit_b4_t5", op="commit", layers=1, B=4, T=5, Hkv=8, D=128, page=16, spare=8, dtype="bf16",
             tree=False, ragged=False),
        # accepted paths of a batch of trees, all layers at once
        dict(name="commit_l32_b64_t33_tree", op="commit", layers=32, B=64, T=33, Hkv=8, D=128, page=64, spare=1,
             dtype="bf16", tree=True, ragged=False),
        # one request's chain over a small vocabulary, fp32 logits
        dict(name="adjust_b1_t5_v32000", op="adjust", B=1, T=5, V=32000, dtype="fp32", hist=700, bias=0, grammar=False,
             tree=False, ragged=False),
        # trees of 16 nodes over an odd vocabulary, a grammar for every row, long histories
        dict(name="adjust_b16_t17_v50257_tree", op="adjust", B=16, T=17, V=50257, dtype="fp32", hist=16000, bias=64,
             grammar=True, tree=True, ragged=False),
        # the benchmark's batch: 128 chains of 7 drafted tokens, every rule on
        dict(name="adjust_b128_t8_v129280", op="adjust", B=128, T=8, V=129280, dtype="bf16", hist=4000, bias=300,
             grammar=True, tree=False, ragged=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "plan", "commit", "adjust", "adjust"])
    ragged = rng.random() < 0.3
    if op == "attn":
        Hkv = rng.choice([1, 2, 4, 8, 8, 16])
        Hq = Hkv * rng.choice([1, 2, 4, 5, 8])
        D = rng.choice([64, 128, 128, 128, 8 * rng.randint(4, 32)])
        T = rng.choice([1, _log_int(rng, 1, 130), _log_int(rng, 2, 17)])
        B = _log_int(rng, 1, 256)
        page = rng.choice([16, 32, 64, 128, 8 * rng.randint(1, 20)])
        most = max(1, min(131072, MAX_KEY_HEADS * 128 // (B * Hkv * max(D, 128)),
                          int(MAX_ATTN_FLOPS / (4 * B * Hq * D * T))))
        hi = _log_int(rng, 1, most)
        return dict(op=op, B=B, T=T, lo=rng.choice([hi, 0, hi // 2]), hi=hi, Hq=Hq, Hkv=Hkv, D=D, page=page,
                    dtype=rng.choice(["bf16", "bf16", "fp16"]), tree=rng.random() < 0.6, ragged=ragged,
                    lse=rng.random() < 0.3)
    if op == "plan":
        B = _log_int(rng, 1, 1024)
        return dict(op=op, B=B, page=rng.choice([8, 16, 64, 24, _log_int(rng, 1, 256)]),
                    table=_log_int(rng, 4, 2048), T=_log_int(rng, 1, 64), used=rng.uniform(0.1, 0.9),
                    tight=rng.random() < 0.5)
    if op == "commit":
        layers, B, T = _log_int(rng, 1, 32), _log_int(rng, 1, 64), _log_int(rng, 1, 33)
        return dict(op=op, layers=layers, B=B, T=T, Hkv=rng.choice([1, 2, 8]), D=rng.choice([64, 80, 128]),
                    page=rng.choice([16, 64, 24]), spare=rng.choice([1, 4]), dtype=rng.choice(["bf16", "fp16"]),
                    tree=rng.random() < 0.5, ragged=ragged)
    V = rng.choice([151936, 129280, 32000, 50257, _log_int(rng, 1000, 160000)])
    T = _log_int(rng, 1, 33)
    B = _log_int(rng, 1, max(1, min(256, MAX_LOGITS // (V * T))))
    return dict(op=op, B=B, T=T, V=V, dtype=rng.choice(["bf16", "bf16", "fp32"]), hist=_log_int(rng, 1, 32000),
                bias=rng.choice([0, _log_int(rng, 1, 300)]), grammar=rng.random() < 0.5, tree=rng.random() < 0.4,
                ragged=ragged)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _spread(lo, hi, n):
    """n lengths from lo to hi, evenly spread: which request has which goes by the seed."""
    return [hi] if n == 1 else [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _rows(case):
    """Rows of each request (before the seed orders them)."""
    return _spread(1, case["T"], case["B"]) if case["ragged"] else [case["T"]] * case["B"]


def _shuffled(values, g, dev):
    order = torch.randperm(len(values), generator=g, device=dev)
    return torch.tensor(values, dtype=torch.int32, device=dev)[order]


def _offsets(rows):
    return torch.cat([torch.zeros_like(rows[:1]), rows.cumsum(0)]).to(torch.int32)


def _chain(B, T, dev):
    return torch.tril(torch.ones(T, T, dtype=torch.uint8, device=dev)).expand(B, T, T).contiguous()


def _trees(B, T, g, dev):
    """Masks of random trees whose row 0 is the last committed token and every
    other row hangs on an earlier one, on a recent one more often."""
    mask = torch.zeros(B, T, T, dtype=torch.uint8, device=dev)
    mask[:, 0, 0] = 1
    batch = torch.arange(B, device=dev)
    parent = torch.full((B, T), -1, dtype=torch.long, device=dev)
    for i in range(1, T):
        back = (torch.rand(B, generator=g, device=dev) ** 2 * i).long()
        parent[:, i] = i - 1 - back.clamp(max=i - 1)
        mask[:, i] = mask[batch, parent[:, i]]
        mask[:, i, i] = 1
    return mask, parent


def _attn_inputs(case, g, dev):
    B, Hq, Hkv, D, page, dt = (case[k] for k in ("B", "Hq", "Hkv", "D", "page", "dtype"))
    ctx = _shuffled(_spread(case["lo"], case["hi"], B), g, dev)
    rows = _shuffled(_rows(case), g, dev)
    width = max(1, -(-case["hi"] // page))
    pages = sum(-(-n // page) for n in _spread(case["lo"], case["hi"], B)) + 3
    # a cache in use: every request's pages scattered over it
    ids = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    held = (ctx + page - 1) // page
    first = held.cumsum(0) - held
    col = torch.arange(width, device=dev)
    at = (first[:, None] + col).clamp(max=pages - 1)
    table = torch.where(col < held[:, None], ids[at], 0).to(torch.int32)
    kv = lambda *shape: torch.randn(*shape, generator=g, device=dev, dtype=DT[dt])  # noqa: E731
    R = sum(_rows(case))
    s = dict(block_table=table.contiguous(), context_lens=ctx, k_cache=kv(pages, page, Hkv, D),
             v_cache=kv(pages, page, Hkv, D), q=kv(R, Hq, D) * 1.5, k_new=kv(R, Hkv, D), v_new=kv(R, Hkv, D))
    s["mask"] = _trees(B, case["T"], g, dev)[0] if case["tree"] else None
    s["row_offsets"] = _offsets(rows) if case["ragged"] else None
    if not case["ragged"]:
        for k in ("q", "k_new", "v_new"):
            s[k] = s[k].view(B, case["T"], *s[k].shape[1:])
    return s


def _plan_inputs(case, g, dev):
    """A batch between two steps: most requests commit a few tokens, some are done and
    give their pages back, some take a few tokens back, some stay."""
    B, page, M, T = case["B"], case["page"], case["table"], case["T"]
    most = max(1, int(case["used"] * M * page))
    ctx = torch.randint(0, most + 1, (B,), generator=g, device=dev, dtype=torch.int32)
    new = torch.randint(0, T + 1, (B,), generator=g, device=dev, dtype=torch.int32)
    kind = torch.rand(B, generator=g, device=dev)
    new = torch.where(kind < 0.05, -ctx, torch.where(kind < 0.1, -torch.minimum(ctx, new), new))
    held = (ctx + page - 1) // page
    total = B * M
    ids = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    first = held.cumsum(0) - held
    col = torch.arange(M, device=dev)
    table = torch.where(col < held[:, None], ids[(first[:, None] + col).clamp(max=total - 1)], -1).to(torch.int32)
    used = held.sum()
    free = torch.where(torch.arange(total, device=dev) < total - used,
                       ids[(used + torch.arange(total, device=dev)).clamp(max=total - 1)], -1).to(torch.int32)
    # a cache that is nearly full: pages for the first requests only
    count = (total - used).clamp(max=B // 8 if case["tight"] else total).to(torch.int32).reshape(1)
    return dict(context_lens=ctx, new_lens=new.to(torch.int32).contiguous(), block_table=table.contiguous(),
                free_pages=free.contiguous(), free_count=count)


def _commit_inputs(case, g, dev):
    L, B, T, Hkv, D, page, dt = (case[k] for k in ("layers", "B", "T", "Hkv", "D", "page", "dtype"))
    rows = _shuffled(_rows(case), g, dev)
    R = sum(_rows(case))
    kept = _shuffled([1 + i % n for i, n in enumerate(_rows(case))], g, dev)
    kept = torch.minimum(kept, rows)
    S = case["T"]
    tokens = -(-B * S * (1 + case["spare"]) // page) * page
    i = torch.arange(S, device=dev)
    start = torch.randperm(tokens // S, generator=g, device=dev)[:B] * S  # every request's slots are its own
    slots = torch.where(i < kept[:, None], start[:, None] + i, -1).to(torch.int32)
    path = None
    if case["tree"]:  # accepted nodes, in rising order
        pick = torch.rand(B, S, generator=g, device=dev)
        pick = torch.where(i[None] < rows[:, None] - 1, pick, 2.0)
        node = pick.argsort(dim=1)
        node = torch.where(i[None] < kept[:, None] - 1, node, S).sort(dim=1).values
        path = torch.where(i[None] < kept[:, None] - 1, node, -1)[:, :max(S - 1, 0)].to(torch.int32).contiguous()
    kv = lambda *shape: torch.randn(*shape, generator=g, device=dev, dtype=DT[dt])  # noqa: E731
    s = dict(k_new=kv(L, R, Hkv, D), v_new=kv(L, R, Hkv, D), k_cache=kv(L, tokens // page, page, Hkv, D),
             v_cache=kv(L, tokens // page, page, Hkv, D), slots=slots.contiguous(), path=path,
             row_offsets=_offsets(rows) if case["ragged"] else None)
    if not case["ragged"]:
        s["k_new"], s["v_new"] = (s[k].view(L, B, T, Hkv, D) for k in ("k_new", "v_new"))
    return s


def _adjust_inputs(case, g, dev):
    B, T, V, dt = (case[k] for k in ("B", "T", "V", "dtype"))
    rows = _shuffled(_rows(case), g, dev)
    R, H = sum(_rows(case)), case["hist"]
    zipf = lambda *shape: (V ** torch.rand(*shape, generator=g, device=dev) - 1).int().clamp(0, V - 1)  # noqa: E731
    uniform = lambda lo, hi: lo + (hi - lo) * torch.rand(B, generator=g, device=dev)  # noqa: E731
    lens = _shuffled(_spread(H // 2, H, B), g, dev)
    s = dict(logits=(2.5 * torch.randn(R, V, generator=g, device=dev)).to(DT[dt]), tokens=zipf(R),
             history=zipf(B, H), history_lens=lens, prompt_lens=lens // 3, repetition=uniform(1.0, 1.5),
             frequency=uniform(0.0, 0.5), presence=uniform(-0.2, 0.8), bias_ids=None, bias=None, allowed=None)
    if case["bias"]:
        s["bias_ids"] = torch.where(torch.rand(B, case["bias"], generator=g, device=dev) < 0.9,
                                    zipf(B, case["bias"]), -1).to(torch.int32)
        s["bias"] = 4.0 * torch.randn(B, case["bias"], generator=g, device=dev)
    if case["grammar"]:
        s["allowed"] = torch.randint(-2 ** 31, 2 ** 31, (R, -(-V // 32)), generator=g, device=dev).to(torch.int32)
    s["mask"] = _trees(B, T, g, dev)[0] if case["tree"] else None
    s["row_offsets"] = _offsets(rows) if case["ragged"] else None
    if not case["ragged"]:
        for k in ("logits", "tokens", "allowed"):
            s[k] = None if s[k] is None else s[k].view(B, T, *s[k].shape[1:])
    return s


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    make = {"attn": _attn_inputs, "plan": _plan_inputs, "commit": _commit_inputs, "adjust": _adjust_inputs}
    return dict(make[case["op"]](case, g, dev), case=case)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    if own:
        return _own(s)
    return {"attn": _plain_attn, "plan": _plain_plan, "commit": _plain_commit, "adjust": _plain_adjust}[
        s["case"]["op"]](s)


def _own(s):
    import sampling_spec_verify_gb300 as ssv

    c = s["case"]
    if c["op"] == "plan":
        o = ssv.plan_cache(s["context_lens"], s["new_lens"], s["block_table"], s["free_pages"], s["free_count"],
                           c["page"], c["T"])
        return {"block_table": o.block_table, "free_pages": o.free_pages, "free_count": o.free_count,
                "context_lens": o.context_lens, "slots": o.slots}
    ragged = dict(row_offsets=s["row_offsets"], max_rows=c["T"]) if c["ragged"] else {}
    if c["op"] == "attn":
        o = ssv.tree_attention(s["q"], s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["block_table"],
                               s["context_lens"], mask=s["mask"], want_lse=c["lse"], **ragged)
        return {"out": o.out, "lse": o.lse} if c["lse"] else {"out": o.out}
    if c["op"] == "commit":
        ssv.commit_cache(s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["slots"], path=s["path"],
                         row_offsets=s["row_offsets"])
        return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    return {"logits": ssv.adjust_logits(s["logits"], s["tokens"], s["history"], s["history_lens"],
                                        prompt_lens=s["prompt_lens"], repetition=s["repetition"],
                                        frequency=s["frequency"], presence=s["presence"], bias_ids=s["bias_ids"],
                                        bias=s["bias"], allowed=s["allowed"], mask=s["mask"], **ragged)}


def _places(s, n_rows):
    """(request, row of the request) of every flattened row, and the flattened row of
    every (request, row), clamped where the request has none."""
    c = s["case"]
    dev = s["row_offsets"].device
    off = s["row_offsets"].long()
    r = torch.arange(n_rows, device=dev)
    b = torch.searchsorted(off[1:].contiguous(), r, right=True)
    at = (off[:-1, None] + torch.arange(c["T"], device=dev)).clamp(max=n_rows - 1)
    return b, r - off[b], at


def _plain_attn(s):
    c = s["case"]
    B, T, Hq, Hkv, D = (c[k] for k in ("B", "T", "Hq", "Hkv", "D"))
    G = Hq // Hkv
    q, kn, vn = s["q"], s["k_new"], s["v_new"]
    if c["ragged"]:
        b, i, at = _places(s, q.shape[0])
        q, kn, vn = q[at], kn[at], vn[at]
    table = s["block_table"].long()
    L = table.shape[1] * c["page"]
    dev = q.device

    def keys(cache, fresh):  # [B, Hkv, L + T, D]
        old = cache[table].reshape(B, L, Hkv, D)
        return torch.cat([old, fresh], 1).permute(0, 2, 1, 3).float()

    x = q.float().view(B, T, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, D)
    z = (x @ keys(s["k_cache"], kn).transpose(2, 3)) * (1.0 / math.sqrt(D))
    mask = torch.tril(torch.ones(T, T, dtype=torch.bool, device=dev)).expand(B, T, T)
    mask = mask if s["mask"] is None else s["mask"] != 0
    if c["ragged"]:
        mask = mask & (torch.arange(T, device=dev) < s["row_offsets"].diff()[:, None])[:, None]
    cached = (torch.arange(L, device=dev) < s["context_lens"][:, None])[:, None].expand(B, T, L)
    sees = torch.cat([cached, mask], 2).repeat_interleave(G, dim=1)[:, None]
    z = torch.where(sees, z, float("-inf"))
    m = z.amax(dim=3, keepdim=True)
    m = torch.where(m == float("-inf"), 0.0, m)
    p = torch.exp(z - m)
    total = p.sum(dim=3, keepdim=True)
    o = (p @ keys(s["v_cache"], vn)) / torch.where(total > 0, total, 1.0)
    o = o.view(B, Hkv, T, G, D).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, D).to(q.dtype)
    lse = (m + torch.log(total)).view(B, Hkv, T, G).permute(0, 2, 1, 3).reshape(B, T, Hq)
    if c["ragged"]:
        o, lse = o[b, i], lse[b, i]
    return {"out": o, "lse": lse} if c["lse"] else {"out": o}


def _plain_plan(s):
    c = s["case"]
    page, T = c["page"], c["T"]
    ctx, new, table, free = (s[k].long() for k in ("context_lens", "new_lens", "block_table", "free_pages"))
    count = s["free_count"].long()
    B, M = table.shape
    col = torch.arange(M, device=table.device)
    after = ctx + new
    fits = (ctx >= 0) & (ctx <= M * page) & (after >= 0) & (after <= M * page) & (new <= T)
    held, want = (ctx + page - 1) // page, (after + page - 1) // page
    back = torch.where(fits, (held - want).clamp(min=0), 0)
    need = torch.where(fits, (want - held).clamp(min=0), 0)
    upto = need.cumsum(0)
    have = count + back.sum()
    served = fits & ((need == 0) | (upto <= have))
    # pages given back go on top of the stack, in the order of the requests and of their pages
    gives = fits[:, None] & (col >= want[:, None]) & (col < held[:, None])
    place = torch.where(gives, (back.cumsum(0) - back)[:, None] + col - want[:, None] + count, free.numel())
    stack = torch.cat([free, free[:1]]).scatter(0, place.reshape(-1), table.reshape(-1))[:-1]
    # pages that are needed come from its top
    takes = served[:, None] & (col >= held[:, None]) & (col < want[:, None])
    top = have - 1 - ((upto - need)[:, None] + col - held[:, None])
    table = torch.where(takes, stack[torch.where(takes, top, 0)], table)
    i = torch.arange(T, device=table.device)
    pos = ctx[:, None] + i
    filled = served[:, None] & (i < new[:, None])
    slots = torch.gather(table, 1, torch.where(filled, pos // page, 0)) * page + pos % page
    out = {"block_table": table, "free_pages": stack, "free_count": have - torch.where(served, need, 0).sum(),
           "context_lens": torch.where(served, after, ctx), "slots": torch.where(filled, slots, -1)}
    return {k: v.to(torch.int32) for k, v in out.items()}


def _plain_commit(s):
    c = s["case"]
    L, Hkv, D, B = c["layers"], c["Hkv"], c["D"], c["B"]
    slots = s["slots"].long()
    i = torch.arange(slots.shape[1], device=slots.device).expand_as(slots)
    row = i if s["path"] is None else torch.cat([torch.zeros_like(i[:, :1]), s["path"].long() + 1], 1)
    first = s["row_offsets"][:-1].long() if c["ragged"] else torch.arange(B, device=slots.device) * c["T"]
    # every request commits its first row; an empty place repeats it
    used = slots >= 0
    dst = torch.where(used, slots, slots[:, :1]).reshape(-1)
    src = (first[:, None] + torch.where(used, row, 0)).reshape(-1)
    for_all = lambda cache, x: cache.view(L, -1, Hkv, D).index_copy_(1, dst, x.reshape(L, -1, Hkv, D)[:, src])  # noqa: E731
    for_all(s["k_cache"], s["k_new"])
    for_all(s["v_cache"], s["v_new"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_adjust(s):
    c = s["case"]
    B, T, V = c["B"], c["T"], c["V"]
    z, tokens, allowed = s["logits"], s["tokens"], s["allowed"]
    dev = z.device
    if c["ragged"]:
        b, i, at = _places(s, z.shape[0])
        tokens = tokens[at]
    sees = torch.tril(torch.ones(T, T, dtype=torch.bool, device=dev)).expand(B, T, T)
    sees = sees if s["mask"] is None else s["mask"] != 0
    # occurrences in the generated history, then in the drafted rows that a row sees
    col = torch.arange(s["history"].shape[1], device=dev)
    past = col < s["history_lens"][:, None]
    prompt = past & (col < s["prompt_lens"][:, None])
    zero = torch.zeros(B, V, dtype=torch.int32, device=dev)
    idx = s["history"].long()
    known = zero.scatter_add(1, idx, prompt.int())
    made = zero.scatter_add(1, idx, (past & ~prompt).int())
    n = made[:, None].repeat(1, T, 1).scatter_add_(2, tokens.long()[:, None].expand(B, T, T), sees.int())
    bias = torch.zeros(B, V + 1, device=dev)
    if c["bias"]:
        bias.scatter_add_(1, torch.where(s["bias_ids"] >= 0, s["bias_ids"].long(), V), s["bias"])
    seen = (n > 0) | (known > 0)[:, None]
    rep, freq, pres = (s[k][:, None, None] for k in ("repetition", "frequency", "presence"))
    bias = bias[:, None, :V]
    if c["ragged"]:
        n, seen, bias, rep, freq, pres = n[b, i], seen[b, i], bias[b, 0], rep[b, 0], freq[b, 0], pres[b, 0]
    x = z.float()
    x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
    x = x - freq * n - pres * (n > 0)
    x = x + bias
    if allowed is not None:
        bit = (allowed[..., None] >> torch.arange(32, device=dev)) & 1
        x = torch.where(bit.flatten(-2)[..., :V] != 0, x, float("-inf"))
    return {"logits": x.to(z.dtype)}


# ---------------------------------------------------------------------------
# cost and exact answer
# ---------------------------------------------------------------------------

def _pages_of(n, page):
    return -(-n // page)


def work(case):
    op = case["op"]
    if op == "attn":
        es, D = DT[case["dtype"]].itemsize, case["D"]
        ctx, rows = sum(_spread(case["lo"], case["hi"], case["B"])), sum(_rows(case))
        b = 2 * (ctx + rows) * case["Hkv"] * D * es + 2 * rows * case["Hq"] * D * es
        mean_ctx = ctx / case["B"]
        return {"bytes": b, "flops": 4 * case["Hq"] * D * rows * (mean_ctx + (case["T"] + 1) / 2)}
    if op == "plan":
        B, M = case["B"], case["table"]
        words = 2 * B * M + 2 * B * M + 3 * B + 2 + B * case["T"]  # table and stack in and out
        return {"bytes": 4 * words, "flops": 8 * B}
    if op == "commit":
        es = DT[case["dtype"]].itemsize
        kept = sum(1 + i % n for i, n in enumerate(_rows(case)))
        return {"bytes": 4 * case["layers"] * kept * case["Hkv"] * case["D"] * es + 8 * case["B"] * case["T"],
                "flops": 0}
    es, V, R = DT[case["dtype"]].itemsize, case["V"], sum(_rows(case))
    b = 2 * R * V * es + 4 * sum(_spread(case["hist"] // 2, case["hist"], case["B"])) + 8 * case["B"] * case["bias"]
    if case["grammar"]:
        b += R * 4 * -(-V // 32)
    return {"bytes": b, "flops": 6 * R * V}


def exact(case, seed):
    """The definitions in 64 bits, request by request."""
    if case["op"] == "commit":
        return None  # nothing is computed
    if case["op"] == "attn" and work(case)["flops"] > EXACT_FLOPS:
        return None
    s = prepare(case, seed)
    return {"attn": _exact_attn, "plan": _exact_plan, "adjust": _exact_adjust}[case["op"]](case, s)


def _starts(case, s):
    if s["row_offsets"] is not None:
        return s["row_offsets"].tolist()
    return [case["T"] * b for b in range(case["B"] + 1)]


def _exact_attn(case, s):
    Hq, Hkv, D, page = (case[k] for k in ("Hq", "Hkv", "D", "page"))
    at = _starts(case, s)
    q, kn, vn = (s[k].reshape(-1, *s[k].shape[-2:]).double() for k in ("q", "k_new", "v_new"))
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], dtype=torch.float64, device=q.device)
    for b, n in enumerate(s["context_lens"].tolist()):
        r0, r1 = at[b], at[b + 1]
        ids = s["block_table"][b, :_pages_of(n, page)].long()
        for h in range(Hkv):
            k = torch.cat([s["k_cache"][ids, :, h].flatten(0, 1)[:n].double(), kn[r0:r1, h]])
            v = torch.cat([s["v_cache"][ids, :, h].flatten(0, 1)[:n].double(), vn[r0:r1, h]])
            hidden = torch.zeros(r1 - r0, n + r1 - r0, dtype=torch.bool, device=q.device)
            if s["mask"] is None:
                hidden[:, n:] = torch.ones(r1 - r0, r1 - r0, device=q.device).triu(1) != 0
            else:
                hidden[:, n:] = s["mask"][b, :r1 - r0, :r1 - r0] == 0
            for head in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
                z = torch.einsum("rd,nd->rn", q[r0:r1, head], k).div(D ** 0.5).masked_fill(hidden, float("-inf"))
                lse[r0:r1, head] = torch.logsumexp(z, dim=1)
                out[r0:r1, head] = torch.einsum("rn,nd->rd", torch.softmax(z, dim=1), v)
    o = {"out": out.view(s["q"].shape)}
    if case["lse"]:
        o["lse"] = lse.view(s["q"].shape[:-1])
    return o


def _exact_plan(case, s):
    """The page allocator, one request after the other on the host."""
    page, T = case["page"], case["T"]
    table, ctx, new = s["block_table"].tolist(), s["context_lens"].tolist(), s["new_lens"].tolist()
    stack, count = s["free_pages"].tolist(), int(s["free_count"])
    room = case["table"] * page
    ok = [0 <= c <= room and 0 <= c + n <= room and n <= T for c, n in zip(ctx, new)]
    for b in range(case["B"]):
        if ok[b]:
            for p in table[b][_pages_of(ctx[b] + new[b], page):_pages_of(ctx[b], page)]:
                stack[count] = p
                count += 1
    slots = [[-1] * T for _ in ctx]
    blocked = False  # once a request finds too few pages, those behind it get none
    for b in range(case["B"]):
        if not ok[b]:
            continue
        first, last = _pages_of(ctx[b], page), _pages_of(ctx[b] + new[b], page)
        if last > first and (blocked or last - first > count):
            blocked = True
            continue
        for j in range(first, last):
            count -= 1
            table[b][j] = stack[count]
        for i in range(max(new[b], 0)):
            p = ctx[b] + i
            slots[b][i] = table[b][p // page] * page + p % page
        ctx[b] += new[b]
    dev = s["block_table"].device
    put = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    return {"block_table": put(table), "free_pages": put(stack), "free_count": put([count]),
            "context_lens": put(ctx), "slots": put(slots)}


def _exact_adjust(case, s):
    V = case["V"]
    at = _starts(case, s)
    z = s["logits"].reshape(-1, V).double()
    tokens = s["tokens"].reshape(-1).long()
    lens, prompts = s["history_lens"].tolist(), s["prompt_lens"].tolist()
    for b in range(case["B"]):
        past = s["history"][b, :lens[b]].long()
        known = torch.bincount(past[:prompts[b]], minlength=V) > 0
        made = torch.bincount(past[prompts[b]:], minlength=V)
        rep, freq, pres = (s[k][b].double() for k in ("repetition", "frequency", "presence"))
        for r in range(at[b], at[b + 1]):
            rows = slice(at[b], at[b + 1])
            sees = s["mask"][b, r - at[b], :at[b + 1] - at[b]] != 0 if s["mask"] is not None else \
                torch.arange(at[b], at[b + 1], device=z.device) <= r
            n = (made + torch.bincount(tokens[rows][sees], minlength=V)).double()
            x = z[r]
            touched = known | (n > 0)
            x = x * torch.where(touched, torch.where(x > 0, 1.0 / rep, rep), 1.0)
            x = x - (freq * n + pres * (n > 0).double())
            if case["bias"]:
                real = s["bias_ids"][b] >= 0
                x = x.index_add(0, s["bias_ids"][b][real].long(), s["bias"][b][real].double())
            if case["grammar"]:
                word = s["allowed"].reshape(-1, s["allowed"].shape[-1])[r].long()
                v = torch.arange(V, device=z.device)
                x = x.masked_fill(((word[v // 32] >> (v % 32)) & 1) == 0, float("-inf"))
            z[r] = x
    return {"logits": z.view(s["logits"].shape)}
