"""Inputs of the decoding step's tests, built on the CPU from a seed."""

import numpy as np
import torch


def random_parents(rng, T):
    return np.array([-1] + [int(rng.integers(-1 if T < 3 else 0, i)) for i in range(1, T)], dtype=np.int32)


def tree_masks(rng, B, T):
    mask = np.zeros((B, T, T), dtype=np.uint8)
    for b in range(B):
        par = random_parents(rng, T)
        for i in range(T):
            if par[i] >= 0:
                mask[b, i] = mask[b, par[i]]
            mask[b, i, i] = 1
    return mask


def attention_case(seed, rows, ctx, Hq, Hkv, D, page, dtype, tree=False, ragged=False, T=None, spare_rows=0,
                   layout="nhd", strided=False, poison=True, spread=1.0):
    """rows, ctx: per request.  Places of the cache that no request's context covers, and rows
    behind the last request, hold NaN (``poison``)."""
    rng = np.random.default_rng(seed)
    B = len(rows)
    T = T or max(rows)
    R = sum(rows) + spare_rows
    need = [-(-n // page) for n in ctx]
    pages, width = sum(need) + 2, max(max(need), 1) + 1
    ids = rng.permutation(pages)
    table = np.full((B, width), pages + 5, dtype=np.int32)  # behind a request's pages: anything
    n = 0
    for b in range(B):
        table[b, :need[b]] = ids[n:n + need[b]]
        n += need[b]
    f = lambda *s: torch.from_numpy(rng.normal(size=s).astype(np.float32)).to(dtype)  # noqa: E731
    shape = (pages, page, Hkv, D)
    kc, vc = f(*shape), f(*shape)
    if poison:
        live = torch.zeros(pages, page, dtype=torch.bool)
        for b in range(B):
            for p in range(need[b]):
                live[table[b, p], :min(page, ctx[b] - p * page)] = True
        kc[~live] = float("nan")
        vc[~live] = float("nan")
    if layout == "hnd":
        kc, vc = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (kc, vc))
    elif layout == "mixed":  # keys token by token, values head by head
        vc = vc.transpose(1, 2).contiguous().transpose(1, 2)
    elif layout == "apart":  # heads that no even dimension continues
        kc, vc = (torch.cat([t, t[:, :, :, :8]], 3)[..., :D] for t in (kc, vc))
    elif layout == "joint":  # one tensor, keys and values side by side
        joint = torch.stack([kc, vc], 1).contiguous()
        kc, vc = joint[:, 0], joint[:, 1]
    if strided:  # q, k and v as slices of one projection
        qkv = f(R, (Hq + 2 * Hkv) * D + 16)
        q = qkv[:, :Hq * D].view(R, Hq, D)
        kn = qkv[:, Hq * D:(Hq + Hkv) * D].view(R, Hkv, D)
        vn = qkv[:, (Hq + Hkv) * D:(Hq + 2 * Hkv) * D].view(R, Hkv, D)
    else:
        q, kn, vn = f(R, Hq, D) * spread, f(R, Hkv, D), f(R, Hkv, D)
    if poison and spare_rows:
        for t in (q, kn, vn):
            t[R - spare_rows:] = float("nan")
    offsets = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    c = dict(q=q, k_new=kn, v_new=vn, k_cache=kc, v_cache=vc, table=table, ctx=np.array(ctx, dtype=np.int32),
             offsets=offsets, mask=tree_masks(rng, B, T) if tree else None, T=T, ragged=ragged, scale=D ** -0.5)
    assert ragged or (len(set(rows)) == 1 and spare_rows == 0)
    return c


def on_gpu(c):
    """(args, kwargs) of ssv.tree_attention."""
    d = lambda t: moved(t)  # noqa: E731
    B = len(c["ctx"])
    fit = (lambda t: t) if c["ragged"] else (lambda t: t.unflatten(0, (B, c["T"])))
    joint = {}
    args = [fit(d(c[k])) for k in ("q", "k_new", "v_new")] + [d(c["k_cache"]), d(c["v_cache"]),
                                                             torch.from_numpy(c["table"]).cuda(),
                                                             torch.from_numpy(c["ctx"]).cuda()]
    kw = dict(mask=None if c["mask"] is None else torch.from_numpy(c["mask"]).cuda(), **joint)
    if c["ragged"]:
        kw.update(row_offsets=torch.from_numpy(c["offsets"]).cuda(), max_rows=c["T"])
    return args, kw


def moved(t):
    """To the GPU with the same strides."""
    span = sum((n - 1) * s for n, s in zip(t.shape, t.stride())) + 1 if t.numel() else 0
    flat = torch.as_strided(t, (span,), (1,), t.storage_offset()).cuda() if span else t.cuda()
    return torch.as_strided(flat, t.shape, t.stride()) if span else flat


def f64(t):
    return t.double().numpy()


def attention_oracle(c):
    from oracle import decode

    return decode.tree_attention(f64(c["q"]), f64(c["k_new"]), f64(c["v_new"]), f64(c["k_cache"]), f64(c["v_cache"]),
                                 c["table"], c["ctx"], c["offsets"], c["mask"], c["scale"])


def attention_bounds(c, r, dtype):
    """(out, lse) tolerances.  u, half a step of dtype: one rounding of each weight (u mass) and one of
    the result (u |out|).  A score is a sum of D products in fp32, at worst (D + 8) 2^-23 of the sum of
    their magnitudes off, which shifts a weight and the normaliser each by that factor; sums over n
    keys lose at most n 2^-24, the exponential 2^-21 and its argument 2^-23 of itself.  Weights of
    fp16 below its normal range are off by up to 2^-25 of the largest one."""
    u = torch.finfo(dtype).eps / 2
    n = max(int(c["ctx"].max(initial=0)) + c["T"], 1)
    D = c["q"].shape[-1]
    s = (D + 8) * 2.0 ** -23 * r.spread + n * 2.0 ** -24 + 2.0 ** -21 + 2.0 ** -22 * r.spread
    big = max(float(np.nanmax(np.abs(f64(c[k])), initial=0.0, where=np.isfinite(f64(c[k])))) for k in ("v_cache", "v_new"))
    low = n * 2.0 ** -25 * big if dtype == torch.float16 else 0.0
    out = u * (r.mass + np.abs(r.out)) * 1.01 + 2 * s[..., None] * r.mass + low + 1e-30
    if dtype == torch.float16:
        out = out + 2.0 ** -25  # results below fp16's normal range
    return out, s + 2.0 ** -23 * np.abs(np.where(np.isfinite(r.lse), r.lse, 0.0))
