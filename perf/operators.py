"""The drafter-training losses over a vocabulary, as measured workloads.

Three operators, each forward alone and forward with gradients:

* ``lce``  -- cross entropy of a vocabulary head, softmax(hidden @ weight.T / T)
  against labels, with the gradients of the hidden states and of the head;
* ``kd``   -- distillation of given student logits from a teacher's top logits,
  with or without the teacher's remaining mass as one bucket;
* ``lkd``  -- that distillation from the hidden states and the head.

``run`` makes the library's calls where ``own`` is true and computes the same
in elementary torch operations otherwise; ``exact`` gives the 64-bit answer.
"""

import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}

# exact() runs three fp64 products over the head; beyond this many operations
# it would take too long
EXACT_FLOPS = 6e12

# the largest drawn cases stay within the largest listed ones
MAX_HEAD_FLOPS = 6 * 4096 * 129280 * 4096
MAX_KD_ELEMS = 1792 * 151936


def listed():
    return [
        # one request's block of drafted positions against a small head: latency
        dict(name="lce_n8_v32000_h1024", op="lce", N=8, V=32000, H=1024, dtype="bf16", grad="both", T=1.0,
             ignored=0.0, weighted=False, reduction="mean"),
        # a drafter's training batch of 256 rows with 7 positions
        dict(name="lce_n1792_v151936_h2048", op="lce", N=1792, V=151936, H=2048, dtype="bf16", grad="both", T=1.0,
             ignored=0.1, weighted=True, reduction="mean"),
        # a long packed batch on a wide model: the largest
        dict(name="lce_n4096_v129280_h4096", op="lce", N=4096, V=129280, H=4096, dtype="bf16", grad="both", T=1.0,
             ignored=0.1, weighted=False, reduction="mean"),
        # odd sizes, fp16, the head frozen (shared with the target model), most rows prompt tokens
        dict(name="lce_n1001_v50257_h1544_frozen", op="lce", N=1001, V=50257, H=1544, dtype="fp16", grad="hidden",
             T=0.8, ignored=0.5, weighted=True, reduction="sum"),
        # scoring: log-probabilities of given tokens, no gradient
        dict(name="lce_n2047_v151936_h2048_score", op="lce", N=2047, V=151936, H=2048, dtype="bf16", grad="none",
             T=1.0, ignored=0.0, weighted=False, reduction="sum"),
        # the smallest distillation call: one row block, fp32 logits
        dict(name="kd_n4_v1024_k8", op="kd", N=4, V=1024, k=8, dtype="fp32", grad="fp32", tail=False, T=1.0,
             padded=False, masked=False, weighted=False, reduction="mean"),
        # a training batch of 128 rows with 7 positions, teacher remainder kept
        dict(name="kd_n896_v129280_k64_tail", op="kd", N=896, V=129280, k=64, dtype="bf16", grad="bf16", tail=True,
             T=1.0, padded=False, masked=False, weighted=True, reduction="mean"),
        # the E2E-TV training batch (256 rows, 7 positions), its fp32 gradient
        dict(name="kd_n1792_v151936_k128", op="kd", N=1792, V=151936, k=128, dtype="bf16", grad="fp32", tail=False,
             T=1.0, padded=False, masked=False, weighted=False, reduction="mean"),
        # odd vocabulary, fp16, rows of ragged (also empty) teacher lists, truncated student
        dict(name="kd_n777_v50257_k50_ragged", op="kd", N=777, V=50257, k=50, dtype="fp16", grad="fp16", tail=True,
             T=2.0, padded=True, masked=True, weighted=True, reduction="sum"),
        # evaluation: the divergence of every position, no gradient
        dict(name="kd_n1024_v151936_k20_eval", op="kd", N=1024, V=151936, k=20, dtype="bf16", grad="none", tail=True,
             T=1.0, padded=False, masked=False, weighted=False, reduction="mean"),
        # a few requests' drafted positions distilled through a small head
        dict(name="lkd_n56_v32000_h1024_k16", op="lkd", N=56, V=32000, H=1024, k=16, dtype="bf16", grad="both",
             T=1.0, padded=False, weighted=False, reduction="mean"),
        # the training batch of 256 rows with 7 positions, distilled through the head, the head frozen
        dict(name="lkd_n1792_v151936_h2048_k64_frozen", op="lkd", N=1792, V=151936, H=2048, k=64, dtype="bf16",
             grad="hidden", T=1.0, padded=True, weighted=True, reduction="mean"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lce", "lce", "kd", "kd", "lkd"])
    V = rng.choice([151936, 129280, 32000, 50257, _log_int(rng, 1000, 160000)])
    common = dict(T=rng.choice([1.0, 1.0, 0.7, 1.7]), weighted=rng.random() < 0.5,
                  reduction=rng.choice(["mean", "sum"]))
    if op == "kd":
        V = rng.choice([V, _log_int(rng, 500, 200000)])
        N = _log_int(rng, 1, max(1, min(4096, MAX_KD_ELEMS // V)))
        dt = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        k = min(V, _log_int(rng, 1, 256))
        tail = rng.random() < 0.5
        return dict(op=op, N=N, V=V, k=k, dtype=dt, grad=rng.choice(["none", dt, dt, "fp32"]), tail=tail,
                    padded=rng.random() < 0.4, masked=rng.random() < 0.3, **common)
    H = 8 * _log_int(rng, 8, 512)
    N = _log_int(rng, 1, max(1, min(8192, MAX_HEAD_FLOPS // (6 * V * H))))
    dt = rng.choice(["bf16", "bf16", "fp16"])
    grad = rng.choice(["none", "hidden", "both", "both"])
    if op == "lce":
        return dict(op=op, N=N, V=V, H=H, dtype=dt, grad=grad, ignored=rng.choice([0.0, 0.1, 0.5]), **common)
    return dict(op=op, N=N, V=V, H=H, k=min(V, _log_int(rng, 1, 256)), dtype=dt, grad=grad,
                padded=rng.random() < 0.4, **common)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

IGNORE = -100


def _grad_scale(case):
    """Half of a two-term objective; 16-bit gradients with a short exponent
    carry a loss scale on top, as fp16 training does, per row of the mean."""
    if "fp16" not in (case["dtype"], case["grad"]) or case["grad"] == "fp32":
        return 0.5
    scale = 0.5 * (2.0 ** 14 if case["op"] == "kd" else 2.0 ** 11)
    return scale * case["N"] if case["reduction"] == "mean" else scale


def _teacher(full, k, T, padded, gen):
    """The k largest entries of each row of the teacher's logits `full`, and
    the logsumexp of the whole row at temperature T."""
    vals, ids = torch.topk(full, k, dim=1)
    lse = torch.logsumexp(full / T, dim=1)
    ids = ids.to(torch.int32)
    if padded:  # nucleus-like lists: every row keeps its own number of entries, some rows none
        keep = torch.randint(0, k + 1, (full.shape[0], 1), generator=gen, device=full.device)
        ids = torch.where(torch.arange(k, device=full.device)[None] < keep, ids, -1)
    return ids.contiguous(), vals.contiguous(), lse.contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    N, V, dt = case["N"], case["V"], DT[case["dtype"]]
    s = dict(case=case, row_weight=None)
    if case["weighted"]:  # position-decayed weights
        s["row_weight"] = 0.8 ** torch.randint(0, 7, (N,), generator=g, device=dev).float()

    if case["op"] == "kd":
        # student logits ~ N(0, 2^2), the teacher a noisy copy (the E2E-TV batch's recipe)
        student = (2.0 * torch.randn(N, V, generator=g, device=dev)).to(dt)
        ids, vals, lse = [], [], []
        for r in range(0, N, 512):
            z = student[r:r + 512].float()
            z += 0.5 * torch.randn(z.shape, generator=g, device=dev)
            a, b, c = _teacher(z, case["k"], case["T"], case["padded"], g)
            ids.append(a), vals.append(b), lse.append(c)
        s["ids"], s["vals"], s["lse"] = torch.cat(ids), torch.cat(vals), torch.cat(lse)
        if not case["tail"]:
            s["lse"] = None
        if case["masked"]:  # truncated student: half of the vocabulary at -inf, the teacher's entries spared
            for r in range(0, N, 512):
                drop = torch.rand(student[r:r + 512].shape, generator=g, device=dev) < 0.5
                i = s["ids"][r:r + 512].long()
                drop = torch.cat([drop, torch.zeros_like(drop[:, :1])], 1)
                drop.scatter_(1, torch.where(i >= 0, i, V), False)
                student[r:r + 512].masked_fill_(drop[:, :V], float("-inf"))
        s["student"] = student
        return s

    H = case["H"]
    # head rows of norm 2: logits of unit-variance hidden states ~ N(0, 2^2)
    s["weight"] = (torch.randn(V, H, generator=g, device=dev) * (2.0 / math.sqrt(H))).to(dt)
    labels = torch.randint(0, V, (N,), generator=g, device=dev)
    # hidden states that point at their label by a per-row amount: confident and unsure rows
    lean = 4.0 * torch.rand(N, 1, generator=g, device=dev)
    hidden = torch.randn(N, H, generator=g, device=dev) + lean * s["weight"][labels].float()
    s["hidden"] = hidden.to(dt)
    if case["op"] == "lce":
        drop = torch.rand(N, generator=g, device=dev) < case["ignored"]
        s["labels"] = torch.where(drop, IGNORE, labels).to(torch.int32)
        return s
    ids, vals = [], []
    for r in range(0, N, 512):
        ht = s["hidden"][r:r + 512].float() + 0.25 * torch.randn(hidden[r:r + 512].shape, generator=g, device=dev)
        z = (ht.to(dt) @ s["weight"].t()).float()
        a, b, _ = _teacher(z, case["k"], case["T"], case["padded"], g)
        ids.append(a), vals.append(b)
    s["ids"], s["vals"] = torch.cat(ids), torch.cat(vals)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import sampling_spec_verify_gb300 as ssv

    c = s["case"]
    kw = dict(row_weight=s["row_weight"], reduction=c["reduction"])
    if c["op"] == "kd":
        if c["grad"] == "none":
            o = ssv.topk_distill(s["student"], s["ids"], s["vals"], c["T"], teacher_lse=s["lse"], **kw)
            return {"loss": o.loss, "row_loss": o.row_loss}
        o = ssv.topk_distill_fwd_bwd(s["student"], s["ids"], s["vals"], c["T"], _grad_scale(c), teacher_lse=s["lse"],
                                     grad_dtype=DT[c["grad"]], **kw)
        return {"loss": o.loss, "row_loss": o.row_loss, "grad": o.grad}
    if c["op"] == "lce":
        fwd, both = ssv.linear_cross_entropy, ssv.linear_cross_entropy_fwd_bwd
        a = (s["hidden"], s["weight"], s["labels"], c["T"])
        kw["ignore_index"] = IGNORE
    else:
        fwd, both = ssv.linear_topk_distill, ssv.linear_topk_distill_fwd_bwd
        a = (s["hidden"], s["weight"], s["ids"], s["vals"], c["T"])
    if c["grad"] == "none":
        o = fwd(*a, **kw)
        return {"loss": o.loss, "row_loss": o.row_loss, "lse": o.lse}
    o = both(*a, _grad_scale(c), want_grad_weight=c["grad"] == "both", **kw)
    out = {"loss": o.loss, "row_loss": o.row_loss, "lse": o.lse, "grad_hidden": o.grad_hidden}
    if c["grad"] == "both":
        out["grad_weight"] = o.grad_weight
    return out


def _lse(z):
    """Logsumexp of every row: 32-bit terms, their long sum and its log in 64."""
    m = z.amax(dim=1, keepdim=True)
    m = torch.where(m == float("-inf"), 0.0, m)
    return m.double() + torch.log(torch.exp(z - m).sum(dim=1, keepdim=True, dtype=torch.float64))


def _row_scale(c, keep, row_weight):
    """w_n / count or w_n, zero for rows that are left out."""
    w = keep.float() if row_weight is None else torch.where(keep, row_weight, 0.0)
    return w / keep.sum().clamp(min=1) if c["reduction"] == "mean" else w


def _targets(ids, vals, lse, T):
    """Teacher probabilities of the listed entries and of the remainder, in 64
    bits: the loss is a small difference of their logarithms."""
    valid = ids >= 0
    x = torch.where(valid, vals.double() / T, float("-inf"))
    if lse is None:
        m = x.amax(dim=1, keepdim=True)
        e = torch.exp(x - torch.where(m == float("-inf"), 0.0, m))
        total = e.sum(dim=1, keepdim=True)
        t = e / torch.where(total > 0, total, 1.0)
        rest = torch.zeros_like(total)
    else:
        t = torch.exp(x - lse.double()[:, None])
        rest = 1.0 - t.sum(dim=1, keepdim=True)
        rest = torch.where(rest > 1e-6, rest, 0.0)  # below: rounding of the sum
    keep = valid.any(dim=1)
    return torch.where(keep[:, None], t, 0.0), torch.where(keep[:, None], rest, 0.0), keep


def _xlog(t, d):
    """t * d with 0 where t is 0."""
    return torch.where(t > 0, t * d, 0.0)


def _plain(s):
    c = s["case"]
    T = c["T"]
    if c["op"] == "kd":
        N, V = s["student"].shape
        z = s["student"].float() / T
        t, rest, keep = _targets(s["ids"], s["vals"], s["lse"], T)
        idx = s["ids"].long()
        slot = torch.where(idx >= 0, idx, V)
        zi = torch.gather(s["student"], 1, idx.clamp(min=0)).double() / T
        lse = _lse(z)
        qi = torch.exp(zi - lse) * (idx >= 0)
        row = _xlog(t, torch.log(t) - (zi - lse)).sum(dim=1)
        if c["tail"]:
            others = torch.cat([z, torch.full_like(z[:, :1], float("-inf"))], 1).scatter_(1, slot, float("-inf"))
            lse_rest = _lse(others)
            # where the entries hold little mass, the rest's is 1 minus theirs: the plain
            # difference of two normalisers would lose it
            sq = qi.sum(dim=1, keepdim=True)
            log_qr = torch.where(sq < 0.5, torch.log1p(-sq.clamp(max=0.5)), lse_rest - lse)
            row = row + _xlog(rest, torch.log(rest) - log_qr)[:, 0]
        scale = _row_scale(c, keep, s["row_weight"])
        out = {"loss": (scale * row).sum().float().reshape(1), "row_loss": row.float()}
        if c["grad"] != "none":
            st = t.sum(dim=1, keepdim=True)
            mass = st + rest
            coef = (scale * (_grad_scale(c) / T))[:, None]
            if c["tail"]:
                # mass q_r - t_r, without the cancellation of two masses near 1
                diff = torch.where(sq < 0.5, st - mass * sq, mass * torch.exp(log_qr) - rest)
                finite = torch.where(lse_rest == float("-inf"), 0.0, lse_rest).float()
                grad = torch.exp(others - finite) * (diff * coef).float()
            else:
                grad = torch.cat([torch.exp(z - lse.float()), torch.zeros_like(z[:, :1])], 1)
                grad *= (mass * coef).float()
            grad.scatter_(1, slot, ((mass * qi - t) * coef).float())
            out["grad"] = grad[:, :V].to(DT[c["grad"]])
        return out

    hidden, weight = s["hidden"].float(), s["weight"].float()
    z = (hidden @ weight.t()) / T
    lse = _lse(z)
    if c["op"] == "lce":
        keep = s["labels"] != IGNORE
        slot = torch.where(keep, s["labels"].long(), 0)[:, None]
        t = keep.double()[:, None]
        row = torch.where(keep, (lse - torch.gather(z, 1, slot))[:, 0], 0.0)
    else:
        t, _, keep = _targets(s["ids"], s["vals"], None, T)
        slot = s["ids"].long().clamp(min=0)
        row = _xlog(t, torch.log(t) - (torch.gather(z, 1, slot) - lse)).sum(dim=1)
    scale = _row_scale(c, keep, s["row_weight"])
    out = {"loss": (scale * row).sum().float().reshape(1), "row_loss": row.float(), "lse": lse[:, 0].float()}
    if c["grad"] != "none":
        dz = torch.exp(z - lse.float())
        dz.scatter_add_(1, slot, -t.float())
        dz *= (scale * (_grad_scale(c) / T))[:, None]
        dt = s["hidden"].dtype
        out["grad_hidden"] = (dz @ weight).to(dt)
        if c["grad"] == "both":
            out["grad_weight"] = (dz.t() @ hidden).to(dt)
    return out


# ---------------------------------------------------------------------------
# cost and exact answer
# ---------------------------------------------------------------------------

def work(case):
    N, V = case["N"], case["V"]
    es = DT[case["dtype"]].itemsize
    if case["op"] == "kd":
        b = N * V * es + N * case["k"] * 8 + N * 4
        f = 4 * N * V  # scale, exponential, sum, maximum
        if case["grad"] != "none":
            b += N * V * DT[case["grad"]].itemsize
            f += 3 * N * V
        return {"bytes": b, "flops": f}
    H = case["H"]
    grads = {"none": 0, "hidden": 1, "both": 2}[case["grad"]]
    b = (N * H + V * H) * es + N * 12
    b += N * case["k"] * 8 if case["op"] == "lkd" else N * 4
    if grads >= 1:
        b += N * H * es
    if grads == 2:
        b += V * H * es
    return {"bytes": b, "flops": 2 * N * V * H * (1 + grads)}


def exact(case, seed):
    """The definition in 64 bits, its gradients by automatic differentiation."""
    N, V, T = case["N"], case["V"], case["T"]
    if case["op"] != "kd" and work(case)["flops"] > EXACT_FLOPS:
        return None
    s = prepare(case, seed)
    if case["op"] == "kd":
        leaf = s["student"].double().requires_grad_(case["grad"] != "none")
        z = leaf / T
    else:
        leaf = s["hidden"].double().requires_grad_(case["grad"] != "none")
        head = s["weight"].double().requires_grad_(case["grad"] == "both")
        z = torch.matmul(leaf, head.transpose(0, 1)) / T
    norm = torch.logsumexp(z, dim=1)

    if case["op"] == "lce":
        kept = s["labels"] != IGNORE
        picked = z[torch.arange(N, device=z.device), s["labels"].long() * kept]
        row = (norm - picked) * kept
    else:
        kept = (s["ids"] >= 0).sum(dim=1) > 0
        has = s["ids"] >= 0
        logt = (s["vals"].double() / T).masked_fill(~has, float("-inf"))
        if case["op"] == "kd" and case["tail"]:
            logt = logt - s["lse"].double()[:, None]
        else:
            logt = torch.log_softmax(logt.masked_fill(~kept[:, None], 0.0), dim=1).masked_fill(~has, float("-inf"))
        t = logt.exp()
        logq = z.gather(1, s["ids"].long() * has) - norm[:, None]
        safe = logt.masked_fill(t == 0, 0.0)
        row = (t * (safe - logq)).masked_fill(t == 0, 0.0).sum(dim=1)
        if case["op"] == "kd" and case["tail"]:
            rest = 1.0 - t.sum(dim=1)
            rows = torch.nonzero((rest > 1e-6) & kept)[:, 0]
            member = torch.zeros(N, V, dtype=torch.bool, device=z.device)
            n, i = torch.nonzero(has, as_tuple=True)
            member[n, s["ids"].long()[n, i]] = True
            log_qr = torch.logsumexp(z[rows].masked_fill(member[rows], float("-inf")), dim=1) - norm[rows]
            row = row.index_add(0, rows, rest[rows] * (rest[rows].log() - log_qr))
    w = kept.double() if s["row_weight"] is None else s["row_weight"].double() * kept
    loss = (w * row).sum()
    if case["reduction"] == "mean":
        loss = loss / max(int(kept.sum()), 1)
    out = {"loss": loss.detach().reshape(1), "row_loss": row.detach()}
    if case["op"] != "kd":
        out["lse"] = norm.detach()
    if case["grad"] != "none":
        wrt = [leaf] if case["op"] == "kd" or case["grad"] == "hidden" else [leaf, head]
        grads = torch.autograd.grad(_grad_scale(case) * loss, wrt)
        out["grad" if case["op"] == "kd" else "grad_hidden"] = grads[0]
        if len(grads) == 2:
            out["grad_weight"] = grads[1]
    return out
