"""Refusals of the drafter-training losses before any launch (CPU)."""

import ctypes

import pytest

OK, INVALID, UNSUPPORTED = 0, 1, 2
F32, BF16, F16 = 0, 1, 2
P = ctypes.c_void_p(0x10000)      # aligned, never dereferenced: every call below is refused
ODD = ctypes.c_void_p(0x10002)
ODD1 = ctypes.c_void_p(0x10001)
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    import os

    import sampling_spec_verify_gb300 as ssv
    if not os.path.exists(ssv.LIB_PATH):
        from sampling_spec_verify_gb300 import build
        build.build()
    return ssv.lib()


def kd(L, bwd=True, **o):
    a = dict(z=P, dt=BF16, N=4, V=100, k=3, T=1.0, gs=1.0, ids=P, x=P, lse=None, w=None, red=0, loss=P, row=None,
             grad=P, gdt=BF16, st=None, ws=P, wsb=1 << 30, stream=None)
    a.update(o)
    if bwd:
        return L.spec_topk_distill_fwd_bwd(a["z"], a["dt"], a["N"], a["V"], a["k"], a["T"], a["gs"], a["ids"], a["x"],
                                           a["lse"], a["w"], a["red"], a["loss"], a["row"], a["grad"], a["gdt"],
                                           a["st"], a["ws"], a["wsb"], a["stream"])
    return L.spec_topk_distill(a["z"], a["dt"], a["N"], a["V"], a["k"], a["T"], a["ids"], a["x"], a["lse"], a["w"],
                               a["red"], a["loss"], a["row"], a["st"], a["ws"], a["wsb"], a["stream"])


@pytest.mark.parametrize("o,want", [
    (dict(N=-1), INVALID), (dict(V=0), INVALID), (dict(k=0), INVALID), (dict(k=257), UNSUPPORTED),
    (dict(dt=3), INVALID), (dict(gdt=F16), INVALID), (dict(dt=F32, gdt=BF16), INVALID),
    (dict(T=0.0), INVALID), (dict(T=-1.0), INVALID), (dict(T=NAN), INVALID), (dict(T=INF), INVALID),
    (dict(T=1e-45), INVALID), (dict(gs=INF), INVALID), (dict(gs=NAN), INVALID), (dict(red=2), INVALID),
    (dict(loss=None), INVALID), (dict(z=None), INVALID), (dict(ids=None), INVALID), (dict(x=None), INVALID),
    (dict(grad=None), INVALID), (dict(z=ODD1), INVALID), (dict(grad=ODD1), INVALID),
    (dict(gdt=F32, grad=ODD), INVALID), (dict(dt=F32, gdt=F32, z=ODD), INVALID),
    (dict(ws=None), INVALID), (dict(wsb=100), INVALID), (dict(ws=ctypes.c_void_p(0x10080)), INVALID),
    (dict(V=2_000_000), UNSUPPORTED), (dict(dt=F32, gdt=F32, V=1_000_000), UNSUPPORTED),
])
def test_distill_refuses(L, o, want):
    assert kd(L, **o) == want
    if not {"gdt", "grad", "gs"} & set(o):
        assert kd(L, bwd=False, **o) == want


def head(L, what="lce", bwd=True, **o):
    a = dict(x=P, w=P, dt=BF16, N=4, V=100, H=64, k=3, T=1.0, gs=1.0, ids=P, tl=P, ign=-100, rw=None, red=0, loss=P,
             row=None, lse=None, gx=P, gw=P, gdt=BF16, st=None, ws=P, wsb=1 << 30, stream=None)
    a.update(o)
    dims = [a["x"], a["w"], a["dt"], a["N"], a["V"], a["H"]] + ([a["k"]] if what == "lkd" else [])
    scal = [a["T"]] + ([a["gs"]] if bwd else [])
    tgt = [a["ids"], a["tl"]] if what == "lkd" else [a["ids"], a["ign"]]
    rows = [a["rw"], a["red"], a["loss"], a["row"], a["lse"]]
    g = [a["gx"], a["gw"], a["gdt"]] if bwd else []
    f = {("lce", True): L.spec_linear_cross_entropy_fwd_bwd, ("lce", False): L.spec_linear_cross_entropy,
         ("lkd", True): L.spec_linear_topk_distill_fwd_bwd, ("lkd", False): L.spec_linear_topk_distill}[what, bwd]
    return f(*dims, *scal, *tgt, *rows, *g, a["st"], a["ws"], a["wsb"], a["stream"])


@pytest.mark.parametrize("what", ["lce", "lkd"])
@pytest.mark.parametrize("o,want", [
    (dict(N=-1), INVALID), (dict(V=0), INVALID), (dict(H=0), INVALID), (dict(H=12), INVALID),
    (dict(dt=F32, gdt=F32), INVALID), (dict(dt=3), INVALID), (dict(gdt=F16), INVALID), (dict(red=-1), INVALID),
    (dict(T=0.0), INVALID), (dict(T=NAN), INVALID), (dict(gs=NAN), INVALID), (dict(loss=None), INVALID),
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(ids=None), INVALID), (dict(x=ODD), INVALID),
    (dict(w=ODD), INVALID), (dict(gx=ODD), INVALID), (dict(gw=ODD), INVALID), (dict(gx=None, gw=None), INVALID),
    (dict(ws=None), INVALID), (dict(wsb=1000), INVALID), (dict(ws=ctypes.c_void_p(0x10080)), INVALID),
    (dict(N=(1 << 20) + 1), UNSUPPORTED), (dict(V=(1 << 24) + 1), UNSUPPORTED), (dict(H=(1 << 16) + 8), UNSUPPORTED),
])
def test_head_refuses(L, what, o, want):
    assert head(L, what, **o) == want
    if not {"gdt", "gx", "gw", "gs"} & set(o):
        assert head(L, what, bwd=False, **o) == want


def test_listed_tokens_of_the_head(L):
    assert head(L, "lkd", k=0) == INVALID
    assert head(L, "lkd", k=257) == UNSUPPORTED
    assert head(L, "lkd", tl=None) == INVALID
    assert head(L, "lkd", bwd=False, tl=None) == INVALID


def test_workspace_sizes(L):
    f = L.spec_topk_distill_workspace_bytes
    assert f(-1, 10, 1) == f(1, 0, 1) == f(1, 10, 0) == f(1, 10, 257) == 0
    assert f(8, 1000, 16) >= 2 * 8 * 16 * 4
    def g(*dims, dt=BF16):
        return L.spec_linear_loss_workspace_bytes(dt, *dims)
    assert g(1, 10, 8, 1, 0, 0, dt=F32) == g(1, 10, 8, 1, 0, 0, dt=3) == 0
    assert g(1, 10, 12, 1, 0, 0) == g(1, 10, 0, 1, 0, 0) == g(-1, 10, 8, 1, 0, 0) == g(1, 10, 8, 257, 1, 1) == 0
    a, b, c = g(100, 5000, 256, 1, 0, 0), g(100, 5000, 256, 1, 1, 0), g(100, 5000, 256, 1, 1, 1)
    assert a > 100 * 20 * 8 and b > a + 100 * 5000 * 2 and c == b
    assert g(100, 5000, 256, 1, 1, 0, dt=F16) > b + 100 * 5000 * 4  # fp32 probabilities beside the gradient
    # the logits are never kept: at 65536 rows of 151936 tokens they would be 19.9 GB in 16 bits
    assert g(65536, 151936, 4096, 1, 1, 1) < 3 << 30
