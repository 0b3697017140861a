"""Refusals of the decoding step's entry points before any launch (CPU)."""

import ctypes
import os
from types import SimpleNamespace

import pytest
import torch

import sampling_spec_verify_gb300 as ssv

OK, INVALID, UNSUPPORTED = 0, 1, 2
P = 0x10000      # aligned, never dereferenced: every call below is refused
ODD = 0x10008
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(ssv.LIB_PATH):
        from sampling_spec_verify_gb300 import build
        build.build()
    return ssv.lib()


def structure(pointers, longs, ints, floats=()):
    class C(ctypes.Structure):
        _fields_ = ([(n, ctypes.c_void_p) for n in pointers.split()]
                    + [(n, ctypes.c_longlong * k if k > 1 else ctypes.c_longlong) for n, k in longs]
                    + [(n, ctypes.c_int) for n in ints.split()] + [(n, ctypes.c_float) for n in floats])
    return C


ATTENTION = structure("q k_new v_new k_cache v_cache out lse block_table context_lens row_offsets mask",
                      (("q_stride", 2), ("k_new_stride", 2), ("v_new_stride", 2), ("k_stride", 3), ("v_stride", 3),
                       ("table_stride", 1)),
                      "B T rows Hq Hkv D pages page_size table_width dtype", ("scale",))
COMMIT_T = structure("k_new v_new k_cache v_cache slots path row_offsets",
                     (("k_new_stride", 3), ("v_new_stride", 3), ("k_stride", 4), ("v_stride", 4), ("path_stride", 1)),
                     "layers B T rows S Hkv D pages page_size dtype")
ADJUST_T = structure("logits out tokens history history_lens prompt_lens repetition frequency presence bias_ids bias "
                     "allowed row_offsets mask", (), "B T rows V history_width biases dtype")


def test_packed_arguments_are_the_structures():
    for packed, c in ((ssv._ATTENTION, ATTENTION), (ssv._COMMIT, COMMIT_T), (ssv._ADJUST, ADJUST_T)):
        assert packed.size == ctypes.sizeof(c)
    a = ATTENTION.from_buffer_copy(ssv._ATTENTION.pack(*range(1, 35), 0.5))
    assert (a.q, a.mask, list(a.v_stride), a.table_stride, a.B, a.dtype, a.scale) == (1, 11, [21, 22, 23], 24, 25, 34, 0.5)


def struct(cls, fields, o):
    a = cls()
    for k, v in dict(fields, **o).items():
        setattr(a, k, getattr(a, k).__class__(*v) if isinstance(v, tuple) else v)
    return a


ATTN = dict(q=P, k_new=P, v_new=P, k_cache=P, v_cache=P, out=P, block_table=P, context_lens=P, q_stride=(256, 64),
            k_new_stride=(128, 64), v_new_stride=(128, 64), k_stride=(2048, 128, 64), v_stride=(2048, 128, 64),
            table_stride=9, B=2, T=3, rows=6, Hq=4, Hkv=2, D=64, pages=20, page_size=16, table_width=9, dtype=1,
            scale=0.125)


@pytest.mark.parametrize("o,want", [
    (dict(B=-1), INVALID), (dict(T=0), INVALID), (dict(rows=-1), INVALID), (dict(rows=5), INVALID),
    (dict(Hkv=0), INVALID), (dict(Hq=5), INVALID), (dict(Hq=258), UNSUPPORTED), (dict(D=0), INVALID), (dict(D=60), UNSUPPORTED),
    (dict(D=264), UNSUPPORTED), (dict(page_size=0), INVALID), (dict(page_size=12), UNSUPPORTED),
    (dict(T=1025, rows=2050), UNSUPPORTED), (dict(table_width=-1), INVALID), (dict(table_stride=8), INVALID),
    (dict(dtype=0), INVALID), (dict(dtype=3), INVALID), (dict(scale=NAN), INVALID), (dict(scale=INF), INVALID),
    (dict(scale=3e38), INVALID),
    (dict(pages=-1), INVALID), (dict(q=None), INVALID), (dict(k_new=None), INVALID), (dict(v_new=None), INVALID),
    (dict(k_cache=None), INVALID), (dict(v_cache=None), INVALID), (dict(out=None), INVALID),
    (dict(block_table=None), INVALID), (dict(context_lens=None), INVALID), (dict(q=ODD), INVALID),
    (dict(k_new=ODD), INVALID), (dict(v_new=ODD), INVALID), (dict(k_cache=ODD), INVALID), (dict(out=ODD), INVALID),
    (dict(q_stride=(256, 60)), INVALID), (dict(q_stride=(0, 64)), INVALID), (dict(k_stride=(2048, 128, 4)), INVALID),
    (dict(v_stride=(2 ** 39, 128, 64)), INVALID), (dict(k_new_stride=(-128, 64)), INVALID),
    (dict(B=0, rows=0), OK), (dict(B=2, rows=0, row_offsets=P), OK)])
def test_attention_refuses(L, o, want):
    a = struct(ATTENTION, ATTN, o)
    assert L.spec_tree_attention(ctypes.byref(a), None, P, 1 << 40, None) == want


def test_attention_workspace(L):
    a = struct(ATTENTION, ATTN, {})
    need = L.spec_tree_attention_workspace_bytes(2, 3, 4, 2, 64)
    assert need > 0
    assert L.spec_tree_attention(ctypes.byref(a), None, None, need, None) == INVALID
    assert L.spec_tree_attention(ctypes.byref(a), None, P, need - 1, None) == INVALID
    assert L.spec_tree_attention(None, None, P, need, None) == INVALID
    for bad in ((-1, 3, 4, 2, 64), (2, 0, 4, 2, 64), (2, 3, 5, 2, 64), (2, 3, 4, 0, 64), (2, 3, 4, 2, 12),
                (2, 3, 4, 2, 264), (2, 1025, 4, 2, 64)):
        assert L.spec_tree_attention_workspace_bytes(*bad) == 0


def plan(L, **o):
    a = dict(lens=0x10000, new=0x20000, table=0x30000, free=0x40000, count=0x50000, B=4, T=3, width=8, capacity=32,
             page=16, out_table=0x60000, out_free=0x70000, out_count=0x80000, out_lens=0x90000, slots=0xA0000)
    a.update(o)
    return L.spec_plan_cache(*a.values(), None, None)


@pytest.mark.parametrize("o,want", [
    (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(width=0), INVALID), (dict(capacity=-1), INVALID),
    (dict(page=0), INVALID), (dict(lens=None), INVALID), (dict(new=None), INVALID), (dict(table=None), INVALID),
    (dict(free=None), INVALID), (dict(count=None), INVALID), (dict(out_table=None), INVALID),
    (dict(out_free=None), INVALID), (dict(out_count=None), INVALID), (dict(out_lens=None), INVALID),
    (dict(slots=None), INVALID), (dict(out_count=0x50000), INVALID), (dict(out_lens=0x10000), INVALID),
    (dict(out_lens=0x20008), INVALID), (dict(out_table=0x30004), INVALID), (dict(out_free=0x40040), INVALID),
    (dict(slots=0x30000), INVALID), (dict(out_lens=0x40000), INVALID),
    (dict(B=1 << 20, width=1 << 12), UNSUPPORTED), (dict(B=1 << 20, T=1 << 12), UNSUPPORTED),
    (dict(width=1 << 16, page=1 << 15), UNSUPPORTED)])
def test_plan_refuses(L, o, want):
    assert plan(L, **o) == want


COMMIT = dict(k_new=P, v_new=P, k_cache=P, v_cache=P, slots=P, k_new_stride=(512, 128, 64), v_new_stride=(512, 128, 64),
              k_stride=(65536, 2048, 128, 64), v_stride=(65536, 2048, 128, 64), path_stride=2, layers=1, B=2, T=3,
              rows=6, S=3, Hkv=2, D=64, pages=20, page_size=16, dtype=1)


@pytest.mark.parametrize("o,want", [
    (dict(layers=-1), INVALID), (dict(B=-1), INVALID), (dict(T=0), INVALID), (dict(rows=7), INVALID),
    (dict(S=-1), INVALID), (dict(Hkv=0), INVALID), (dict(D=0), INVALID), (dict(D=12), UNSUPPORTED),
    (dict(page_size=0), INVALID), (dict(pages=1 << 30), UNSUPPORTED), (dict(dtype=0), INVALID),
    (dict(k_new=None), INVALID), (dict(v_cache=None), INVALID), (dict(slots=None), INVALID), (dict(v_new=ODD), INVALID),
    (dict(k_cache=ODD), INVALID), (dict(path=P, path_stride=1), INVALID), (dict(k_stride=(1, 2048, 128, 64)), INVALID),
    (dict(v_new_stride=(512, -8, 64)), INVALID), (dict(layers=0), OK), (dict(S=0), OK), (dict(B=0, rows=0), OK)])
def test_commit_refuses(L, o, want):
    a = struct(COMMIT_T, COMMIT, o)
    assert L.spec_commit_cache(ctypes.byref(a), None, None) == want
    assert L.spec_commit_cache(None, None, None) == INVALID


ADJUST = dict(logits=P, out=P, tokens=P, history=P, history_lens=P, B=2, T=3, rows=6, V=100, history_width=7, biases=0,
              dtype=1)


@pytest.mark.parametrize("o,want", [
    (dict(B=-1), INVALID), (dict(T=0), INVALID), (dict(rows=5), INVALID), (dict(V=0), INVALID), (dict(V=1 << 25), UNSUPPORTED),
    (dict(history_width=-1), INVALID), (dict(history_width=1 << 19), UNSUPPORTED), (dict(biases=-1), INVALID),
    (dict(biases=1025, bias_ids=P, bias=P), UNSUPPORTED), (dict(biases=3), INVALID), (dict(biases=3, bias=P), INVALID),
    (dict(T=1025, rows=2050), UNSUPPORTED), (dict(dtype=2), INVALID), (dict(logits=None), INVALID),
    (dict(out=None), INVALID), (dict(tokens=None), INVALID), (dict(history=None), INVALID),
    (dict(history_lens=None), INVALID), (dict(logits=P + 1), INVALID), (dict(out=P + 2), INVALID),
    (dict(out=P + 1198), INVALID), (dict(B=0, rows=0), OK), (dict(rows=0, row_offsets=P), OK)])
def test_adjust_refuses(L, o, want):
    a = struct(ADJUST_T, ADJUST, o)
    assert L.spec_adjust_logits(ctypes.byref(a), None, None) == want
    assert L.spec_adjust_logits(None, None, None) == INVALID


class Fake:
    """Stands for a contiguous CUDA tensor."""

    def __init__(self, *shape, dtype=torch.int32, index=0, stride=None):
        self.shape, self.dtype, self.device, self.is_cuda = torch.Size(shape), dtype, torch.device("cuda", index), True
        self._stride = stride or torch.empty(shape, device="meta").stride()

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def stride(self, d=None):
        return self._stride if d is None else self._stride[d]

    def get_device(self):
        return self.device.index

    def is_contiguous(self):
        return self._stride == torch.empty(self.shape, device="meta").stride()

    def data_ptr(self):
        return P


class Calls:
    def __init__(self):
        self.n = 0

    def __getattr__(self, name):
        def call(*a):
            self.n += 1
            return 0
        return (lambda *a: 4096) if name.endswith("workspace_bytes") else call


@pytest.fixture
def calls(monkeypatch):
    c = Calls()
    monkeypatch.setattr(ssv, "lib", lambda: c)
    monkeypatch.setattr(torch, "Tensor", Fake)
    monkeypatch.setattr(torch, "empty_like", lambda t, **k: t)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(ssv, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(ssv, "_loss_buffers", lambda *a: (Fake(1), SimpleNamespace(data_ptr=lambda: P, nbytes=1 << 20),
                                                          [Fake(*s, dtype=d) for s, d in a[-1]]))
    return c


def attn(i=0, **o):
    h = lambda *s, **k: Fake(*s, dtype=torch.bfloat16, index=i, **k)  # noqa: E731
    a = dict(q=h(2, 3, 4, 64), k_new=h(2, 3, 2, 64), v_new=h(2, 3, 2, 64), k_cache=h(9, 16, 2, 64),
             v_cache=h(9, 16, 2, 64), block_table=Fake(2, 5, index=i), context_lens=Fake(2, index=i))
    a.update({k: o.pop(k) for k in list(o) if k in a})
    return ssv.tree_attention(*a.values(), **o)


def planned(i=0, **o):
    f = lambda *s: Fake(*s, index=i)  # noqa: E731
    a = dict(context_lens=f(2), new_lens=f(2), block_table=f(2, 5), free_pages=f(9), free_count=f(1), page_size=16,
             max_new=3)
    a.update({k: o.pop(k) for k in list(o) if k in a})
    return ssv.plan_cache(*a.values(), **o)


def commit(i=0, **o):
    h = lambda *s, **k: Fake(*s, dtype=torch.float16, index=i, **k)  # noqa: E731
    a = dict(k_new=h(2, 3, 2, 64), v_new=h(2, 3, 2, 64), k_cache=h(9, 16, 2, 64), v_cache=h(9, 16, 2, 64),
             slots=Fake(2, 3, index=i))
    a.update({k: o.pop(k) for k in list(o) if k in a})
    return ssv.commit_cache(*a.values(), **o)


def adjust(i=0, **o):
    f = lambda *s, **k: Fake(*s, index=i, **k)  # noqa: E731
    a = dict(logits=f(2, 3, 70, dtype=torch.float32), tokens=f(2, 3), history=f(2, 9), history_lens=f(2))
    a.update({k: o.pop(k) for k in list(o) if k in a})
    return ssv.adjust_logits(*a.values(), **o)


@pytest.mark.parametrize("call", [attn, planned, commit, adjust])
def test_another_device_is_refused(calls, call):
    call()
    call(stream=SimpleNamespace(cuda_stream=7, device_index=0)) if call is not adjust else call()
    assert calls.n == 2
    with pytest.raises(ValueError, match="current device"):
        call(i=1)
    with pytest.raises(ValueError):
        call(stream=SimpleNamespace(cuda_stream=7, device_index=1), **({"out": Fake(2, 3, 70, dtype=torch.float32)} if call is adjust else {}))
    assert calls.n == 2


H = torch.bfloat16


@pytest.mark.parametrize("o", [
    dict(q=Fake(2, 3, 4, 64, dtype=torch.float32)), dict(q=Fake(6, 4, 64, dtype=H)),
    dict(q=Fake(2, 3, 4, 32, dtype=H)), dict(k_new=Fake(2, 3, 1, 64, dtype=H)), dict(v_new=Fake(2, 2, 2, 64, dtype=H)),
    dict(v_new=Fake(2, 3, 2, 64, dtype=torch.float16)), dict(v_cache=Fake(9, 16, 1, 64, dtype=H)),
    dict(k_cache=Fake(9, 16, 2, 64, dtype=H, stride=(2048, 128, 64, 2))),
    dict(q=Fake(2, 3, 4, 64, dtype=H, stride=(1000, 256, 64, 1))), dict(block_table=Fake(3, 5)),
    dict(block_table=Fake(2, 5, dtype=torch.int64)), dict(context_lens=Fake(3)), dict(max_rows=3),
    dict(mask=Fake(2, 3, 3, dtype=torch.bool)), dict(mask=Fake(2, 3, 4, dtype=torch.uint8)),
    dict(row_offsets=Fake(3)), dict(out=ssv.AttentionOutput(Fake(2, 3, 4, 63, dtype=H), None, Fake(1))),
    dict(out=ssv.AttentionOutput(Fake(2, 3, 4, 64, dtype=H), Fake(2, 3, 4), Fake(1)))])
def test_attention_arguments(calls, o):
    with pytest.raises((ValueError, TypeError)):
        attn(**o)
    assert calls.n == 0


def test_ragged_attention_arguments(calls):
    rows = {k: Fake(7, n, 64, dtype=H) for k, n in (("q", 4), ("k_new", 2), ("v_new", 2))}
    attn(**rows, row_offsets=Fake(3), max_rows=5)
    for o in (dict(max_rows=None), dict(max_rows=0), dict(row_offsets=Fake(4)), dict(row_offsets=Fake(2, 3)),
              dict(row_offsets=Fake(3, dtype=torch.int64)), dict(k_new=Fake(6, 2, 64, dtype=H))):
        with pytest.raises((ValueError, TypeError)):
            attn(**{**rows, **dict(row_offsets=Fake(3), max_rows=5), **o})
    assert calls.n == 1


@pytest.mark.parametrize("call,o", [
    (planned, dict(new_lens=Fake(3))), (planned, dict(block_table=Fake(2, 5, dtype=torch.int64))),
    (planned, dict(free_count=Fake(2))), (planned, dict(max_new=-1)), (planned, dict(free_pages=Fake(3, 3))),
    (planned, dict(out=ssv.CachePlan(Fake(2, 5), Fake(9), Fake(1), Fake(2), Fake(2, 4), Fake(1)))),
    (commit, dict(slots=Fake(3, 3))), (commit, dict(path=Fake(2, 1))), (commit, dict(k_new=Fake(2, 3, 1, 64, dtype=torch.float16))),
    (commit, dict(k_new=Fake(6, 2, 64, dtype=torch.float16))), (commit, dict(v_cache=Fake(9, 16, 2, 64))),
    (commit, dict(row_offsets=Fake(3))), (commit, dict(k_cache=Fake(16, 2, 64, dtype=torch.float16))),
    (adjust, dict(tokens=Fake(2, 4))), (adjust, dict(history=Fake(3, 9))), (adjust, dict(history_lens=Fake(3))),
    (adjust, dict(logits=Fake(2, 3, 70, dtype=torch.float16))), (adjust, dict(bias=Fake(2, 3, dtype=torch.float32))),
    (adjust, dict(bias=Fake(2, 3, dtype=torch.float32), bias_ids=Fake(2, 4))), (adjust, dict(allowed=Fake(2, 3, 2))),
    (adjust, dict(repetition=Fake(3, dtype=torch.float32))), (adjust, dict(out=Fake(2, 3, 71, dtype=torch.float32))),
    (adjust, dict(mask=Fake(1, 3, 3, dtype=torch.uint8))), (adjust, dict(max_rows=2))])
def test_arguments(calls, call, o):
    with pytest.raises((ValueError, TypeError)):
        call(**o)
    assert calls.n == 0


def test_the_rules_threads_share_their_verdict_on_a_wait():
    """A wait that runs out in any thread ends the kernel's loop over rows, and thread 0 has to report
    it and to wait for the copies in flight.  No GPU test can make one thread's wait run out
    there, so this one reads the source: the loop ends by the block's answer, kept in the variable that
    thread 0 asks behind it."""
    text = open(os.path.join(os.path.dirname(ssv.__file__), "csrc", "adjust.cuh")).read()
    loop = text[text.index("bool ok = true;\n  for (int i = 0; i < rows; ++i)"):]
    assert "ok = block_waited(ok);\n    if (!ok) break;" in loop
    assert "__syncthreads_and" not in text and loop.count("break;") == 1
    assert "if (!ok) {\n      raise(P.status, SPEC_DEV_TIMEOUT);" in loop


def test_lse_that_has_no_place_is_refused(calls):
    out = lambda lse: ssv.AttentionOutput(Fake(2, 3, 4, 64, dtype=H), lse, Fake(1))  # noqa: E731
    with pytest.raises(ValueError, match="lse"):
        attn(out=out(None), want_lse=True)
    assert calls.n == 0
    attn(out=out(Fake(2, 3, 4, dtype=torch.float32)), want_lse=True)
    attn(out=out(None))
    assert calls.n == 2


def test_adjust_refuses_more_than_65535_requests(L):
    a = struct(ADJUST_T, ADJUST, dict(B=65536, T=1, rows=65536))
    assert L.spec_adjust_logits(ctypes.byref(a), None, None) == UNSUPPORTED
    text = open(os.path.join(os.path.dirname(ssv.__file__), "..", "include", "spec_verify.h")).read()
    assert "B <= 65535" in text.split("Sampling rules on the logits")[1].split("spec_adjust_logits(")[0]
