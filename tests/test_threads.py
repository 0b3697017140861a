"""What the binding caches for a stream: host threads that call on it do not share a
workspace, workspaces can be given up, status words outlive inference mode (CPU).

The library is replaced by one that takes its time, as the launches of a call do, and
notes which workspaces are in use; the tensors are never looked at."""

import ctypes
import threading
import time
from types import SimpleNamespace

import pytest
import torch

import sampling_spec_verify_gb300 as ssv


class SlowLibrary:
    def __init__(self):
        self.busy, self.mixed, self.calls, self.guard = set(), 0, 0, threading.Lock()

    def __getattr__(self, name):
        if name.endswith("workspace_bytes"):
            return lambda *a: 4096

        def call(*a):
            ws = a[-3].value if isinstance(a[-3], ctypes.c_void_p) else a[-3]
            with self.guard:
                self.mixed += ws in self.busy
                self.busy.add(ws)
                self.calls += 1
            time.sleep(0.002)
            with self.guard:
                self.busy.discard(ws)
            return 0
        return call


@pytest.fixture
def slow(monkeypatch):
    L = SlowLibrary()
    monkeypatch.setattr(ssv, "lib", lambda: L)
    monkeypatch.setattr(ssv, "_need", lambda *a, **k: None)
    monkeypatch.setattr(ssv, "_loss_stream", lambda given, device: 0)
    monkeypatch.setattr(ssv, "_stream_handle", lambda s, device: (ctypes.c_void_p(0), SimpleNamespace(cuda_stream=0)))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    for cache in ("_WS", "_SCRATCH", "_STATUS"):
        monkeypatch.setattr(ssv, cache, {})
    monkeypatch.setattr(ssv, "_STATUS_WORDS", 2)  # the block of status words runs out often
    return L


def zeros(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


def calls():
    x, w, y = zeros(4, 8, dtype=torch.bfloat16), zeros(16, 8, dtype=torch.bfloat16), zeros(4, dtype=torch.int32)
    ids, tl = zeros(4, 2, dtype=torch.int32), zeros(4, 2)
    t, d = zeros(2, 4, 16), zeros(2, 3, 16)
    tok, u, uf = zeros(2, 3, dtype=torch.int32), zeros(2, 3), zeros(2)
    return [lambda: ssv.linear_cross_entropy_fwd_bwd(x, w, y), lambda: ssv.linear_topk_distill(x, w, ids, tl),
            lambda: ssv.topk_distill_fwd_bwd(zeros(4, 16), ids, tl), lambda: ssv.topk_distill(zeros(4, 16), ids, tl),
            lambda: ssv.verify(t, d, tok, u, uf, 1.0), lambda: ssv.verify_relaxed(t, d, tok, uf, 1.0),
            lambda: ssv.overlap(t, d, 1.0), lambda: ssv.e2e_tv_fwd_bwd(t, d, 1.0), lambda: ssv.diagnostics(t, d, 1.0),
            lambda: ssv.tree_verify_greedy(t, tok, tok),
            lambda: ssv.verify_ragged(zeros(4, 16), zeros(2, 16), zeros(3, dtype=torch.int32), tok[:, 0], uf, uf, 1.0)]


@pytest.mark.parametrize("which", [slice(0, 4), slice(4, 11)], ids=["losses", "others"])
def test_calls_of_two_threads_do_not_mix(slow, which):
    failed = []

    def work(first):
        try:
            fs = calls()[which]
            for i in range(12):
                fs[(first + i) % len(fs)]()
        except Exception as e:  # noqa: BLE001
            failed.append(repr(e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed and slow.calls == 48 and slow.mixed == 0


def test_a_refused_call_releases_its_stream(slow, monkeypatch):
    x = zeros(4, 8, dtype=torch.bfloat16)
    monkeypatch.setattr(ssv, "_loss_buffers", lambda *a: 1 / 0)
    with pytest.raises(ZeroDivisionError):
        ssv.linear_cross_entropy(x, x, zeros(4, dtype=torch.int32))
    assert not ssv._held(x.device, 0).locked()


def test_cached_workspaces_can_be_released(slow):
    loss = calls()[0]
    loss()
    assert [w.numel() for w in ssv._SCRATCH.values()] == [4096]
    held = ssv._held(torch.device("cpu"), 0)
    held.acquire()  # a call is between its look-up and its last launch
    t = threading.Thread(target=ssv.release_workspaces)
    t.start()
    time.sleep(0.05)
    assert len(ssv._SCRATCH) == 1 and t.is_alive()
    held.release()
    t.join()
    assert not ssv._SCRATCH
    loss()
    assert len(ssv._SCRATCH) == 1 and slow.calls == 2
    ssv.release_workspaces()


def test_status_words_of_a_block_made_in_inference_mode(slow):
    """An evaluation call makes the block of status words, a training call's may be written to."""
    with torch.inference_mode():
        calls()[3]()
    o = calls()[2]()
    o.status.zero_()
    o.status |= 1
    assert not o.status.is_inference()
