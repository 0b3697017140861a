"""Tensors or streams of another device than the current one are refused before any
launch, by every entry point (CPU: the library is replaced by one that counts calls)."""

from types import SimpleNamespace

import pytest
import torch

import sampling_spec_verify_gb300 as ssv


class Counting:
    def __init__(self):
        self.calls = 0

    def __getattr__(self, name):
        def call(*a):
            self.calls += 1
            return 0
        return (lambda *a: 4096) if name.endswith("workspace_bytes") else call


class OnDevice:
    """Stands for a CUDA tensor of device `index`."""

    def __init__(self, index, *shape, dtype=torch.float32):
        self.device, self.shape, self.dtype = torch.device("cuda", index), torch.Size(shape), dtype

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def data_ptr(self):
        return 256

    def element_size(self):
        return 4


def calls(i, stream):
    f = lambda *shape: OnDevice(i, *shape)  # noqa: E731
    n = lambda *shape: OnDevice(i, *shape, dtype=torch.int32)  # noqa: E731
    h = lambda *shape: OnDevice(i, *shape, dtype=torch.bfloat16)  # noqa: E731
    kw = dict(stream=stream)
    return {
        "linear_cross_entropy": lambda: ssv.linear_cross_entropy(h(4, 8), h(9, 8), n(4), **kw),
        "linear_cross_entropy_fwd_bwd": lambda: ssv.linear_cross_entropy_fwd_bwd(h(4, 8), h(9, 8), n(4), **kw),
        "linear_topk_distill": lambda: ssv.linear_topk_distill(h(4, 8), h(9, 8), n(4, 2), f(4, 2), **kw),
        "linear_topk_distill_fwd_bwd": lambda: ssv.linear_topk_distill_fwd_bwd(h(4, 8), h(9, 8), n(4, 2), f(4, 2), **kw),
        "topk_distill": lambda: ssv.topk_distill(f(4, 9), n(4, 2), f(4, 2), **kw),
        "topk_distill_fwd_bwd": lambda: ssv.topk_distill_fwd_bwd(f(4, 9), n(4, 2), f(4, 2), **kw),
        "verify": lambda: ssv.verify(f(1, 3, 9), f(1, 2, 9), n(1, 2), f(1, 2), f(1), 1.0, **kw),
        "overlap": lambda: ssv.overlap(f(1, 3, 9), f(1, 2, 9), 1.0, **kw),
        "truncate_logits": lambda: ssv.truncate_logits(f(3, 9), 1.0, 2, **kw),
        "schedule_lengths": lambda: ssv.schedule_lengths(f(3, 2), f(10), **kw),
    }


@pytest.fixture
def library(monkeypatch):
    L = Counting()
    monkeypatch.setattr(ssv, "lib", lambda: L)
    monkeypatch.setattr(ssv, "_need", lambda *a, **k: None)
    for name in ("empty", "zeros", "empty_like"):
        monkeypatch.setattr(torch, name, lambda *a, **k: OnDevice(0, 1))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: SimpleNamespace(cuda_stream=0, device_index=0))
    monkeypatch.setattr(ssv, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(ssv, "_loss_buffers", lambda *a: (None, SimpleNamespace(data_ptr=lambda: 256, nbytes=1 << 20),
                                                          [OnDevice(0, 1)] * len(a[-1])))
    monkeypatch.setattr(ssv, "_workspace", lambda *a: OnDevice(0, 1 << 20))
    return L


@pytest.mark.parametrize("name", sorted(calls(0, None)))
def test_another_device_is_refused(library, name):
    calls(0, None)[name]()
    calls(0, SimpleNamespace(cuda_stream=7, device_index=0))[name]()
    assert library.calls == 2
    with pytest.raises(ValueError, match="current device"):
        calls(1, None)[name]()
    with pytest.raises(ValueError, match="current device"):
        calls(1, SimpleNamespace(cuda_stream=7, device_index=1))[name]()
    with pytest.raises(ValueError, match="stream belongs"):
        calls(0, SimpleNamespace(cuda_stream=7, device_index=1))[name]()
    assert library.calls == 2
