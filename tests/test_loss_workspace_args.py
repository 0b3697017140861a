"""Arguments of the training losses that the binding looks at before the library is
called: workspaces that the kernels cannot write to, values that an int32 cannot hold
(CPU; the tensors only claim to be on a GPU)."""

import pytest
import torch

import sampling_spec_verify_gb300 as ssv


class OnGpu(torch.Tensor):
    is_cuda = True
    device = torch.device("cuda", 0)


class OnAnother(torch.Tensor):
    is_cuda = True
    device = torch.device("cuda", 1)


def gpu(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)


class Library:
    def __init__(self):
        self.sizes, self.args = [], None

    def __getattr__(self, name):
        if name.endswith("workspace_bytes"):
            return lambda *a: 4096

        def call(*a):
            self.sizes.append(a[-2])
            self.args = a
            return 0
        return call


@pytest.fixture
def library(monkeypatch):
    L = Library()
    monkeypatch.setattr(ssv, "lib", lambda: L)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(ssv, "_raw_stream", lambda index: 0)
    return L


def calls(ws):
    x, w, y = gpu(4, 8, dtype=torch.bfloat16), gpu(9, 8, dtype=torch.bfloat16), gpu(4, dtype=torch.int32)
    ids, tl, status = gpu(4, 2, dtype=torch.int32), gpu(4, 2), gpu(1, dtype=torch.int32)
    head = lambda *g: ssv.LinearLossOutput(gpu(1), gpu(4), gpu(4), *g, status)  # noqa: E731
    grads = (gpu(4, 8, dtype=torch.bfloat16), gpu(9, 8, dtype=torch.bfloat16))
    z = gpu(4, 9)
    return [lambda: ssv.linear_cross_entropy(x, w, y, out=head(None, None), workspace=ws),
            lambda: ssv.linear_cross_entropy_fwd_bwd(x, w, y, out=head(*grads), workspace=ws),
            lambda: ssv.linear_topk_distill(x, w, ids, tl, out=head(None, None), workspace=ws),
            lambda: ssv.linear_topk_distill_fwd_bwd(x, w, ids, tl, out=head(*grads), workspace=ws),
            lambda: ssv.topk_distill(z, ids, tl, out=ssv.DistillOutput(gpu(1), gpu(4), None, status), workspace=ws),
            lambda: ssv.topk_distill_fwd_bwd(z, ids, tl, out=ssv.DistillOutput(gpu(1), gpu(4), gpu(4, 9), status),
                                             workspace=ws)]


@pytest.mark.parametrize("which", range(6))
def test_workspaces(library, which):
    calls(gpu(5000, dtype=torch.uint8))[which]()
    calls(gpu(700, 3))[which]()  # of any type
    assert library.sizes == [5000, 8400]
    for bad in (torch.zeros(1 << 20, dtype=torch.uint8),                        # host memory
                torch.zeros(1 << 20, dtype=torch.uint8).as_subclass(OnAnother),
                gpu(1, dtype=torch.uint8).expand(1 << 20)):                       # less memory than it says
        with pytest.raises(ValueError, match="workspace"):
            calls(bad)[which]()
    with pytest.raises(TypeError):
        calls(12345678)[which]()
    assert library.sizes == [5000, 8400]


@pytest.mark.parametrize("bwd", [False, True])
def test_ignore_index(library, bwd):
    """An index that 32 bits would cut to another label is refused."""
    x, w, y = gpu(4, 8, dtype=torch.bfloat16), gpu(9, 8, dtype=torch.bfloat16), gpu(4, dtype=torch.int32)
    out = ssv.LinearLossOutput(gpu(1), gpu(4), gpu(4), gpu(4, 8, dtype=torch.bfloat16) if bwd else None,
                               gpu(9, 8, dtype=torch.bfloat16) if bwd else None, gpu(1, dtype=torch.int32))
    call = ssv.linear_cross_entropy_fwd_bwd if bwd else ssv.linear_cross_entropy
    for i in (-100, 0, 2 ** 31 - 1, -2 ** 31, torch.tensor(-7)):
        call(x, w, y, ignore_index=i, out=out, workspace=gpu(5000))
        assert int(i) in library.args
    for i in (2 ** 31, -2 ** 31 - 1, 2 ** 32, 3 * 2 ** 40):
        with pytest.raises(ValueError, match="ignore_index"):
            call(x, w, y, ignore_index=i, out=out, workspace=gpu(5000))
