"""The binding makes a tensor's device current before it asks the library
anything that depends on the device (on the host, with a stand-in for the
library and for torch's notion of the current device)."""
import contextlib
import types

import pytest
import torch

from post_weight_quantization_10_b200 import admmq as A


class _Tensor:
    """As much of a CUDA tensor as the binding looks at."""
    is_cuda, requires_grad = True, False

    def __init__(self, shape, dtype, index):
        self.shape, self.dtype = torch.Size(shape), dtype
        self.device = torch.device("cuda", index)

    def dim(self):
        return len(self.shape)

    def stride(self, i):
        return 1 if i == self.dim() - 1 else self.shape[-1]

    def is_contiguous(self):
        return True

    def numel(self):
        return self.shape.numel()

    def data_ptr(self):
        return 0x1000


@pytest.fixture
def asked(monkeypatch):
    """(entry point, device current at the time) of every call."""
    current, calls = [0], []

    @contextlib.contextmanager
    def device(d):
        before, current[0] = current[0], torch.device(d).index
        yield
        current[0] = before

    def entry(name, result):
        def f(*args):
            calls.append((name, current[0]))
            return result
        return f

    fake = types.SimpleNamespace(
        admmq_mx_linear_workspace_bytes=entry("workspace", 512), admmq_mx_linear=entry("linear", 0))
    monkeypatch.setattr(A, "_lib", fake)
    monkeypatch.setattr(A, "_raw_stream", lambda i: 0)
    monkeypatch.setattr(A, "_empty", lambda shape, dtype, dev, stream: _Tensor(shape, dtype, dev.index))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    return calls


@pytest.mark.parametrize("index", [0, 1])
def test_linear_asks_for_its_workspace_on_the_tensors_device(asked, index):
    x = _Tensor((40, 64), torch.bfloat16, index)
    w = A.MxTensor._of(_Tensor((16, 32), torch.uint8, index), _Tensor((512,), torch.uint8, index),
                       "mxfp4", None)
    y = A.mx_linear(x, w)
    assert y.shape == (40, 16) and y.device.index == index
    assert asked == [("workspace", index), ("linear", index)]
    assert torch.cuda.current_device() == 0
