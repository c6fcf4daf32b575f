"""Operators called from other host threads than the one that set things up."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def A():
    from post_weight_quantization_10_b200 import admmq
    admmq.lib()
    return admmq


def _packed(A, m, n, k, bits=4):
    gen = torch.Generator(device="cuda").manual_seed(m + k)
    codes = torch.randint(0, 2 ** bits, (n, k), generator=gen, device="cuda").to(torch.uint8)
    scale = torch.rand((n, k // 128), generator=gen, device="cuda")
    zero = torch.randint(0, 2 ** bits, (n, k // 128), generator=gen, device="cuda").float()
    x = torch.randn((m, k), generator=gen, device="cuda").bfloat16()
    return x, A.pack(codes, bits), scale, zero, bits


def _mx(A, m, n, k, fmt="mxfp4"):
    gen = torch.Generator(device="cuda").manual_seed(m + k)
    w = A.mx_quantize(torch.randn((n, k), generator=gen, device="cuda"), fmt)
    return torch.randn((m, k), generator=gen, device="cuda").bfloat16(), w


@pytest.mark.parametrize("op,m", [("packed", 1), ("packed", 40), ("packed", 2000), ("matmul", 4),
                                  ("matmul", 200), ("linear", 1), ("linear", 40), ("linear", 200),
                                  ("dequantize", 40)])
def test_first_call_of_a_thread(A, op, m):
    """A thread's first use of the GPU is the operator itself, writing into a
    given output."""
    if op == "packed":
        args = _packed(A, m, 256, 512)
        f = A.packed_matmul
    else:
        x, w = _mx(A, m, 256, 512)
        f, args = {"matmul": (A.mx_matmul, (A.mx_quantize(x), w)), "linear": (A.mx_linear, (x, w)),
                   "dequantize": (A.mx_dequantize, (w,))}[op]
    want = f(*args)
    out, errors = torch.zeros_like(want), []
    torch.cuda.synchronize()

    def work():
        try:
            f(*args, out=out)
        except Exception as e:  # noqa: BLE001 (the main thread reports it)
            errors.append(repr(e))

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not errors and torch.equal(out, want), errors


def _launcher(A, op, m, n, k):
    """The operator's C call on a stream of its own, and its output."""
    stream = torch.cuda.Stream()
    if op == "packed":
        x, packed, scale, zero, bits = _packed(A, m, n, k)
        out = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
        args = [x.data_ptr(), 1, m, k, packed.data_ptr(), scale.data_ptr(), zero.data_ptr(), k, n,
                bits, 128, out.data_ptr(), 1, stream.cuda_stream]
        keep, f = (x, packed, scale, zero), A.lib().admmq_packed_matmul
    else:
        x, w = _mx(A, m, n, k)
        a = A.mx_quantize(x)
        out = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
        args = [a.codes.data_ptr(), a.scale.data_ptr(), None, w.codes.data_ptr(), w.scale.data_ptr(),
                None, m, n, k, 0, out.data_ptr(), 1, stream.cuda_stream]
        keep, f = (a, w), A.lib().admmq_mx_matmul
    return (lambda: f(*args)), out, keep


@pytest.mark.parametrize("op,sizes", [
    ("packed", ((1, 64, 128), (8, 64, 4096), (4, 64, 4096))),
    ("packed", ((12, 64, 256), (9, 64, 4096))),
    ("packed", ((13, 128, 128), (40, 19200, 128), (64, 128, 8192), (33, 256, 1024))),
    ("mx", ((1, 64, 256), (16, 128, 4096), (4, 64, 12288))),
])
def test_calls_of_different_sizes_at_once(A, op, sizes):
    """One kernel, launched with different amounts of shared memory by several
    threads: no call is refused, and each has its own result."""
    calls = [_launcher(A, op, *s) for s in sizes]
    torch.cuda.synchronize()
    want = []
    for call, out, _ in calls:
        assert call() == 0
        torch.cuda.synchronize()
        want.append(out.clone())
        out.zero_()
    torch.cuda.synchronize()
    refused = [0] * len(calls)

    def work(i):
        for _ in range(20000):
            refused[i] += calls[i][0]() != 0

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert refused == [0] * len(calls)
    for (_, out, _), w in zip(calls, want):
        assert torch.equal(out, w)
