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
