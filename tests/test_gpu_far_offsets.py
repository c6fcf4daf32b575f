"""Matrices whose offsets pass 32 bits (elements past 2^31, bytes past 2^32):
their last rows have to equal a call on these rows alone, which is small."""
import pytest
import torch

from test_gpu_packed_splits import layer, tokens

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def A():
    from post_weight_quantization_10_b200 import admmq
    admmq.lib()
    yield admmq
    torch.cuda.empty_cache()


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_quantised_and_back(A, fmt):
    rows, k, tail = 128 * 550, 32768, 128 * 2
    assert rows * k > 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty((rows, k), dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=gen)
    q = A.mx_quantize(x, fmt)
    last = A.mx_quantize(x[-tail:], fmt)
    assert torch.equal(q.codes[-tail:], last.codes)
    assert torch.equal(q.scale[-last.scale.numel():], last.scale)
    out = A.mx_dequantize(q)
    assert torch.equal(out[-tail:], A.mx_dequantize(last))


def test_mx_product(A):
    m, n, k, tail = 131100, 16500, 64, 300
    assert m * n > 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((m, k), generator=gen, device="cuda").bfloat16()
    w = A.mx_quantize(torch.randn((n, k), generator=gen, device="cuda").bfloat16())
    y = A.mx_linear(x, w)
    assert torch.equal(y[-tail:], A.mx_linear(x[-tail:], w))


@pytest.mark.parametrize("m,n,k,bits", [(131100, 16500, 64, 3), (1, 2_200_000, 4096, 8), (12, 2_200_000, 4096, 8),
                                        (40, 2_200_000, 4096, 8)])
def test_packed_product(A, m, n, k, bits):
    group = 64
    if m * n > 2 ** 31:
        packed, scale, zero, w = layer(A, n, k, bits, group, 3)
        x = tokens(m, k, torch.bfloat16, 4)
        y = A.packed_matmul(x, packed, scale, zero, bits)
        assert torch.equal(y[-300:], (x[-300:].double() @ w.T).bfloat16())
        return
    assert n * k * bits // 32 > 2 ** 31
    # the same 1000 rows over and over; the last ones are different
    rows, last = 1000, 1000
    packed, scale, zero, w = layer(A, rows, k, bits, group, 5)
    p2, s2, z2, w2 = layer(A, last, k, bits, group, 6)
    x = tokens(m, k, torch.bfloat16, 7)
    packed = torch.cat([packed.repeat(n // rows - 1, 1), p2])
    scale, zero = (torch.cat([a.repeat(n // rows - 1, 1), b]) for a, b in ((scale, s2), (zero, z2)))
    y = A.packed_matmul(x, packed, scale, zero, bits, torch.float32)
    assert torch.equal(y[:, -last:], (x.double() @ w2.T).float())
    want = (x.double() @ w.T).float()
    assert bool((y[:, :-last].view(m, -1, rows) == want[:, None]).all())
