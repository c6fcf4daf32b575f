"""Quantisation and dequantisation of matrices large enough for the wide blocks
(four 128 x 512 blocks an SM and more), and rows of the output that lie apart.

The small matrices of test_gpu_mx.py are held to the oracle; a large one has to
equal, bit for bit, its 128-row tiles taken a few at a time, which are small.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def A():
    from post_weight_quantization_10_b200 import admmq
    admmq.lib()
    return admmq


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("rows,k", [(128 * 90 + 70, 3104), (128 * 150, 2080), (128 * 600 + 1, 96)])
def test_wide_blocks_equal_narrow_ones(A, fmt, dtype, rows, k):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    blocks = -(-k // 512)
    assert -(-rows // 128) * blocks >= 4 * sms                 # wide
    some = 128 * (4 * sms // blocks // 2)
    assert some // 128 * blocks < 4 * sms                      # narrow
    gen = torch.Generator(device="cuda").manual_seed(rows + k)
    x = torch.randn((rows, k), generator=gen, device="cuda")
    x *= torch.exp(torch.rand((rows, 1), generator=gen, device="cuda") * 12 - 6)
    x[rows // 3] = 0
    x[rows // 2, 5], x[rows - 1, k - 1] = float("nan"), float("inf")
    x = x.to(dtype)
    g = None
    if fmt == "nvfp4":
        g = (x.float().nan_to_num(0, 0, 0).abs().amax() / 2688).reshape(1)
    q = A.mx_quantize(x, fmt, g)
    wide = A.mx_dequantize(q, dtype)
    per = q.scale.numel() // -(-rows // 128)                   # scale bytes of 128 rows
    for r in range(0, rows, some):
        part = A.mx_quantize(x[r:r + some], fmt, g)
        assert torch.equal(part.codes, q.codes[r:r + some])
        assert torch.equal(part.scale, q.scale[r // 128 * per:(r + some) // 128 * per if r + some < rows else None])
        assert torch.equal(A.mx_dequantize(part, dtype).nan_to_num(7.0), wide[r:r + some].nan_to_num(7.0))


@pytest.mark.parametrize("rows,k,ld", [(70, 160, 168), (300, 96, 1024), (128 * 600 + 1, 96, 104)])
@pytest.mark.parametrize("dtype,code", [(torch.float32, 0), (torch.bfloat16, 1)])
def test_dequantised_rows_that_lie_apart(A, rows, k, ld, dtype, code):
    """Through the C entry point: what lies between the rows stays as it was."""
    gen = torch.Generator(device="cuda").manual_seed(rows)
    q = A.mx_quantize(torch.randn((rows, k), generator=gen, device="cuda"))
    out = torch.full((rows, ld), 3.0, dtype=dtype, device="cuda")
    assert A.lib().admmq_mx_dequantize(q.codes.data_ptr(), q.scale.data_ptr(), rows, k, 0, None,
                                       out.data_ptr(), code, ld,
                                       torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(out[:, :k], A.mx_dequantize(q, dtype))
    assert bool((out[:, k:] == 3.0).all())
