"""The packed product at layer sizes whose reduction is split unevenly over a
cluster, a few tokens at a time.

Inputs are exact: activations whole numbers up to 2, scales 1/4 to 1, so every
partial sum is a multiple of 1/4 no larger than 2 (2^bits - 1) d_in < 2^22,
which fp32 holds in any order, and the outputs have to be equal to float64's.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def A():
    from post_weight_quantization_10_b200 import admmq
    admmq.lib()
    return admmq


def layer(A, n, k, bits, group, seed):
    """packed, scale, zero of random codes, and the weights in float64."""
    assert 2 * (2 ** bits - 1) * k < 2 ** 22
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def whole(lo, hi, shape, dtype):
        return torch.randint(lo, hi, shape, generator=gen, device="cuda").to(dtype)

    codes = whole(0, 2 ** bits, (n, k), torch.uint8)
    zero = whole(0, 2 ** bits, (n, k // group), torch.float32)
    scale = torch.exp2(whole(-2, 1, (n, k // group), torch.float32))
    w = codes.double().view(n, -1, group) - zero.double()[:, :, None]
    return A.pack(codes, bits), scale, zero, (w * scale.double()[:, :, None]).view(n, k)


def tokens(m, k, dtype, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-2, 3, (m, k), generator=gen, device="cuda").to(dtype)


# m, d_in, d_out, bits, group, whether scales move in 16-byte pieces
SPLITS = [(8, 5120, 5120, 4, 128, False), (12, 5120, 4096, 3, 128, False), (10, 2560, 4096, 4, 128, False),
          (9, 2560, 2560, 2, 128, False), (12, 3584, 3584, 3, 128, False), (2, 25600, 5120, 3, 128, False),
          (4, 9728, 2560, 5, 128, False), (8, 13824, 5120, 4, 128, False), (9, 2304, 4096, 4, 64, False),
          (9, 768, 768, 4, 64, False), (10, 8704, 34, 3, 64, False), (10, 8448, 34, 3, 64, False),
          (12, 1536, 768, 8, 64, False), (9, 2080, 640, 4, 32, False), (10, 4096, 4096, 4, 128, True),
          (11, 12288, 4096, 2, 128, True)]


@pytest.mark.parametrize("m,k,n,bits,group,pieces", SPLITS)
def test_uneven_splits(A, m, k, n, bits, group, pieces):
    plan = A.debug_packed_plan(m, k, n, bits, group)
    assert plan["ranks"] > 1 and plan["vec_scales"] == pieces, plan
    packed, scale, zero, w = layer(A, n, k, bits, group, m + k)
    for dtype in (torch.bfloat16, torch.float16):
        x = tokens(m, k, dtype, n)
        want = x.double() @ w.T
        for out in (torch.float32, dtype):
            assert torch.equal(A.packed_matmul(x, packed, scale, zero, bits, out), want.to(out)), out
