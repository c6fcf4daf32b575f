"""Products with more tiles than run at once: a block (or cluster) goes on to a
second and third tile with the ring positions, accumulator slots and turns that
the first one left.

Inputs are exact, so the outputs have to be equal to float64's: packed products
as in test_gpu_packed_splits.py; 4-bit products of elements that are multiples
of 1/2 up to 12 (steps 1 and 2), every partial sum a multiple of 1/4 below 2^22.
"""
import numpy as np
import pytest
import torch

from oracle import mx
from test_gpu_packed_splits import layer, tokens

pytestmark = pytest.mark.gpu

DTYPES = (torch.bfloat16, torch.float16)


@pytest.fixture(scope="module")
def A():
    from post_weight_quantization_10_b200 import admmq
    admmq.lib()
    return admmq


def _into_room(f, want, m, n):
    """Each output type, in front of memory that has to stay as it was."""
    for dt in (torch.float32, *DTYPES):
        room = torch.full((m * n + 4096,), 3.0, dtype=dt, device="cuda")
        got = f(dt, room[:m * n].view(m, n))
        assert torch.equal(got, want.to(dt)), dt
        assert bool((room[m * n:] == 3.0).all()), dt


# tokens of a tile, then m, d_in, d_out, bits, group
PACKED = [(512, 2000, 160, 4100, 3, 32), (512, 2000, 160, 4100, 5, 32), (512, 1800, 192, 5000, 8, 64),
          (512, 1100, 384, 6600, 4, 128), (512, 1537, 1280, 4100, 3, 128), (512, 1030, 64, 6530, 7, 64),
          (128, 250, 512, 9700, 2, 64), (128, 256, 384, 9700, 4, 128), (128, 100, 288, 19300, 5, 32),
          (64, 33, 640, 24576, 3, 128), (64, 33, 96, 24500, 3, 32), (64, 64, 192, 40000, 4, 64),
          (8, 1, 512, 9000, 3, 128), (8, 8, 128, 5000, 4, 32), (8, 5, 96, 14000, 1, 32),
          (8, 3, 2560, 5200, 8, 128), (8, 2, 1280, 9700, 3, 64)]


@pytest.mark.parametrize("x_type", DTYPES)
@pytest.mark.parametrize("tile,m,k,n,bits,group", PACKED)
def test_packed_past_the_first_tile(A, tile, m, k, n, bits, group, x_type):
    plan = A.debug_packed_plan(m, k, n, bits, group)
    assert plan["tokens"] == tile and plan["tiles"] > plan["at_once"], plan
    packed, scale, zero, w = layer(A, n, k, bits, group, m + n)
    x = tokens(m, k, x_type, k)
    _into_room(lambda dt, out: A.packed_matmul(x, packed, scale, zero, bits, dt, out=out),
               x.double() @ w.T, m, n)


# two CTAs on one tile of 512 tokens: tails of tokens (an odd half, a half without
# any) and of columns, every width and group
@pytest.mark.parametrize("x_type", DTYPES)
@pytest.mark.parametrize("bits,group,k", [(1, 32, 160), (2, 64, 320), (3, 128, 384), (4, 32, 96), (5, 64, 192),
                                          (6, 128, 256), (7, 32, 224), (8, 128, 512)])
def test_packed_on_pairs_of_ctas(A, bits, group, k, x_type):
    for m, n in ((1100, 6600), (1281, 6530), (2048, 4100), (1500, 6401)):
        plan = A.debug_packed_plan(m, k, n, bits, group)
        assert plan["tokens"] == 512 and plan["ranks"] == 2, plan
        packed, scale, zero, w = layer(A, n, k, bits, group, m)
        x = tokens(m, k, x_type, n)
        got = A.packed_matmul(x, packed, scale, zero, bits, torch.float32)
        assert torch.equal(got, (x.double() @ w.T).float()), (m, n)


def _operand(A, rows, k, fmt, seed):
    rng = np.random.default_rng(seed)
    code = rng.integers(0, 16, (rows, k)).astype(np.uint8)
    one, per = (127, 1) if fmt == "mxfp4" else (56, 8)       # bytes of the steps 1 and 2
    byte = (one + per * rng.integers(0, 2, (rows, k // mx.BLOCK[fmt]))).astype(np.uint8)
    q = A.MxTensor(torch.from_numpy(mx.pack_codes(code)).cuda(),
                   torch.from_numpy(mx.scale_tiles(byte)).cuda(), fmt)
    return q, torch.from_numpy(mx.values(code, byte, fmt)).cuda()


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("m,n,k", [(300, 10000, 96), (600, 10100, 320), (129, 19100, 288), (5000, 1000, 544),
                                   (257, 19400, 64)])
def test_mx_past_the_first_tile(A, fmt, m, n, k):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert m > 128 and -(-m // 256) * -(-n // 256) > sms // 2 and 144 * k < 2 ** 22
    a, av = _operand(A, m, k, fmt, m)
    b, bv = _operand(A, n, k, fmt, n)
    _into_room(lambda dt, out: A.mx_matmul(a, b, dt, out=out), av @ bv.T, m, n)


def test_pairs_in_two_graphs_at_once(A):
    """The same bits from two captured graphs replayed at once on other streams."""
    m, k, n = 1100, 384, 6600
    packed, scale, zero, _ = layer(A, n, k, 4, 128, 1)
    gen = torch.Generator(device="cuda").manual_seed(2)
    xs = [torch.randn((m, k), generator=gen, device="cuda").bfloat16() for _ in range(2)]
    want = [A.packed_matmul(x, packed, scale * 0.3, zero, 4) for x in xs]
    scale = scale * 0.3
    graphs = []
    for x in xs:
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            out = A.packed_matmul(x, packed, scale, zero, 4)
        graphs.append((graph, out, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(3):
        for graph, _, stream in graphs:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for (_, out, _), w in zip(graphs, want):
        assert torch.equal(out, w)
