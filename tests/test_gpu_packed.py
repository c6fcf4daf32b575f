"""The product with packed codes on the GPU against float64.

Exact inputs (activations small integers, scales powers of two) make every
partial sum a multiple of 1/4 below 2^22, which fp32 holds in any order: the
outputs have to be equal.  General inputs: k + d_in / group + 2 roundings of
partial sums no larger than S = sum s |c - z| |x|, each at most 2^-23 S
(truncation included), and one output rounding:
|err| <= (k + k / group + 2) 2^-23 S + eps / 2 |y|.
"""
import numpy as np
import pytest
import torch

from oracle import admmq_oracle as O
from oracle import mx

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def A():
    from post_weight_quantization_10_b200 import admmq
    admmq.lib()
    return admmq


def _layer(n, k, bits, group, seed, exact):
    rng = np.random.default_rng(seed)
    top = (1 << bits) - 1
    codes = rng.integers(0, top + 1, (n, k)).astype(np.uint8)
    zero = rng.integers(0, top + 1, (n, k // group)).astype(np.float32)
    if exact:
        scale = np.ldexp(1.0, rng.integers(-2, 1, zero.shape)).astype(np.float32)
    else:
        scale = np.exp(rng.uniform(-6, 2, zero.shape)).astype(np.float32)
    return codes, O.pack(codes, bits), scale, zero


def _cuda(words, scale, zero):
    return (torch.from_numpy(np.ascontiguousarray(words).view(np.int32)).cuda(),
            torch.from_numpy(scale).cuda(), torch.from_numpy(zero).cuda())


SHAPES = [(1, 1, 128), (1, 130, 256), (2, 33, 128), (3, 640, 4096), (8, 17, 384), (9, 100, 640),
          (16, 257, 512), (17, 64, 1152), (33, 384, 256), (64, 129, 1024), (65, 200, 128),
          (129, 260, 384), (300, 520, 640), (12, 515, 2048), (13, 64, 640)]


@pytest.mark.parametrize("xt", ["bf16", "fp16"])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_exact_inputs(A, m, n, k, xt):
    rng = np.random.default_rng(m + n + k)
    for bits in (2, 3, 4, 8):
        for group in (32, 64, 128):
            codes, words, scale, zero = _layer(n, k, bits, group, bits + group, True)
            # |c - z| <= 255, |x| <= 2, s <= 1: 510 k < 2^22
            x = rng.integers(-2, 3, (m, k)).astype(np.float32)
            w = mx.packed_weights(words, scale, zero, bits, k)
            want = torch.from_numpy((x.astype(np.float64) @ w.T).astype(np.float32))
            xd = torch.from_numpy(x).to(DT[xt]).cuda()
            for dt in DT.values():
                got = A.packed_matmul(xd, *_cuda(words, scale, zero), bits, dt).cpu()
                assert torch.equal(got, want.to(dt)), (bits, group, dt)


@pytest.mark.parametrize("bits", range(1, 9))
@pytest.mark.parametrize("group,k", [(32, 32), (32, 96), (64, 192), (128, 128), (128, 1280)])
def test_every_width_and_group(A, bits, group, k):
    rng = np.random.default_rng(bits)
    for m, n in ((1, 50), (12, 131), (90, 70)):
        codes, words, scale, zero = _layer(n, k, bits, group, m, True)
        x = rng.integers(-2, 3, (m, k)).astype(np.float32)
        want = x.astype(np.float64) @ mx.packed_weights(words, scale, zero, bits, k).T
        got = A.packed_matmul(torch.from_numpy(x).bfloat16().cuda(), *_cuda(words, scale, zero),
                              bits, torch.float32).cpu()
        assert torch.equal(got, torch.from_numpy(want.astype(np.float32))), (m, n)


@pytest.mark.parametrize("xt", ["bf16", "fp16"])
@pytest.mark.parametrize("m,n,k,bits,group", [(1, 300, 4096, 3, 128), (20, 200, 2048, 2, 64),
                                              (33, 100, 1056, 5, 32), (200, 300, 1024, 4, 128),
                                              (600, 700, 4096, 3, 128), (140, 150, 576, 8, 64),
                                              (1200, 400, 4096, 4, 128)])
def test_general_inputs(A, m, n, k, bits, group, xt):
    codes, words, scale, zero = _layer(n, k, bits, group, 7, False)
    rng = np.random.default_rng(8)
    x = torch.from_numpy((rng.standard_normal((m, k)) * np.exp(rng.uniform(-2, 2, (m, 1)))).astype(np.float32)).to(DT[xt])
    xd = x.double().numpy()
    w = mx.packed_weights(words, scale, zero, bits, k)
    want, size = xd @ w.T, np.abs(xd) @ np.abs(w).T
    slack = (k + k // group + 2) * 2.0 ** -23 * size
    for dt in DT.values():
        got = A.packed_matmul(x.cuda(), *_cuda(words, scale, zero), bits, dt).cpu().double().numpy()
        fine = np.isfinite(got)
        assert fine.all() or dt == torch.float16
        bound = slack + torch.finfo(dt).eps / 2 * np.abs(want) + torch.finfo(dt).tiny
        assert (np.abs(got - want)[fine] <= bound[fine]).all(), dt
        assert (np.abs(want)[~fine] + slack[~fine] >= 65504).all()


@pytest.mark.parametrize("xt", ["bf16", "fp16"])
@pytest.mark.parametrize("m,n,k,bits,group", [(1024, 128, 128, 4, 128), (1025, 300, 1280, 3, 128),
                                              (1030, 130, 96, 5, 32), (1300, 257, 192, 8, 64),
                                              (2000, 1, 160, 1, 32), (1024, 513, 320, 2, 64),
                                              (1111, 70, 256, 6, 128), (1024, 66, 64, 7, 32)])
def test_many_tokens(A, m, n, k, bits, group, xt):
    rng = np.random.default_rng(m + n)
    codes, words, scale, zero = _layer(n, k, bits, group, m, True)
    x = rng.integers(-2, 3, (m, k)).astype(np.float32)
    want = torch.from_numpy((x.astype(np.float64) @ mx.packed_weights(words, scale, zero, bits, k).T).astype(np.float32))
    xd, layer = torch.from_numpy(x).to(DT[xt]).cuda(), _cuda(words, scale, zero)
    for dt in DT.values():
        room = torch.full((m * n + 4096,), 3.0, dtype=dt, device="cuda")
        got = A.packed_matmul(xd, *layer, bits, dt, out=room[:m * n].view(m, n))
        assert torch.equal(got.cpu(), want.to(dt)), dt
        assert bool((room[m * n:] == 3.0).all())


def test_strided_activations_and_memory_behind(A):
    for m, n, k in ((5, 100, 256), (130, 140, 256)):
        codes, words, scale, zero = _layer(n, k, 3, 64, 1, True)
        rng = np.random.default_rng(2)
        big = torch.from_numpy(rng.integers(-2, 3, (m + 2, 2 * k)).astype(np.float32)).bfloat16().cuda()
        x = big[1:m + 1, 64:64 + k]
        layer = _cuda(words, scale, zero)
        room = torch.full((m * n + 4096,), 3.0, dtype=torch.bfloat16, device="cuda")
        got = A.packed_matmul(x, *layer, 3, out=room[:m * n].view(m, n))
        assert torch.equal(got, A.packed_matmul(x.contiguous(), *layer, 3))
        assert bool((room[m * n:] == 3.0).all())
        assert A.packed_matmul(x[:0], *layer, 3).shape == (0, n)
        with pytest.raises(A.AdmmqError):
            A.packed_matmul(big[:, 3:3 + k], *layer, 3)


@pytest.mark.parametrize("m", [2, 150])
def test_nonfinite_activations_stay_in_their_row(A, m):
    codes, words, scale, zero = _layer(70, 256, 4, 128, 3, True)
    x = torch.ones((m, 256), dtype=torch.bfloat16)
    x[1, 5] = float("nan")
    y = A.packed_matmul(x.cuda(), *_cuda(words, scale, zero), 4, torch.float32).cpu()
    assert torch.isnan(y[1]).all()
    keep = torch.arange(m) != 1
    want = x.double()[keep] @ torch.from_numpy(mx.packed_weights(words, scale, zero, 4, 256)).T
    assert torch.equal(y[keep].double(), want)


def test_refusals_on_the_device(A):
    codes, words, scale, zero = _layer(16, 128, 3, 64, 1, True)
    p, s, z = _cuda(words, scale, zero)
    x = torch.zeros((4, 128), dtype=torch.bfloat16, device="cuda")
    bad = [lambda: A.packed_matmul(x.float(), p, s, z, 3), lambda: A.packed_matmul(x, p, s, z, 4),
           lambda: A.packed_matmul(x[:, :64], p, s, z, 3), lambda: A.packed_matmul(x, p, s[:8], z, 3),
           lambda: A.packed_matmul(x, p, s, z[:, :1], 3), lambda: A.packed_matmul(x, p, s.cpu(), z, 3),
           lambda: A.packed_matmul(x, p.long(), s, z, 3),
           lambda: A.packed_matmul(x, p, s[:, :1].repeat(1, 8), z[:, :1].repeat(1, 8), 3),
           lambda: A.packed_matmul(x, p, s, z, 3, torch.float64),
           lambda: A.packed_matmul(x, p, s, z, 3, out=torch.empty((4, 16), device="cuda"))]
    for i, call in enumerate(bad):
        with pytest.raises(A.AdmmqError) as e:
            call()
        assert e.value.status == -1, i


def test_streams_graphs_and_repeats(A):
    for m in (1, 24, 160, 1500):
        codes, words, scale, zero = _layer(300, 512, 3, 128, m, False)
        layer = _cuda(words, scale, zero)
        gen = torch.Generator(device="cuda").manual_seed(m)
        x, x2 = (torch.randn((m, 512), generator=gen, device="cuda").bfloat16() for _ in range(2))
        want, want2 = A.packed_matmul(x, *layer, 3), A.packed_matmul(x2, *layer, 3)
        for _ in range(5):
            assert torch.equal(A.packed_matmul(x, *layer, 3), want)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        y = A.packed_matmul(x, *layer, 3, stream=side)
        side.synchronize()
        assert torch.equal(y, want)
        graphs = []
        for _ in range(2):
            buf, graph = x.clone(), torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(graph):
                out = A.packed_matmul(buf, *layer, 3)
            graphs.append((graph, buf, out))
        graphs[1][1].copy_(x2)
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        torch.cuda.synchronize()
        for _ in range(3):
            for (graph, _, _), s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(graphs[0][2], want) and torch.equal(graphs[1][2], want2)
