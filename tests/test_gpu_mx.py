"""Microscaled 4-bit formats on the GPU against the oracle.

Codes and scale bytes are whole numbers and have to be equal.  Dequantisation
is one fp32 multiplication and one rounding: equal bit for bit.  The product:
  - on operands whose every partial sum is a multiple of 1/4 below 2^22 the
    fp32 sum is exact in any order, so the fp32 output has to be equal and a
    16-bit output equal to the rounded value;
  - on general operands each of the k additions loses at most one unit in the
    last place of a partial sum no larger than S = sum |a b| (2^-23 S, which
    covers truncation), and the output one rounding, half of
    torch.finfo(dtype).eps: |err| <= k 2^-23 S + eps / 2 |y|.
"""
import numpy as np
import pytest
import torch

from oracle import mx

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def A():
    from post_weight_quantization_10_b200 import admmq
    admmq.lib()
    return admmq


def _matrix(rows, k, seed, dt=torch.float32, border_t=None):
    """Rows of very different sizes, zero rows and blocks, elements on borders."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, k)) * np.exp(rng.uniform(-6, 6, (rows, 1)))
    x[:, ::7] = np.round(x[:, ::7] * 4) / 4
    if rows > 3:
        x[rows // 2] = 0
    x[0, :min(k, 32)] = 0
    return torch.from_numpy(x.astype(np.float32)).to(dt)


def _g(x):
    return np.float32(float(x.float().abs().max()) / (448 * 6))


def _dev_g(g):
    return None if g is None else torch.full((1,), float(g), dtype=torch.float32, device="cuda")


def _check_codes(q, x, fmt, g):
    code, byte = mx.quantize(x.float().numpy(), fmt, g)
    got = q.codes.cpu().numpy()
    np.testing.assert_array_equal(q.scale.cpu().numpy(), mx.scale_tiles(byte))
    np.testing.assert_array_equal(got, mx.pack_codes(code))
    return code, byte


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("rows,k", [(1, 32), (1, 4096), (3, 96), (127, 160), (129, 288), (300, 544)])
def test_quantize_and_dequantize_equal_the_oracle(A, fmt, dtype, rows, k):
    x = _matrix(rows, k, rows + k, DT[dtype])
    g = _g(x) if fmt == "nvfp4" else None
    q = A.mx_quantize(x.cuda(), fmt, _dev_g(g))
    code, byte = _check_codes(q, x, fmt, g)
    v = mx.values(code, byte, fmt, g)
    for out in DT.values():
        got = A.mx_dequantize(q, out).cpu()
        want = torch.from_numpy(v.astype(np.float32)).to(out)
        assert torch.equal(got, want), out


def test_quantize_borders_and_extremes(A):
    """Elements on and one unit next to every rounding border, scales on theirs;
    subnormal, largest and non-finite values."""
    rng = np.random.default_rng(5)
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    for fmt, g in (("mxfp4", None), ("nvfp4", np.float32(0.0137)), ("nvfp4", np.float32(2.0 ** -100)),
                   ("nvfp4", np.float32(3e-42)), ("nvfp4", None)):
        b = mx.BLOCK[fmt]
        x = np.zeros((512, 64), np.float32)
        base = np.exp(rng.uniform(-9, 9, (512, 64 // b))) * (1.0 if g is None else 1e3 * float(g))
        x[:, ::b] = (6 * base).astype(np.float32)
        if fmt == "nvfp4":   # scales on the borders between e4m3 values
            e = (mx.E4M3[1:] + mx.E4M3[:-1])[rng.integers(0, 125, 200)] / 2 * 6 * (1.0 if g is None else float(g))
            e = np.float32(e)
            x[:200, 0] = np.where(rng.random(200) < 0.5, e, np.nextafter(e, np.float32(0)))
        _, byte = mx.quantize(x, fmt, g)
        t = np.repeat(mx.step(byte, fmt, g), b, axis=1)
        v = (rng.choice(mids, x.shape) * t).astype(np.float32)
        v = np.where(rng.random(x.shape) < 0.3, np.nextafter(v, np.float32(3e38)), v)
        v = np.where(rng.random(x.shape) < 0.3, np.nextafter(v, np.float32(0)), v)
        v *= rng.choice([1, -1], x.shape)
        keep = np.arange(64) % b == 0
        x = np.where(keep[None, :], x, v).astype(np.float32)
        x = np.where(np.abs(x) > np.abs(np.repeat(x[:, ::b], b, axis=1)), 0, x).astype(np.float32)
        xt = torch.from_numpy(x)
        _check_codes(A.mx_quantize(xt.cuda(), fmt, _dev_g(g)), xt, fmt, g)
    x = np.zeros((6, 64), np.float32)
    x[0, 1], x[1, 40], x[2, 5] = np.nan, np.inf, -np.inf
    x[3, :] = 1e-42
    x[4, :] = 3.4e38
    x[5, ::2] = np.float32(2.0 ** -126)
    xt = torch.from_numpy(x)
    for fmt in mx.BLOCK:
        q = A.mx_quantize(xt.cuda(), fmt)
        code, byte = _check_codes(q, xt, fmt, None)
        got = A.mx_dequantize(q, torch.float32).cpu().numpy()
        np.testing.assert_array_equal(got, mx.values(code, byte, fmt).astype(np.float32))


def test_quantize_strided_rows_and_out(A):
    big = _matrix(70, 256, 9, torch.bfloat16).cuda()
    x = big[3:40, 64:224]                     # rows 256 apart, first element 16-byte aligned
    q = A.mx_quantize(x)
    _check_codes(q, x.cpu(), "mxfp4", None)
    with pytest.raises(A.AdmmqError):         # rows that do not start on 16 bytes
        A.mx_quantize(big[:, 3:163])
    with pytest.raises(A.AdmmqError):         # columns apart
        A.mx_quantize(big.t()[:64, :64])
    out = torch.full((37, 160), 7.0, dtype=torch.float32, device="cuda")
    assert A.mx_dequantize(q, torch.float32, out=out) is out
    assert torch.equal(out, A.mx_dequantize(q, torch.float32))
    empty = A.mx_quantize(big[:0])
    assert empty.rows == 0 and A.mx_dequantize(empty).shape == (0, 256)


# ----------------------------------------------------------------- product


def _exact_operand(rows, k, fmt, seed, top=2):
    """Random codes with steps 1, 2, ...: elements are multiples of 1/2."""
    rng = np.random.default_rng(seed)
    code = rng.integers(0, 16, (rows, k)).astype(np.uint8)
    one = 127 if fmt == "mxfp4" else 56            # byte of the step 1.0
    per = 1 if fmt == "mxfp4" else 8               # byte distance of the step 2.0
    byte = (one + per * rng.integers(0, top, (rows, k // mx.BLOCK[fmt]))).astype(np.uint8)
    return code, byte


def _mx_tensor(A, code, byte, fmt, g=None):
    return A.MxTensor(torch.from_numpy(mx.pack_codes(code)).cuda(),
                      torch.from_numpy(mx.scale_tiles(byte)).cuda(), fmt, _dev_g(g))


SHAPES = [(1, 1, 32), (1, 130, 96), (2, 64, 4096), (7, 257, 160), (16, 128, 256), (17, 640, 288),
          (33, 100, 1024), (64, 129, 544), (65, 384, 512), (130, 33, 2080), (300, 520, 320),
          (257, 1, 64), (5, 4100, 128)]


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product_exact_operands(A, fmt, m, n, k):
    a, sa = _exact_operand(m, k, fmt, m + n)
    b, sb = _exact_operand(n, k, fmt, k + n)
    want = mx.values(a, sa, fmt) @ mx.values(b, sb, fmt).T
    # 12 x 12 x k < 2^22: every partial sum is a multiple of 1/4 that fp32 holds
    assert np.abs(want).max() < 2 ** 22 and 144 * k < 2 ** 22
    qa, qb = _mx_tensor(A, a, sa, fmt), _mx_tensor(A, b, sb, fmt)
    for dt in DT.values():
        got = A.mx_matmul(qa, qb, dt).cpu()
        assert torch.equal(got, torch.from_numpy(want.astype(np.float32)).to(dt)), dt


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("m,n,k", [(1, 300, 4096), (31, 200, 2048), (200, 300, 1056), (600, 700, 4096)])
def test_product_general_operands(A, fmt, m, n, k):
    x, w = _matrix(m, k, 1), _matrix(n, k, 2)
    gx, gw = (_g(x), _g(w)) if fmt == "nvfp4" else (None, None)
    qx = A.mx_quantize(x.cuda(), fmt, _dev_g(gx))
    qw = A.mx_quantize(w.cuda(), fmt, _dev_g(gw))
    a = mx.values(*mx.quantize(x.numpy(), fmt, gx), fmt, gx)
    b = mx.values(*mx.quantize(w.numpy(), fmt, gw), fmt, gw)
    want, size = a @ b.T, np.abs(a) @ np.abs(b).T
    # nvfp4: the library multiplies by g_a g_b once, the oracle's steps carry
    # one fp32 rounding each, two per product: 2^-23 S more
    slack = (k + 2) * 2.0 ** -23 * size
    for dt in DT.values():
        got = A.mx_matmul(qx, qw, dt).cpu().double().numpy()
        w16 = np.clip(want, -65504, 65504) if dt == torch.float16 else want
        fine = np.isfinite(got)
        assert fine.all() or dt == torch.float16
        bound = slack + torch.finfo(dt).eps / 2 * np.abs(w16) + torch.finfo(dt).tiny
        assert (np.abs(got - w16)[fine] <= bound[fine]).all(), dt
        assert (np.abs(want)[~fine] + slack[~fine] >= 65504).all()


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("m,n", [(3, 200), (150, 200)])
def test_product_nan_blocks_stay_in_their_row_and_column(A, fmt, m, n):
    k = 512
    a, sa = _exact_operand(m, k, fmt, 1)
    b, sb = _exact_operand(n, k, fmt, 2)
    nan = 255 if fmt == "mxfp4" else 127
    sa[2, 3] = nan
    sb[7, 1] = sb[199, 0] = nan
    got = A.mx_matmul(_mx_tensor(A, a, sa, fmt), _mx_tensor(A, b, sb, fmt), torch.float32).cpu().numpy()
    want = mx.values(a, sa, fmt) @ mx.values(b, sb, fmt).T
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
    np.testing.assert_array_equal(got[np.isfinite(want)], want[np.isfinite(want)])


def test_product_writes_its_rows_only(A):
    """The memory behind the output's last row stays as it was."""
    for m, n in ((5, 100), (70, 130)):
        a, sa = _exact_operand(m, 256, "mxfp4", 1)
        b, sb = _exact_operand(n, 256, "mxfp4", 2)
        room = torch.full((m * n + 4096,), 3.0, dtype=torch.bfloat16, device="cuda")
        out = room[:m * n].view(m, n)
        got = A.mx_matmul(_mx_tensor(A, a, sa, "mxfp4"), _mx_tensor(A, b, sb, "mxfp4"), out=out)
        assert got is out and bool((room[m * n:] == 3.0).all())
        assert A.mx_matmul(_mx_tensor(A, a[:0], sa[:0], "mxfp4"),
                           _mx_tensor(A, b, sb, "mxfp4")).shape == (0, n)


def test_linear_is_quantize_then_product(A):
    for fmt in mx.BLOCK:
        for m in (1, 3, 9, 16, 17, 40, 200):
            x = _matrix(m, 320, m, torch.bfloat16).cuda()
            w = _matrix(210, 320, 3).cuda()
            g = _dev_g(_g(x)) if fmt == "nvfp4" else None
            qw = A.mx_quantize(w, fmt)
            y = A.mx_linear(x, qw, tensor_scale=g)
            assert y.dtype == torch.bfloat16
            assert torch.equal(y, A.mx_matmul(A.mx_quantize(x, fmt, g), qw, torch.bfloat16))


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("m,n,k", [(1, 19300, 2080), (9, 19300, 2048), (5, 300, 12288),
                                   (100, 19300, 2048), (90, 129, 12320), (400, 3000, 4128)])
def test_linear_with_more_stages_than_fit(A, fmt, m, n, k):
    """Many tiles or a long reduction: the stages' ring goes round, activations of
    few tokens are quantised by a launch of their own.  Against float64 on the
    dequantised matrices (exact in fp32), and equal to the product's own bits."""
    gen = torch.Generator(device="cuda").manual_seed(m + n)
    x = torch.randn((m, k), generator=gen, device="cuda").bfloat16()
    w = (torch.randn((n, k), generator=gen, device="cuda") * 0.02).bfloat16()
    g = _dev_g(_g(x)) if fmt == "nvfp4" else None
    qw, qx = A.mx_quantize(w, fmt), A.mx_quantize(x, fmt, g)
    y = A.mx_linear(x, qw, torch.float32, tensor_scale=g)
    assert torch.equal(y, A.mx_matmul(qx, qw, torch.float32))
    a, b = A.mx_dequantize(qx, torch.float32).double(), A.mx_dequantize(qw, torch.float32).double()
    bound = (k + 2) * 2.0 ** -23 * (a.abs() @ b.abs().T)
    assert bool(((y.double() - a @ b.T).abs() <= bound).all())


def test_refusals_on_the_device(A):
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    g = torch.ones(1, device="cuda")
    q, v = A.mx_quantize(x), A.mx_quantize(x, "nvfp4", g)
    bad = [lambda: A.mx_quantize(x, "mxfp4", g), lambda: A.mx_quantize(x, "fp4"),
           lambda: A.mx_quantize(x[:, :48]), lambda: A.mx_quantize(x.int()),
           lambda: A.mx_quantize(x, "nvfp4", g.double()), lambda: A.mx_quantize(x, "nvfp4", g.cpu()),
           lambda: A.mx_matmul(q, v), lambda: A.mx_matmul(q, A.mx_quantize(x[:, :32])),
           lambda: A.mx_matmul(q, A.mx_quantize(x[:0])), lambda: A.mx_matmul(q, q, torch.int32),
           lambda: A.mx_matmul(q, q, out=torch.empty((4, 5), dtype=torch.bfloat16, device="cuda")),
           lambda: A.MxTensor(q.codes, q.scale[:-1], "mxfp4"),
           lambda: A.MxTensor(q.codes, q.scale, "mxfp4", g),
           lambda: A.mx_dequantize(q, torch.float64)]
    for i, call in enumerate(bad):
        with pytest.raises(A.AdmmqError) as e:
            call()
        assert e.value.status == -1, i


# ------------------------------------------------- streams, graphs, repeats


def test_streams_graphs_and_repeats(A):
    """The same bits on another stream, in a captured graph replayed on new
    inputs, with two graphs replayed at once, and on every repeat."""
    for m in (1, 24, 160):
        x = _matrix(m, 512, m, torch.bfloat16).cuda()
        x2 = _matrix(m, 512, m + 1, torch.bfloat16).cuda()
        w = A.mx_quantize(_matrix(300, 512, 4).cuda())
        want, want2 = A.mx_linear(x, w), A.mx_linear(x2, w)
        for _ in range(5):
            assert torch.equal(A.mx_linear(x, w), want)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        y = A.mx_linear(x, w, stream=side)
        side.synchronize()
        assert torch.equal(y, want)
        graphs = []
        torch.cuda.synchronize()
        for _ in range(2):
            buf, graph = x.clone(), torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(graph):
                out = A.mx_linear(buf, w)
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


@pytest.mark.parametrize("tokens", [8, 128, 256])
@pytest.mark.parametrize("element,byte,g", [(6.0, 0x7E, 2.0**-77), (0.5, 0x01, 2.0**66)])
def test_tensor_scales_whose_product_leaves_the_range(A, tokens, element, byte, g):
    """The output is representable, the product of the tensor scales is not:
    a^2 k with a = element x block scale, a whole multiple of a power of two
    (2688^2 = 441 x 2^14), exact in fp32, times two scales of 2^-77 and 2^-78
    (2^-155) or 2^66 each (2^132)."""
    k, n = 1024, 256
    step = 448.0 if byte == 0x7E else 2.0**-9
    ga, gb = (2.0**-77, 2.0**-78) if g < 1 else (g, g)
    code = 7 if element == 6.0 else 1

    def tensor(rows, gg):
        tiles = torch.full((-(-rows // 128) * (k // 64) * 512,), byte, dtype=torch.uint8, device="cuda")
        codes = torch.full((rows, k // 2), 17 * code, dtype=torch.uint8, device="cuda")
        return A.MxTensor(codes, tiles, "nvfp4", _dev_g(gg))

    want = (element * step) ** 2 * k * ga * gb
    assert float(np.float32(want)) == want
    w = tensor(n, gb)
    if tokens == 8:
        # quantised on the way in: largest element 6, block scale 448 or 2^-9
        # (an element of 6 keeps that block scale; the others are 1/2)
        x = torch.full((tokens, k), element * step * ga, dtype=torch.float32, device="cuda")
        if byte == 0x01:
            x[:, ::16] = 6 * step * ga
            want *= (1 + 11 / 16)
        y = A.mx_linear(x, w, torch.float32, tensor_scale=_dev_g(ga))
    else:
        y = A.mx_matmul(tensor(tokens, ga), w, torch.float32)
    assert y.shape == (tokens, n)
    assert torch.equal(y.cpu(), torch.full((tokens, n), want, dtype=torch.float32))
