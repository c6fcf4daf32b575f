"""The quantised-weight operators at work together on one layer: solve it,
pack it, and run the calibration activations through what was packed and
through the 4-bit formats."""
import numpy as np
import pytest
import torch

from oracle import admmq_oracle as O
from oracle import mx
from post_weight_quantization_10_b200 import workloads

pytestmark = pytest.mark.gpu


def test_packed_layer_reproduces_the_objective():
    """1/2 ||X (D - W)^T||^2 + lambda/2 ||D - W||^2 is the objective that the
    solve reports; the outputs X D^T come from the packed codes.  The sum of
    squares inherits the fp32 outputs' error: a relative 1e-3 on a difference
    of outputs whose size is 1/30 of theirs at the least."""
    from post_weight_quantization_10_b200 import admmq as A
    p = workloads.scaled(workloads.PRESETS["q_proj"], 2048, 256, 192, group=64, iters=40, rank=16)
    X = workloads.make_activations(p, seed=1, device="cuda")
    W = workloads.make_weights(p, seed=1, device="cuda", dtype=torch.float32)
    s = A.solve_layer(X, W, A.Params(bits=3, group=64, iters=40))
    packed = A.pack(s.codes, 3)
    y = A.packed_matmul(X, packed, s.scale, s.zero, 3, torch.float32)
    G = O.gram(X.float().cpu().numpy())
    lam = p.lambda_rel * np.trace(G) / 256
    Wd = W.double()
    D = torch.from_numpy(mx.packed_weights(packed.cpu().numpy().view(np.uint32), s.scale.cpu().numpy(),
                                           s.zero.cpu().numpy(), 3, 256)).cuda()
    out = X.double() @ Wd.T
    obj = 0.5 * float((y.double() - out).square().sum()) + 0.5 * lam * float((D - Wd).square().sum())
    assert float((y.double() - out).norm() / out.norm()) > 1 / 30
    assert obj == pytest.approx(float(s.objective.cpu()), rel=1e-3)
    # one token at a time gives what the batch gives, up to the order of fp32 sums
    one = torch.cat([A.packed_matmul(X[i:i + 1], packed, s.scale, s.zero, 3, torch.float32)
                     for i in range(4)])
    size = X[:4].double().abs() @ D.abs().T
    assert bool(((one - y[:4]).double().abs() <= 2 * (256 + 6) * 2.0 ** -23 * size).all())


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_four_bit_layer_end_to_end(fmt):
    """Weights and activations quantised, multiplied, against the product of the
    dequantised matrices in float64; and the error against the unquantised
    layer is the one that the formats' rounding explains (below the sum of the
    two matrices' own relative errors and their product)."""
    from post_weight_quantization_10_b200 import admmq as A
    p = workloads.scaled(workloads.PRESETS["q_proj"], 300, 512, 260, rank=16)
    X = workloads.make_activations(p, seed=2, device="cuda")
    W = workloads.make_weights(p, seed=2, device="cuda")
    g = None
    if fmt == "nvfp4":
        g = (X.float().abs().amax() / (448 * 6)).reshape(1)
    qw = A.mx_quantize(W, fmt)
    y = A.mx_linear(X, qw, torch.float32, tensor_scale=g).double()
    qx = A.mx_quantize(X, fmt, g)
    xd, wd = A.mx_dequantize(qx, torch.float32).double(), A.mx_dequantize(qw, torch.float32).double()
    size = xd.abs() @ wd.abs().T
    assert bool(((y - xd @ wd.T).abs() <= (512 + 2) * 2.0 ** -23 * size).all())
    ex = torch.linalg.matrix_norm((xd - X.double())) * torch.linalg.matrix_norm(wd, 2)
    ew = torch.linalg.matrix_norm((wd - W.double())) * torch.linalg.matrix_norm(X.double(), 2)
    assert float((y - X.double() @ W.double().T).norm()) <= float(ex + ew) * 1.001
