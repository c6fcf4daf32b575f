"""Argument checks of the quantised-weight operators: every call below is
refused before the device is touched (the pointers are never dereferenced)."""
import ctypes

import pytest
import torch

INVALID = -1


@pytest.fixture(scope="module")
def lib():
    from post_weight_quantization_10_b200 import admmq, build
    build.build()
    return admmq.lib()


def _p(i):
    return ctypes.c_void_p(0x10000 * (i + 1))


def _refused(f, good, changes):
    for at, bad in changes:
        args = list(good)
        args[at] = bad
        assert f(*args) == INVALID, (at, bad)


def test_scale_bytes(lib):
    f = lib.admmq_mx_scale_bytes
    assert f(1, 32, 0) == 512 and f(1, 32, 1) == 512
    assert f(129, 160, 0) == 2 * 2 * 512 and f(128, 160, 1) == 3 * 512
    assert f(0, 64, 0) == 0 and f(4, 48, 0) == 0 and f(4, 64, 2) == 0 and f(-1, 64, 0) == 0


def test_quantize_and_dequantize_refusals(lib):
    # x dtype rows k ld fmt tensor_scale codes scale stream
    good = [_p(0), 1, 8, 64, 64, 1, _p(1), _p(2), _p(3), None]
    off = ctypes.c_void_p(0x10008)
    _refused(lib.admmq_mx_quantize, good,
             [(0, None), (0, off), (1, 3), (1, -1), (2, -1), (2, 1 << 31), (3, 48), (3, 0),
              (4, 63), (4, 68), (5, 2), (5, 0), (6, ctypes.c_void_p(2)), (7, None), (7, off),
              (8, None), (8, off)])
    # codes scale rows k fmt tensor_scale out dtype ld stream
    good = [_p(0), _p(1), 8, 64, 1, _p(2), _p(3), 1, 64, None]
    _refused(lib.admmq_mx_dequantize, good,
             [(0, None), (0, off), (1, None), (1, off), (2, -1), (3, 33), (4, -1), (4, 0),
              (5, ctypes.c_void_p(2)), (6, None), (6, off), (7, 3), (8, 32), (8, 65)])


def test_matmul_refusals(lib):
    # a: codes scale g, b: codes scale g, m n k fmt out dtype stream
    good = [_p(0), _p(1), _p(2), _p(3), _p(4), _p(5), 8, 16, 64, 1, _p(6), 1, None]
    off = ctypes.c_void_p(0x10008)
    _refused(lib.admmq_mx_matmul, good,
             [(0, None), (1, None), (3, None), (4, None), (10, None), (0, off), (1, off), (3, off),
              (4, off), (10, off), (2, ctypes.c_void_p(2)), (6, -1), (7, 0), (8, 40), (9, 3),
              (9, 0), (11, 3)])
    # no rows: nothing to do, whatever the pointers
    assert lib.admmq_mx_matmul(None, None, None, None, None, None, 0, 16, 64, 0, None, 1, None) == 0
    assert lib.admmq_mx_quantize(None, 1, 0, 64, 64, 0, None, None, None, None) == 0


def test_packed_refusals(lib):
    # x dtype m ldx packed scale zero d_in d_out bits group out dtype stream
    good = [_p(0), 1, 8, 256, _p(1), _p(2), _p(3), 256, 16, 3, 128, _p(4), 1, None]
    off = ctypes.c_void_p(0x10008)
    _refused(lib.admmq_packed_matmul, good,
             [(0, None), (0, off), (1, 0), (1, 3), (2, -1), (3, 248), (3, 260), (4, None), (4, off),
              (5, None), (6, None), (5, ctypes.c_void_p(2)), (7, 40), (7, 320), (8, 0), (9, 0),
              (9, 9), (10, 48), (11, None), (11, off), (12, 5)])
    assert lib.admmq_packed_matmul(None, 1, 0, 256, None, None, None, 256, 16, 3, 128, None, 1,
                                   None) == 0


def test_binding_refuses_host_tensors():
    from post_weight_quantization_10_b200 import admmq as A
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    for call in (lambda: A.mx_quantize(x),
                 lambda: A.MxTensor(torch.zeros((4, 32), dtype=torch.uint8),
                                    torch.zeros(512, dtype=torch.uint8)),
                 lambda: A.packed_matmul(x, torch.zeros((8, 6), dtype=torch.int32),
                                         torch.ones((8, 1)), torch.ones((8, 1)), 3)):
        with pytest.raises(A.AdmmqError) as e:
            call()
        assert e.value.status == INVALID


def test_linear_refusals(lib):
    # x dtype m ldx gx, w: codes scale g, n k fmt out dtype ws ws_bytes stream
    good = [_p(0), 1, 40, 64, _p(1), _p(2), _p(3), _p(4), 16, 64, 1, _p(5), 1, _p(6), 1 << 30, None]
    off = ctypes.c_void_p(0x10008)
    _refused(lib.admmq_mx_linear, good,
             [(0, None), (0, off), (1, 3), (2, -1), (3, 32), (3, 68), (4, ctypes.c_void_p(2)),
              (5, None), (5, off), (6, None), (6, off), (7, ctypes.c_void_p(2)), (8, 0), (9, 40),
              (10, 2), (10, 0), (11, None), (11, off), (12, 5), (13, None),
              (13, ctypes.c_void_p(0x10080))])
    bad = list(good)
    bad[14] = 100
    assert lib.admmq_mx_linear(*bad) == -7
    f = lib.admmq_mx_linear_workspace_bytes
    assert f(0, 16, 64, 0) == 0 and f(40, 16, 48, 0) == 0 and f(40, 0, 64, 0) == 0
    assert f(40, 16, 64, 0) == (40 * 32 + 255) // 256 * 256 + 512
