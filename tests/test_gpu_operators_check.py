"""A bounded wait of an operator's kernel that gives up is reported to the
host: once, from every translation unit and stream, and calls go on after it."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def A():
    from post_weight_quantization_10_b200 import admmq
    admmq.lib()
    return admmq


@pytest.mark.parametrize("unit,side", [(0, False), (1, True), (2, False), (3, True)])
def test_a_wait_that_gives_up_is_reported_once(A, unit, side):
    x = torch.randn((20, 256), device="cuda").bfloat16()
    w = A.mx_quantize(torch.randn((128, 256), device="cuda"))
    want = A.mx_linear(x, w)
    A.operators_check()
    stream = torch.cuda.Stream() if side else None
    A.debug_give_up(unit, stream=stream)
    with pytest.raises(A.AdmmqError) as e:
        A.operators_check("cuda", stream=stream)
    assert e.value.status == A.ERR_TIMEOUT
    A.operators_check(device=0)
    assert torch.equal(A.mx_linear(x, w), want)
    A.operators_check(stream=torch.cuda.Stream())


def test_units(A):
    with pytest.raises(A.AdmmqError):
        A.debug_give_up(4)
