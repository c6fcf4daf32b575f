"""How the packed product lays a call out, checked on the host: every copy of
the few-token kernel has to start on its size and to stay inside its row."""
import ctypes

import pytest

SMS = 148


@pytest.fixture(scope="module")
def A():
    from post_weight_quantization_10_b200 import admmq, build
    build.build()
    admmq.lib()
    return admmq


def _scale_copies(plan, k, group):
    """(first group, groups) of every stage's copy of a row's scales."""
    per = 128 // group
    spans, total = -(-k // 128), k // group
    for rank in range(plan["ranks"]):
        for sp in range(rank * plan["range"], min((rank + 1) * plan["range"], spans), plan["stage"]):
            yield sp * per, min(plan["groups"], total - sp * per)


D_IN = sorted({128 * i for i in range(1, 41)} | {96, 160, 224, 416, 2080, 5504, 6144, 6912, 7168, 8192,
              8704, 9728, 10240, 11008, 12288, 13824, 14336, 17408, 18944, 25600, 27648, 28672})
D_OUT = [1, 16, 34, 130, 768, 1024, 2048, 2560, 3584, 4096, 4864, 5120, 6144, 8192, 14336, 25600]


@pytest.mark.parametrize("group", [32, 64, 128])
def test_scales_in_16_byte_pieces_start_on_16_bytes_and_stay_in_their_row(A, group):
    vec = split = 0
    for m in range(1, 13):
        for k in D_IN:
            if k % group:
                continue
            for n in D_OUT:
                for bits in (1, 3, 4, 8):
                    plan = A.debug_packed_plan(m, k, n, bits, group, SMS)
                    assert plan["tokens"] in (8, 16)
                    if not plan["vec_scales"]:
                        continue
                    vec += 1
                    split += plan["ranks"] > 1
                    assert (k // group) % 4 == 0      # rows apart by whole pieces
                    for g0, groups in _scale_copies(plan, k, group):
                        assert g0 % 4 == 0 and groups % 4 == 0, (m, k, n, bits, plan)
    assert vec and split      # both kinds were met


def test_every_column_has_one_rank(A):
    for m in (1, 2, 8, 12):
        for k in D_IN:
            for n in D_OUT:
                plan = A.debug_packed_plan(m, k, n, 4, 32, SMS)
                assert plan["ranks"] * plan["range"] * 128 >= k
                assert plan["groups"] == plan["stage"] * 4
                assert plan["tiles"] * plan["rows"] >= n


def test_the_longest_rows(A):
    """Rows up to 2^30 columns: their activations do not fit the shared memory,
    every position is a 32-bit number.  Longer ones are refused."""
    for m in (1, 8, 12):
        plan = A.debug_packed_plan(m, 1 << 30, 16, 1, 32, SMS)
        assert plan["staged"] == 1 and plan["ranks"] * plan["range"] * 128 >= 1 << 30
    assert A.debug_packed_plan(13, 1 << 30, 16, 1, 32, SMS)["range"] * 8 * 128 == 1 << 30
    p = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(5)]
    for k in ((1 << 30) + 32, (1 << 31) - 64):
        for m in (1, 40):
            assert A.lib().admmq_packed_matmul(p[0], 1, m, k, p[1], p[2], p[3], k, 16, 1, 32, p[4],
                                               1, None) == A.ERR_INVALID_ARG
