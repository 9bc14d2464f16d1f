"""How matmul8 cuts a product (the host-only matmul8_plan, which is the code that the launches
run): the cuts that the rule's comment names with their times, and the limits of every form."""
import ctypes

import pytest

import matrix_orthogonalising_optimizer_02_amd as muon
from matrix_orthogonalising_optimizer_02_amd import binding as B

torch = pytest.importorskip("torch")
INVALID, LARGE = B.MUON_ERR_INVALID_ARG, B.MUON_ERR_TOO_LARGE


@pytest.mark.parametrize("m,n,k,dtype,tile,parts", [
    (2048, 2048, 2048, "bfloat16", 128, 1), (4096, 4096, 4096, "bfloat16", 256, 1), (2048, 5120, 20480, "bfloat16", 256, 1),
    (512, 5120, 5120, "bfloat16", 128, 1), (256, 5120, 5120, "bfloat16", 128, 3), (128, 5120, 20480, "bfloat16", 128, 6),
    (2048, 2048, 65536, "float32", 256, 4), (8192, 20480, 5120, "bfloat16", 256, 1)])
def test_cuts_with_a_measured_time(m, n, k, dtype, tile, parts):
    plan = muon.matmul8_plan(m, n, k, getattr(torch, dtype))
    assert plan == dict(tile=tile, parts=parts, groups=0, stream=0, waves=0, share=0)
    need = muon.matmul8_workspace_bytes(m, n, k, getattr(torch, dtype))
    assert need == (parts * m * n * 4 if parts > 1 else 0)


@pytest.mark.parametrize("m,n,k,groups,stream,parts", [(1, 4096, 4096, 1, 0, 1), (8, 30720, 5120, 1, 1, 1), (16, 5120, 5120, 1, 1, 5),
                                                       (17, 5120, 5120, 2, 1, 5), (33, 5120, 5120, 4, 1, 5), (64, 16, 128, 4, 0, 1)])
def test_cuts_of_few_rows(m, n, k, groups, stream, parts):
    plan = muon.matmul8_plan(m, n, k)
    assert (plan["tile"], plan["groups"], plan["stream"], plan["parts"]) == (0, groups, stream, parts)
    assert muon.matmul8_workspace_bytes(m, n, k) == (parts * m * n * 4 if parts > 1 else 0)


def test_limits_of_the_forms():
    """What the kernels take for granted of a plan, over many sizes."""
    sizes = [1, 3, 16, 17, 33, 64, 65, 128, 200, 257, 1000, 2048, 5120, 8200, 20480, 60000]
    for m in sizes:
        for n in sizes:
            for k in (1, 128, 129, 512, 1000, 5120, 16384, 65536, 1 << 20):
                for products in (8, 16):
                    p = muon.matmul8_plan(m, n, k, products=products)
                    fours = -(-(-(-k // 128)) // 4)
                    assert 1 <= p["parts"] <= max(1, fours), (m, n, k, p)
                    if m > 64:
                        assert p["tile"] in (128, 256) and p["parts"] <= 16 and p["groups"] == 0
                        continue
                    assert p["tile"] == 0 and 16 * p["groups"] >= m and p["groups"] == (1 if m <= 16 else 2 if m <= 32 else 4)
                    if p["stream"]:  # a part's powers fit LDS: 128 steps
                        longest = max((i + 1) * fours // p["parts"] - i * fours // p["parts"] for i in range(p["parts"]))
                        assert 4 * longest <= 128 and p["waves"] == p["share"] == 0, (m, n, k, p)
                    else:  # whole teams, one launch, 512 threads
                        assert p["parts"] == 1 and 1 <= p["share"] <= p["waves"] <= 8 and p["waves"] % p["share"] == 0, (m, n, k, p)


def test_refusals():
    lib = B.load_library()
    out = (ctypes.c_int32 * 6)(*[7] * 6)
    for args, status in (((-1, 5, 5, 1, 0), INVALID), ((5, 5, 5, 4, 0), INVALID), ((5, 5, 5, 1, 9), INVALID),
                         ((5, 5, (1 << 22) + 1, 1, 0), LARGE), ((1 << 30, 1 << 30, 128, 1, 0), LARGE)):
        assert lib.matmul8_plan(*args, out) == status
    assert lib.matmul8_plan(5, 5, 5, 1, 0, None) == INVALID and list(out) == [7] * 6
    assert lib.matmul8_plan(0, 5, 5, 1, 0, out) == 0 and list(out) == [0] * 6
    with pytest.raises(B.MuonError):
        muon.matmul8_plan(5, 5, -1)
