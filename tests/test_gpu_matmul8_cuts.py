"""matmul8 in the cuts that few sizes take, each asserted to be taken: parts of k in 256-tiles,
and few rows with several groups of 16 columns a block, with and without waves that share them."""
import pytest

import matrix_orthogonalising_optimizer_02_amd as muon
from test_gpu_blocks8 import check_product, draw, dtype_of, log, operand, torch_dev  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name,products", [("f32", 16), ("f32", 8), ("bf16", 8), ("f16", 16)])
@pytest.mark.parametrize("m,n,k,parts", [(2048, 2048, 20480, 4), (1537, 1300, 20000, 6), (1900, 2047, 33000, 4)])
def test_parts_of_256_tiles(torch_dev, m, n, k, parts, name, products):  # noqa: F811
    """Whole and ragged, into new memory and added to a view whose surroundings stay."""
    torch, dev = torch_dev
    plan = muon.matmul8_plan(m, n, k, dtype_of(torch, name), products)
    assert (plan["tile"], plan["parts"]) == (256, parts)
    a, b = operand(torch, dev, 900, m, k), operand(torch, dev, 901, n, k, m == 1537, 0.02)
    one = check_product(torch, a, b, name, products, (m, n, k, name, products))
    assert torch.equal(one, muon.matmul8(a, b, dtype=dtype_of(torch, name), products=products))
    buf = draw(torch, dev, 902, (m + 2, n + 7), dtype_of(torch, name), 0.1)
    kept, out = buf.clone(), buf[1:-1, 3:-4]
    check_product(torch, a, b, name, products, (m, n, k, name, "accumulate"), old=out.clone(), out=out, accumulate=True)
    buf[1:-1, 3:-4], kept[1:-1, 3:-4] = 0, 0
    assert torch.equal(buf, kept)


@pytest.mark.parametrize("name,products", [("bf16", 8), ("f32", 16)])
@pytest.mark.parametrize("m,n,k,waves,share", [(1, 8200, 250, 2, 1), (20, 8200, 250, 2, 1), (50, 8200, 250, 2, 1), (1, 16390, 250, 4, 1),
                                               (20, 16390, 250, 4, 1), (50, 16390, 250, 4, 1), (3, 65551, 250, 8, 1), (20, 11201, 509, 4, 2),
                                               (50, 9001, 509, 4, 2), (64, 8192, 1000, 8, 4), (9, 11200, 1300, 6, 3)])
def test_few_rows_and_groups_of_columns(torch_dev, m, n, k, waves, share, name, products):  # noqa: F811
    torch, dev = torch_dev
    plan = muon.matmul8_plan(m, n, k, dtype_of(torch, name), products)
    assert (plan["tile"], plan["stream"], plan["waves"], plan["share"]) == (0, 0, waves, share)
    a, b = operand(torch, dev, 910, m, k), operand(torch, dev, 911, n, k, k == 509, 0.02)
    check_product(torch, a, b, name, products, (m, n, k, name))
    out = draw(torch, dev, 912, (m, n), dtype_of(torch, name), 0.1)
    check_product(torch, a, b, name, products, (m, n, k, name, "accumulate"), old=out.clone(), out=out, accumulate=True)
    log(f"{name} products {products} [{m}, {k}] x [{n}, {k}]")
