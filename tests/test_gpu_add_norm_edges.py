"""Residual norm: what its ends leave. NaN in rows shorter than a lane's vector, and gradients in
place where a row's last vector begins in another wave's part."""
import pytest

import matrix_orthogonalising_optimizer_02_amd as muon
from test_gpu_add_norm import check_backward, decode, draw, dtype_of, log, torch_dev  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("value", ["nan", "inf"])
def test_padding_of_short_rows(torch_dev, name, value):  # noqa: F811
    """A row's NaN stays out of the codes behind its end (decode asserts zeros there)."""
    torch, dev = torch_dev
    for cols in (1, 2, 3, 4, 5, 7, 8, 9, 15, 130):
        x = draw(torch, dev, 670, cols, (6, cols), dtype_of(torch, name))
        x[2, cols // 2] = float(value)
        for w in (None, draw(torch, dev, 671, cols, (cols,), torch.float32, 0.3, 1.0)):
            _, y, y8, _ = muon.add_rms_norm_forward(x, None, w, codes=True)
            torch.cuda.synchronize()
            decode(y8)
            assert torch.equal(y8.dequantise().isnan(), y.isnan()) and bool(y[2].isnan().any())
