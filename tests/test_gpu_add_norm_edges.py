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


@pytest.mark.parametrize("name,rname", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f16", "f16")])
def test_in_place_across_waves(torch_dev, name, rname):  # noqa: F811
    """d over dh in rows whose last vector is the first of a wave (or of a lane's next vector) and
    reads what the wave before it writes."""
    torch, dev = torch_dev
    vec = 4 if name == "f32" else 8
    for i, waves in enumerate((1, 2, 3, 5, 8, 10, 13, 16)):
        for beside in (1, vec - 1):
            cols, rows = 64 * vec * waves + beside, 700
            dy, h, dh = (draw(torch, dev, 680 + i, j, (rows, cols), dtype_of(torch, t), 1.0 + j)
                         for j, t in enumerate((name, rname, rname)))
            w = draw(torch, dev, 680 + i, 3, (cols,), torch.float32, 0.3, 1.0)
            rstd = 0.5 + torch.rand(rows, device=dev)
            want = muon.add_rms_norm_backward(dy, dh, h, w, rstd)
            for _ in range(3):
                over = dh.clone()
                got = muon.add_rms_norm_backward(dy, over, h, w, rstd, out=over)
                assert torch.equal(over, want[1]) and torch.equal(got[0], want[0]) and torch.equal(got[2], want[2]), cols
        check_backward(torch, name, rname, dy, dh, h, w, rstd, 0.0, out=dh.clone())
        log(f"{name} residual {rname} {cols}")
