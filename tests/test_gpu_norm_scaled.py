"""The norms' call with neither norm, y nor gate: out = residual_scale x, one product in fp32 and one rounding, exact."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_norm import B, TYPES, _normal  # noqa: E402, F401


@pytest.mark.parametrize("R,d,typ,gate_rows", [(1, 8, 0, 0), (3, 8192, 2, 2), (700, 1032, 1, 7), (5000, 264, 0, 1), (650, 4104, 2, 0),
                                               (1300, 2048, 1, 1300), (640, 8192, 1, 0), (4000, 64, 2, 0)])
def test_a_scaled_stream(B, R, d, typ, gate_rows):
    x = _normal((R, d), 1, TYPES[typ], 2.0)
    for scale in (0.3, -1.0):
        cfg = B.make_norm(R, d, typ, gate_rows, scale)
        want = (x.float() * torch.tensor(cfg.residual_scale, device="cuda")).to(x.dtype)
        out, place = torch.full_like(x, 7), x.clone()
        B.moe_w4a16_norm(cfg, x, None, None, None, None, out, None)
        B.moe_w4a16_norm(cfg, place, None, None, None, None, place, None)
        assert torch.equal(out, want) and torch.equal(place, want)
        # y alone is the same without a factor
        out = torch.full_like(x, 7)
        B.moe_w4a16_norm(cfg, None, x, None, None, None, out, None)
        assert torch.equal(out, x)
