"""Clipping where max_norm / norm is below fp32's normal range (2^-126).

Bounds: those of test_gpu_clip, 11 v and the rounding to the type (half of its smallest step where the result is
that small); a factor in two parts has one rounding more, v = 2^-24, and a step of the product's first part that is
subnormal is 2^-150 times 2^-126: nothing.
"""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_clip import B, B16, F32, HALF, SMALL, V, _clip, _norm  # noqa: E402, F401


@pytest.mark.parametrize("dtype", [F32, B16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("sizes", [[5, 4097], [300001, 7, 40000], [33] * 700], ids=["few", "many", "long list"])
@pytest.mark.parametrize("scale,max_norm", [(1e35, 1e-3), (1e35, 1e-6), (3e34, 1.0), (1e30, 1e-30), (1e10, 2.0 ** -140), (1e-30, 0.0),
                                            (1e35, 1e3)])
def test_a_factor_below_the_normal_range(B, dtype, sizes, scale, max_norm):
    g = torch.Generator(device="cuda").manual_seed(9)
    tensors = [(torch.randn(n, generator=g, device="cuda", dtype=torch.float64) * scale).to(dtype) for n in sizes]
    before, want = [t.clone() for t in tensors], _norm(tensors)
    assert math.isfinite(want) and max_norm < want < 3e38
    outs = [torch.full_like(t, 7) for t in tensors]
    for where in (outs, None):
        norm = _clip(B, tensors, max_norm, where)
        assert abs(float(norm) - want) <= 9 * V * want
        for o, t in zip(tensors if where is None else where, before):
            ref = t.double() * (max_norm / want)
            assert bool(((o.double() - ref).abs() <= (12 * V + HALF[dtype]) * ref.abs() + SMALL[dtype]).all())
