"""The norms and their gradient on rows far from one: large ones, and small ones without eps.

Bounds: those of test_gpu_norm, whose terms are relative to the values and so to the rows' scale, with the call's eps,
and half of the type's smallest step (bf16 2^-134, fp32 2^-150) for the result's own rounding. The scales keep the sums of
squares, and of the products of two rows, in fp32's normal range (2^-126 to 2^128): the largest is 256 (2.5e17)^2 =
2^123.6, the smallest squares are about 1e-32 = 2^-106, and those of columns a thousand times below that change a row's
sum by less than its own roundings.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import test_gpu_norm as N  # noqa: E402
from test_gpu_norm import B  # noqa: E402, F401

BF16, FP32 = 1, 2
STEP = {BF16: 2.0 ** -134, FP32: 2.0 ** -150}

# rows of the stream, rows of y, R, d, type, form, gate_rows, eps
CASES = [
    (1e14, 1.0, 700, 1032, FP32, "xypu", 7, 1e-6), (1.0, 1e14, 700, 1032, FP32, "xypu", 700, 1e-6),
    (1e16, 1e16, 333, 264, FP32, "xypu", 1, 1e-6), (2.5e17, 1.0, 50, 256, FP32, "xu", 0, 1e-6),
    (1.0, 2.5e17, 50, 256, FP32, "xyp", 3, 1e-6), (2.5e17, 1e3, 50, 256, FP32, "xypu", 50, 1e-6),
    (1e14, 1e14, 640, 2048, BF16, "xypu", 640, 1e-6), (1e16, 1.0, 333, 2056, BF16, "xypu", 5, 1e-6),
    (1.0, 2.5e17, 40, 256, BF16, "xyp", 1, 1e-6), (1e15, 1e15, 9, 8192, FP32, "xypu", 2, 1e-6),
    (1e-15, 1.0, 700, 1032, FP32, "xypu", 7, 0.0), (1.0, 1e-15, 700, 1032, FP32, "xypu", 700, 0.0),
    (1e-15, 1e-15, 333, 264, FP32, "xypu", 1, 0.0), (1e-15, 1e-15, 640, 2048, BF16, "xypu", 640, 0.0),
    (1e-16, 1.0, 40, 512, BF16, "xu", 0, 0.0), (1.0, 1e-16, 40, 512, BF16, "xyp", 40, 0.0),
    (1e-15, 1e-15, 9, 8192, FP32, "xypu", 2, 0.0),
]
IDS = ["-".join(map(str, c)) for c in CASES]


@pytest.mark.parametrize("big,big_y,R,d,typ,form,gate_rows,eps", CASES, ids=IDS)
def test_gradient_of_rows_far_from_one(B, monkeypatch, big, big_y, R, d, typ, form, gate_rows, eps):
    monkeypatch.setattr(N, "EPS", eps)
    dt = N.TYPES[typ]
    s = N._inputs(R, d, typ, form, gate_rows, seed=70)
    s.pop("x")
    if "y" in s:
        s["y"] = N._normal((R, d), 73, dt, big_y)
    stream = N._normal((R, d), 71, dt, big)
    # what arrives at out is as large as what comes through the next norm
    dout = N._normal((R, d), 72, dt, 1 / big if "u" in form else 1.0)
    du = N._normal((R, d), 74, dt) if "u" in form else None
    cfg = B.make_norm(R, d, typ, gate_rows, 1.0, eps)
    for arrives in (dout, None) if du is not None else (dout,):
        got = N._backward(B, cfg, s, stream, arrives, du, R, d, dt, N.ALL)
        want, lim = N._want(s, R, gate_rows, 1.0, stream, arrives, du)
        assert set(got) == set(want)
        for n in want:
            u, small = (N.HALF[typ], STEP[typ]) if n in ("x", "y") else (N.V, STEP[FP32])
            err = (got[n].double() - want[n]).abs()
            bound = lim[n] + u * (want[n].abs() + lim[n]) + small
            assert bool((err <= bound).all()), (n, float((err / (want[n].abs().mean() + 1e-300)).max()))


@pytest.mark.parametrize("big,big_y,R,d,typ,form,gate_rows,eps", CASES, ids=IDS)
def test_forward_of_rows_far_from_one(B, monkeypatch, big, big_y, R, d, typ, form, gate_rows, eps):
    monkeypatch.setattr(N, "EPS", eps)
    dt = N.TYPES[typ]
    s = N._inputs(R, d, typ, form, gate_rows, seed=70)
    x = N._normal((R, d), 71, dt, big)
    out, nxt = (torch.full((R, d), 7, dtype=dt, device="cuda") for _ in range(2))
    y = N._normal((R, d), 73, dt, big_y) if "y" in s else None
    pre = s.get("gamma_pre")
    B.moe_w4a16_norm(B.make_norm(R, d, typ, gate_rows, 1.0, eps), x, y, s.get("gamma_post"), s.get("gate"), pre, out,
                     nxt if pre is not None else None)
    o, e = x.double(), N.V * x.double().abs()
    if y is not None:
        gv = N._gate(s, R, gate_rows) * y.double() * N._rinv(y.double()) * s["gamma_post"].double()
        o, e = o + gv, e + (N.RMS + 3 * N.V) * gv.abs()
        e = e + N.V * o.abs()
    assert bool(((out.double() - o).abs() <= e + N.HALF[typ] * (o.abs() + e) + STEP[typ]).all())
    if pre is not None:
        r = N._rinv(o)
        ref = o * r * pre.double()
        lim = (pre.double() * r).abs() * e + ref.abs() * (N.RMS + 3 * N.V + N._norm(e) / N._norm(o))
        assert bool(((nxt.double() - ref).abs() <= lim + N.HALF[typ] * (ref.abs() + lim) + STEP[typ]).all())
