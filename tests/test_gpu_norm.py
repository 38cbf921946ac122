"""The norms around a block and their gradient against plain 64-bit forms.

Tolerances, u the half step of the rows' type (2^-11 fp16, 2^-8 bf16, 2^-24 fp32), v = 2^-24. A
row's sum of squares passes through at most 64 + 5 + 16 roundings (a thread's chain, a warp's tree, the
warps), all terms positive; the mean and eps add three, the inverse root halves what comes in and adds one: its
relative error is at most r = (88 / 2 + 1) v. The other sums over a row are off by 85 v of the sum of their terms'
magnitudes. Each product or addition on the way adds v of its value, and a term's error is carried through the
formulas below by its magnitude; the last rounding adds u of the result, or half of fp16's smallest step. The
gradient's sum of w dv m over a row is taken as the three sums that make it up (g = dout + r gamma_pre du - n mean), so
its error is that of the sum of the three's magnitudes. Sums over rows pass through at most R / 304 + 1 rows of a unit, 8 units of a CTA and 304 / 32 + 32 partial sums.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

V = 2.0 ** -24
RMS = 45 * V
ROW = 85 * V
TYPES = {0: torch.float16, 1: torch.bfloat16, 2: torch.float32}
HALF = {0: 2.0 ** -11, 1: 2.0 ** -8, 2: 2.0 ** -24}
SMALL = {0: 2.0 ** -25, 1: 0.0, 2: 0.0}
EPS = 1e-6


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from w4a16_moe_expert_router_gb300 import build as libbuild
    libbuild.build()
    from w4a16_moe_expert_router_gb300 import binding
    return binding


def _normal(shape, seed, dtype, scale=1.0, shift=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float64) * scale + shift).to(dtype)


def _inputs(R, d, typ, form, gate_rows, seed=0):
    dt, f32 = TYPES[typ], torch.float32
    s = {"x": _normal((R, d), seed + 1, dt, 2.0)}
    if "p" in form:    # the norm after the block
        s["gamma_post"] = _normal((d,), seed + 2, f32, 0.1, 1.0)
    if "y" in form:
        s["y"] = _normal((R, d), seed + 3, dt, 3.0)
    if gate_rows:
        s["gate"] = _normal((-(-R // gate_rows), d), seed + 4, f32, 0.3, 0.5)
    if "u" in form:
        s["gamma_pre"] = _normal((d,), seed + 5, f32, 0.1, 1.0)
    if "x" not in form:
        s["x"] = None
    return s


def _gate(s, R, gate_rows):
    if "gate" not in s:
        return torch.ones((), dtype=torch.float64, device="cuda")
    return s["gate"].double()[torch.arange(R, device="cuda") // gate_rows]


def _rinv(v):
    return 1 / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)


def _norm(v):
    return v.norm(dim=1, keepdim=True)


# R, d, type, form (x: residual, y: block output, p: its norm, u: the next norm), gate_rows, residual_scale
CASES = [
    (1, 2048, 0, "xypu", 1, 1.0), (1, 8, 1, "xypu", 0, 1.0), (3, 8192, 2, "xypu", 2, 0.5), (5, 8192, 1, "xypu", 5, 1.0),
    (7, 1000, 0, "xyp", 3, 0.25), (33, 264, 2, "yp", 33, 1.0), (2, 4104, 0, "xu", 0, 1.0), (600, 520, 1, "xyu", 7, -1.0),
    (1217, 256, 0, "xypu", 1217, 1.0), (1300, 8, 0, "xypu", 1, 1.0), (1501, 1000, 1, "xypu", 300, 0.5),
    (1500, 2048, 1, "xypu", 1, 1.0), (1400, 1024, 2, "xypu", 1399, 2.0), (1250, 512, 0, "xu", 0, 0.5),
    (1222, 2056, 1, "xypu", 100, 1.0), (4000, 64, 2, "xyp", 11, 1.0), (700, 4096, 2, "xypu", 64, 1.0),
    (640, 8192, 0, "ypu", 639, 1.0), (5000, 136, 1, "xy", 1700, 1.0), (609, 16, 2, "xypu", 1 << 22, 1.0),
]
IDS = ["-".join(map(str, c)) for c in CASES]


@pytest.mark.parametrize("R,d,typ,form,gate_rows,scale", CASES, ids=IDS)
def test_norm_matches_the_definition(B, R, d, typ, form, gate_rows, scale):
    s = _inputs(R, d, typ, form, gate_rows)
    dt, u, small = TYPES[typ], HALF[typ], SMALL[typ]
    want_out = "y" in form
    out = torch.full((R, d), 7, dtype=dt, device="cuda") if want_out else None
    nxt = torch.full((R, d), 7, dtype=dt, device="cuda") if "u" in form else None
    cfg = B.make_norm(R, d, typ, gate_rows, scale, EPS)
    B.moe_w4a16_norm(cfg, s["x"], s.get("y"), s.get("gamma_post"), s.get("gate"), s.get("gamma_pre"), out, nxt)
    # what the kernel holds in fp32 and how far it may be off
    o = torch.zeros(R, d, dtype=torch.float64, device="cuda")
    e = torch.zeros_like(o)
    if s["x"] is not None:
        o = cfg.residual_scale * s["x"].double()
        e = V * o.abs()
    if "y" in form:
        y = s["y"].double()
        v = y * _rinv(y) * s["gamma_post"].double() if "p" in form else y
        gv = _gate(s, R, gate_rows) * v
        o = o + gv
        e = e + (RMS + 3 * V) * gv.abs() + V * o.abs()
    if out is not None:
        err = (out.double() - o).abs()
        assert bool((err <= e + u * (o.abs() + e) + small).all()), float((err / (o.abs() + 1e-30)).max())
    if nxt is not None:
        r = _rinv(o)
        ref = o * r * s["gamma_pre"].double()
        lim = (s["gamma_pre"].double() * r).abs() * e + ref.abs() * (RMS + 3 * V + _norm(e) / _norm(o))
        err = (nxt.double() - ref).abs()
        assert bool((err <= lim + u * (ref.abs() + lim) + small).all()), float((err / (ref.abs() + 1e-30)).max())


def _backward(B, cfg, s, stream, dout, du, R, d, dt, want, cuda_stream=None):
    out = {"x": torch.full((R, d), 7, dtype=dt, device="cuda")}
    if "y" in s:
        out["y"] = torch.full((R, d), 7, dtype=dt, device="cuda")
    for n in ("gamma_post", "gate", "gamma_pre"):
        if n in s and (n != "gamma_pre" or du is not None):
            out[n] = torch.full_like(s[n], 7)
    out = {k: v for k, v in out.items() if k in want}
    ws = torch.full((B.moe_w4a16_norm_backward_workspace_bytes(cfg),), 255, dtype=torch.uint8, device="cuda")
    B.moe_w4a16_norm_backward(cfg, s.get("y"), s.get("gamma_post"), s.get("gate"), stream, s.get("gamma_pre"), dout, du,
                              out.get("x"), out.get("y"), out.get("gamma_post"), out.get("gate"),
                              out.get("gamma_pre"), ws, cuda_stream)
    return out


ALL = ("x", "y", "gamma_post", "gate", "gamma_pre")


def _want(s, R, gate_rows, scale, stream, dout, du):
    """The gradients in 64 bits and what the kernel's may be off by before their last rounding."""
    g = dout.double() if dout is not None else 0.0 * (du if du is not None else stream).double()
    eg = torch.zeros_like(g)
    parts = g.abs()  # the magnitudes of what g is made of
    want, lim = {}, {}
    rows = R / 304 + 1 + 8 + 10 + 32
    if du is not None:
        o, w = stream.double(), s["gamma_pre"].double() * du.double()
        d = o.shape[1]
        r = _rinv(o)
        n = o * r
        mean = (w * n).mean(1, keepdim=True)
        em = r * (ROW + 2 * V) * (w * o).abs().mean(1, keepdim=True) + mean.abs() * (RMS + 3 * V)
        g = g + r * (w - n * mean)
        parts = parts + r * (w.abs() + (n * mean).abs())
        eg = r * ((w.abs() + (n * mean).abs()) * (2 * RMS + 6 * V) + n.abs() * em) + V * g.abs()
        want["gamma_pre"] = (du.double() * n).sum(0)
        lim["gamma_pre"] = (du.double() * n).abs().sum(0) * (RMS + (2 + rows) * V)
    want["x"], lim["x"] = scale * g, abs(scale) * eg + V * (scale * g).abs()
    if "y" in s:
        y, q = s["y"].double(), _gate(s, R, gate_rows)
        dv, edv = q * g, q.abs() * eg + V * (q * g).abs()
        if "gamma_post" in s:
            w = s["gamma_post"].double()
            r = _rinv(y)
            m = y * r
            mean = (w * dv * m).mean(1, keepdim=True)
            em = r * ((w.abs() * edv + (ROW + 6 * V) * (w * q).abs() * parts) * y.abs()).mean(
                1, keepdim=True) + \
                mean.abs() * (RMS + 3 * V)
            want["y"] = r * (w * dv - m * mean)
            lim["y"] = r * (w.abs() * edv + ((w * dv).abs() + (m * mean).abs()) * (2 * RMS + 6 * V) + m.abs() * em)
            want["gamma_post"] = (dv * m).sum(0)
            lim["gamma_post"] = (edv * m.abs() + (dv * m).abs() * (RMS + (2 + rows) * V)).sum(0)
            v, ev = w * m, (RMS + 2 * V) * (w * m).abs()
        else:
            want["y"], lim["y"] = dv, edv
            v, ev = y, 0 * y
        if "gate" in s:
            at = torch.arange(R, device="cuda") // gate_rows
            zero = torch.zeros(s["gate"].shape, dtype=torch.float64, device="cuda")
            want["gate"] = zero.index_add(0, at, g * v)
            lim["gate"] = zero.index_add(0, at, eg * v.abs() + g.abs() * ev + (2 + rows + gate_rows / (R / 304 + 1))
                                         * V * (g * v).abs() if R < 304 else
                                         eg * v.abs() + g.abs() * ev + (2 + rows) * V * (g * v).abs())
    return want, lim


@pytest.mark.parametrize("R,d,typ,form,gate_rows,scale", CASES, ids=IDS)
def test_gradient_matches_the_definition(B, R, d, typ, form, gate_rows, scale):
    dt = TYPES[typ]
    s = _inputs(R, d, typ, form, gate_rows, seed=10)
    s.pop("x")
    stream, dout = _normal((R, d), 21, dt, 2.0), _normal((R, d), 22, dt)
    du = _normal((R, d), 23, dt) if "u" in form else None
    cfg = B.make_norm(R, d, typ, gate_rows, scale, EPS)
    got = _backward(B, cfg, s, stream, dout, du, R, d, dt, ALL)
    want, lim = _want(s, R, gate_rows, cfg.residual_scale, stream, dout, du)
    assert set(got) == set(want)
    for n in want:
        rows = n in ("x", "y")
        u, small = (HALF[typ], SMALL[typ]) if rows else (V, 0.0)
        err = (got[n].double() - want[n]).abs()
        bound = lim[n] + u * (want[n].abs() + lim[n]) + small
        assert bool((err <= bound).all()), (n, float((err - bound).max()))
    again = _backward(B, cfg, s, stream, dout, du, R, d, dt, ALL)
    assert all(torch.equal(got[n], again[n]) for n in got)  # the same bits in every run
    # one output at a time gives the same values
    for n in got:
        alone = _backward(B, cfg, s, stream, dout, du, R, d, dt, (n,))
        assert torch.equal(alone[n], got[n]), n


# A gate row per row, in every number of pieces; gate rows that go on in the next unit, in two units and in many.
GATES = [
    (2000, 2048, 1, "xypu", 1, 1.0), (1500, 520, 2, "xypu", 1, 0.5), (900, 1032, 0, "xyu", 1, 1.0), (650, 4096, 2, "xyp", 1, 1.0),
    (640, 8192, 2, "xypu", 1, 2.0), (700, 8192, 1, "yp", 1, 1.0), (3, 264, 0, "xypu", 1, 1.0), (20000, 8, 2, "xypu", 1, 1.0),
    (3001, 2048, 0, "xypu", 2, 1.0), (4097, 1200, 1, "xypu", 31, 1.0), (2500, 712, 2, "xypu", 900, 1.0), (1999, 4104, 0, "xyp", 500, 1.0),
    (30000, 16, 1, "ypu", 17, 0.5), (800, 1344, 0, "xypu", 799, 1.0), (2000, 1536, 1, "xu", 0, 1.0), (2000, 5000, 2, "xyp", 0, 1.0),
]
GATE_IDS = ["-".join(map(str, c)) for c in GATES]


@pytest.mark.parametrize("R,d,typ,form,gate_rows,scale", GATES, ids=GATE_IDS)
def test_gate_rows_and_widths(B, R, d, typ, form, gate_rows, scale):
    test_norm_matches_the_definition(B, R, d, typ, form, gate_rows, scale)
    test_gradient_matches_the_definition(B, R, d, typ, form, gate_rows, scale)


@pytest.mark.parametrize("R,d,typ,form,gate_rows", [(700, 1032, 1, "xypu", 1), (1300, 256, 0, "xu", 0), (650, 8192, 2, "xypu", 9),
                                                    (5, 2048, 1, "xyu", 2)])
def test_outputs_in_place_of_inputs(B, R, d, typ, form, gate_rows):
    dt = TYPES[typ]
    s = _inputs(R, d, typ, form, gate_rows)
    cfg = B.make_norm(R, d, typ, gate_rows, 0.5, EPS)

    def forward(x, y, out, u):
        B.moe_w4a16_norm(cfg, x, y, s.get("gamma_post"), s.get("gate"), s["gamma_pre"], out, u)
        return out, u

    new = lambda: torch.full((R, d), 7, dtype=dt, device="cuda")
    want = forward(s["x"], s.get("y"), new(), new())
    for swap in (False, True):
        x, y = s["x"].clone(), s["y"].clone() if "y" in s else new()
        got = forward(x, y if "y" in s else None, *((y, x) if swap else (x, y)))
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    if "y" not in s:
        return
    dout, du = _normal((R, d), 31, dt), _normal((R, d), 32, dt)
    ws = torch.empty(B.moe_w4a16_norm_backward_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")

    def backward(dout, du, dx, dy):
        B.moe_w4a16_norm_backward(cfg, s["y"], s.get("gamma_post"), s.get("gate"), want[0], s["gamma_pre"], dout, du, dx, dy,
                                  None, None, None, ws)
        return dx, dy

    wanted = backward(dout, du, new(), new())
    for swap in (False, True):
        a, b = dout.clone(), du.clone()
        got = backward(a, b, *((b, a) if swap else (a, b)))
        assert all(torch.equal(p, q) for p, q in zip(got, wanted))


@pytest.mark.parametrize("R,d,typ,form,gate_rows", [(333, 1032, 1, "xypu", 7), (40, 512, 0, "xu", 0), (900, 264, 2, "xypu", 1)])
def test_a_gradient_of_the_next_norm_alone(B, R, d, typ, form, gate_rows):
    """No gradient arrives at out: the same as one of zeros."""
    dt = TYPES[typ]
    s = _inputs(R, d, typ, form, gate_rows)
    s.pop("x")
    stream, du = _normal((R, d), 21, dt, 2.0), _normal((R, d), 23, dt)
    cfg = B.make_norm(R, d, typ, gate_rows, 1.0, EPS)
    got = _backward(B, cfg, s, stream, None, du, R, d, dt, ALL)
    zeros = _backward(B, cfg, s, stream, torch.zeros_like(du), du, R, d, dt, ALL)
    assert all(torch.equal(got[n], zeros[n]) for n in zeros)


def test_no_rows_clear_the_sums(B):
    cfg = B.make_norm(0, 264, 1, 4)
    empty = torch.empty((0, 264), dtype=torch.bfloat16, device="cuda")
    gamma, post, pre = (torch.full((264,), 7.0, device="cuda") for _ in range(3))
    ws = torch.empty(max(B.moe_w4a16_norm_backward_workspace_bytes(cfg), 16), dtype=torch.uint8, device="cuda")
    B.moe_w4a16_norm(cfg, empty, empty, gamma, None, gamma, empty, empty)
    B.moe_w4a16_norm_backward(cfg, empty, gamma, None, empty, gamma, empty, empty, empty, empty, post, None, pre, ws)
    assert not bool(post.any()) and not bool(pre.any()) and bool((gamma == 7).all())


def test_a_row_that_is_no_number_stays_its_own(B):
    """Infinities and NaN of one row reach no other row."""
    for R, d, typ, gate_rows in ((700, 1032, 1, 1), (700, 256, 0, 300), (3, 8192, 2, 3)):
        dt = TYPES[typ]
        s = _inputs(R, d, typ, "xypu", gate_rows)
        cfg = B.make_norm(R, d, typ, gate_rows, 1.0, EPS)

        def forward():
            out, u = (torch.full((R, d), 7, dtype=dt, device="cuda") for _ in range(2))
            B.moe_w4a16_norm(cfg, s["x"], s["y"], s["gamma_post"], s["gate"], s["gamma_pre"], out, u)
            return out, u

        want = forward()
        s["x"][1, 5], s["y"][R - 1, 3] = float("inf"), float("nan")
        got = forward()
        keep = [r for r in range(R) if r not in (1, R - 1)]
        assert all(torch.equal(a[keep], b[keep]) for a, b in zip(got, want))
        assert not bool(torch.isfinite(got[1][1, 5])) and not bool(torch.isfinite(got[1][R - 1]).any())


def test_streams_and_a_replayed_graph(B):
    """Forward and backward captured together, replayed with other inputs, beside an eager call on another stream."""
    R, d, typ = 777, 1032, 1
    dt = TYPES[typ]
    s, other = (_inputs(R, d, typ, "xypu", 9, seed=i) for i in (0, 50))
    dout, du = _normal((R, d), 61, dt), _normal((R, d), 62, dt)
    cfg = B.make_norm(R, d, typ, 9, 0.5, EPS)

    def step(s):
        out, u = torch.empty((R, d), dtype=dt, device="cuda"), torch.empty((R, d), dtype=dt, device="cuda")
        B.moe_w4a16_norm(cfg, s["x"], s["y"], s["gamma_post"], s["gate"], s["gamma_pre"], out, u)
        return [out, u, *_backward(B, cfg, s, out, dout, du, R, d, dt, ALL).values()]

    want, want_other = step(s), step(other)
    live = {k: v.clone() for k, v in s.items()}
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = step(live)
    side = torch.cuda.Stream()
    for source, ref in ((s, want), (other, want_other), (s, want)):
        for k in live:
            live[k].copy_(source[k])
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        with torch.cuda.stream(side):
            beside = step(other)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
        assert all(torch.equal(a, b) for a, b in zip(beside, want_other))


def test_rows_past_32_bits_of_offset(B):
    R, d, dt = (1 << 20) + 3, 4104, torch.bfloat16  # 4.3 billion elements
    x = torch.empty((R, d), dtype=dt, device="cuda")
    for i in range(0, R, 1 << 17):
        x[i:i + (1 << 17)].normal_()
    gamma = _normal((d,), 5, torch.float32, 0.1, 1.0)
    u, gx, gg = torch.empty_like(x), torch.empty_like(x), torch.empty_like(gamma)

    def step(R, x, u, gx):
        cfg = B.make_norm(R, d, 1, 0, 1.0, EPS)
        ws = torch.empty(B.moe_w4a16_norm_backward_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
        B.moe_w4a16_norm(cfg, x, None, None, None, gamma, None, u)
        B.moe_w4a16_norm_backward(cfg, None, None, None, x, gamma, None, u, gx, None, None, None, gg, ws)
        return u, gx

    step(R, x, u, gx)
    tail = x[-5:].clone()
    want = step(5, tail, torch.empty_like(tail), torch.empty_like(tail))
    assert torch.equal(u[-5:], want[0]) and torch.equal(gx[-5:], want[1])
    middle = x[1046500:1046505].clone()  # on both sides of 2^32 elements
    want = step(5, middle, torch.empty_like(middle), torch.empty_like(middle))
    assert torch.equal(u[1046500:1046505], want[0]) and torch.equal(gx[1046500:1046505], want[1])
