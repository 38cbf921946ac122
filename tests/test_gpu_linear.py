"""Products of rows with weights, with bias, activation, gate and residual, dense and
by experts, and their gradients, against plain 64-bit forms.

Tolerances, u the half step of the type (2^-11 fp16, 2^-8 bf16), t = 2^-23 the step of
fp32.  Products of 16-bit values are exact in fp32; each of the n additions of a sum is off by
at most one step of a partial sum, at most S = sum of the magnitudes: (n + 1) t S.  The
activations change by at most 1.13 times their argument's error, and are themselves good to
2^-17 of |z|, their logistic part's relative error; a rounding to the type adds u |y| (or half
of fp16's smallest step).  A product over dz carries the roundings of dz, u sum |w dz|.
Those are worst cases that add up for sums of a thousand terms, so the whole output is
held to the roundings as they add up at random too: its difference, over its norm, is at most
u for one rounding to the type and 1.42 u (sqrt 2) for two, plus the sums' t sqrt(n) |S| / |y|
and the activations' 2^-17.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

T23 = 2.0 ** -23
ACT = 2.0 ** -17
TYPES = {0: torch.float16, 1: torch.bfloat16}
HALF = {0: 2.0 ** -11, 1: 2.0 ** -8}
SMALL = {0: 2.0 ** -25, 1: 0.0}


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from w4a16_moe_expert_router_gb300 import build as libbuild
    libbuild.build()
    from w4a16_moe_expert_router_gb300 import binding
    return binding


def _normal(shape, seed, dtype, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float64) * scale).to(dtype)


def _offsets(R, E, seed, spare=0):
    """Random rows for the experts, some without any; the last `spare` rows belong to none."""
    rng = np.random.default_rng(seed)
    p = rng.random(E) * (rng.random(E) < 0.7)
    if p.sum() == 0:
        p[E // 2] = 1
    n = rng.multinomial(max(R - spare, 0), p / p.sum())
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int32)


def _act(z, kind):
    if kind == 3:
        return z
    if kind == 2:
        return z / (1 + torch.exp(-z))
    if kind == 1:
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2))
    return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))


def _act_grad(z, kind):
    z = z.detach().clone().requires_grad_()
    with torch.enable_grad():
        return torch.autograd.grad(_act(z, kind).sum(), z)[0]


def _check(got, want, tol, rel):
    got, want = got.double(), want.double()
    assert bool(torch.isfinite(got).all())
    err = (got - want).abs()
    assert bool((err <= tol).all()), ("element", float((err / tol.clamp(min=1e-300)).max()))
    if float(want.norm()) > 0:
        assert float(err.norm() / want.norm()) <= rel, ("norm", float(err.norm() / want.norm()), rel)


class Case:
    def __init__(self, R, K, N, E, act, gated, typ, bias, res, seed, spare=0):
        self.R, self.K, self.N, self.E, self.act, self.gated, self.typ = R, K, N, E, act, gated, typ
        dt = TYPES[typ]
        self.Nw = 2 * N if gated else N
        self.off = _offsets(R, E, seed, spare) if E else np.array([0, R], np.int32)
        self.used = int(self.off[-1])
        self.offd = torch.from_numpy(self.off).cuda() if E else None
        self.x = _normal((R, K), seed + 1, dt)
        self.x[self.used:] = float("nan")  # rows of no expert are not used
        self.w = _normal((max(E, 1), self.Nw, K), seed + 2, dt, K ** -0.5)
        self.b = _normal((max(E, 1), self.Nw), seed + 3, torch.float32, 0.5) if bias else None
        self.res = _normal((R, N), seed + 4, dt) if res else None

    def forward(self):
        """y, z in 64 bits and the tolerances of both for the used rows."""
        z = torch.zeros(self.used, self.Nw, dtype=torch.float64, device="cuda")
        S = torch.zeros_like(z)
        for e in range(len(self.off) - 1):
            i, j = int(self.off[e]), int(self.off[e + 1])
            x, w = self.x[i:j].double(), self.w[e].double()
            z[i:j], S[i:j] = x @ w.T, x.abs() @ w.abs().T
            if self.b is not None:
                z[i:j] += self.b[e].double()
                S[i:j] += self.b[e].double().abs()
        e_z = (self.K + 2) * T23 * S
        g, eg = z[:, :self.N], e_z[:, :self.N]
        y = _act(g, self.act)
        e_y = 1.13 * eg + ACT * g.abs() + 1e-9
        if self.gated:
            u, eu = z[:, self.N:], e_z[:, self.N:]
            e_y = e_y * (u.abs() + eu) + y.abs() * eu
            y = y * u
        if self.res is not None:
            y = y + self.res[:self.used].double()
        u = HALF[self.typ]
        e_y = (1 + u) * e_y + (u + T23) * y.abs() + SMALL[self.typ]
        self.noise = T23 * math.sqrt(self.K) * float(S.norm() / max(float(z.norm()), 1e-30))
        return y, z, e_y, (1 + u) * e_z + u * z.abs() + SMALL[self.typ]


def _run_forward(B, c, save=True, stream=None):
    cfg = B.make_linear(c.R, c.K, c.N, max(c.E, 1), c.act, int(c.gated), c.typ)
    out = torch.full((c.R, c.N), 7, dtype=TYPES[c.typ], device="cuda")
    z = torch.full((c.R, c.Nw), 7, dtype=TYPES[c.typ], device="cuda") if save else None
    ws = torch.empty(B.moe_w4a16_linear_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
    B.moe_w4a16_workspace_init(ws)
    B.moe_w4a16_linear(cfg, c.x, c.offd, c.w, c.b, c.res, out, z, ws, stream)
    torch.cuda.synchronize()
    assert B.moe_w4a16_read_error(ws) == B.OK
    return out, z


def _check_forward(B, c):
    out, z = _run_forward(B, c)
    y, zz, e_y, e_z = c.forward()
    u = HALF[c.typ]
    _check(z[:c.used], zz, e_z, u + c.noise)
    _check(out[:c.used], y, e_y, u + 3 * c.noise + ACT)
    assert bool((out[c.used:] == 7).all()) and bool((z[c.used:] == 7).all())
    only, _ = _run_forward(B, c, save=False)
    assert torch.equal(only, out)


# R, K, N, E (0: dense), activation, gated, type, bias, residual, rows of no expert
FORWARD = [
    # up to 32 rows: the kernel for single tokens and small batches (16 at most), and tiles of 32 columns
    (1, 8, 8, 0, 3, 0, 0, False, False, 0), (1, 2048, 136, 0, 0, 0, 0, True, True, 0), (2, 264, 72, 0, 1, 1, 1, True, True, 0),
    (3, 1000, 16, 0, 2, 0, 1, True, False, 0), (5, 72, 200, 0, 0, 1, 0, False, True, 0), (8, 2056, 40, 0, 3, 0, 1, True, True, 0),
    (1, 64, 64, 5, 0, 1, 0, True, False, 0), (8, 704, 72, 128, 0, 1, 1, False, True, 0), (8, 136, 8, 256, 3, 0, 0, True, False, 3),
    (7, 200, 24, 3, 2, 0, 0, True, True, 2), (8, 64, 32, 1, 1, 0, 0, False, False, 0),
    (9, 8, 8, 0, 3, 0, 0, False, False, 0), (16, 64, 128, 0, 3, 0, 0, False, False, 0), (31, 72, 136, 0, 0, 0, 1, True, True, 0),
    (32, 1000, 264, 0, 2, 1, 0, True, True, 0), (9, 65536, 8, 0, 3, 0, 1, True, False, 0),
    (17, 40, 24, 0, 1, 1, 1, True, True, 0), (32, 200, 72, 5, 0, 1, 0, True, True, 2), (24, 2056, 40, 2, 2, 0, 1, False, False, 0),
    (32, 64, 16, 256, 3, 0, 0, True, True, 0), (16, 72, 8, 3, 0, 1, 0, True, False, 16),
    # tiles
    (33, 65536, 8, 0, 3, 0, 1, True, False, 0), (48, 8, 8, 0, 0, 1, 0, True, True, 0),
    # tiles of 32 to 256 columns, in steps of 32, and their edges
    (33, 136, 72, 0, 1, 0, 0, True, False, 0), (64, 520, 200, 0, 0, 1, 1, False, True, 0), (65, 64, 1032, 0, 3, 0, 0, True, True, 0),
    (127, 200, 136, 0, 2, 0, 1, True, True, 0), (128, 256, 128, 0, 0, 1, 0, True, False, 0), (129, 72, 264, 0, 0, 0, 0, True, True, 0),
    (257, 264, 136, 0, 1, 1, 1, True, True, 0), (777, 1000, 520, 0, 2, 0, 0, True, True, 0), (300, 16, 8, 0, 3, 0, 1, False, True, 0),
    (1500, 2048, 2056, 0, 0, 0, 1, True, False, 0), (4100, 136, 264, 0, 3, 0, 0, True, False, 0),
    # by experts
    (9, 64, 64, 8, 3, 0, 0, False, False, 0), (40, 136, 72, 7, 0, 1, 1, True, True, 5), (300, 704, 136, 128, 0, 1, 0, False, False, 0),
    (500, 72, 200, 256, 2, 0, 1, True, True, 40), (600, 264, 72, 3, 1, 1, 0, True, True, 1), (1000, 200, 264, 4, 0, 0, 1, True, False, 100),
    (2000, 64, 72, 2, 3, 0, 0, True, True, 0), (3000, 136, 136, 9, 0, 1, 1, False, True, 999), (64, 64, 64, 1, 0, 0, 0, True, False, 63),
    (33, 64, 64, 4, 0, 0, 0, True, False, 33),
]


# few tiles with a long contraction, which two, three and four pairs of CTAs share: the same columns
SHARED = [
    (40, 4096, 264, 0, 0, 0, 0, True, True, 0), (33, 2056, 1032, 0, 2, 1, 1, True, True, 0), (100, 4000, 520, 0, 1, 0, 1, False, True, 0),
    (300, 8200, 136, 0, 3, 0, 0, True, False, 0), (128, 2048, 72, 0, 0, 1, 0, True, True, 0), (64, 4096, 4096, 0, 2, 0, 1, True, True, 0),
    (100, 2056, 6000, 0, 3, 0, 0, False, True, 0), (1000, 4104, 600, 0, 0, 1, 0, True, False, 0),
    # single tokens and small batches: long rows shared by up to eight CTAs, and CTAs with several items
    (1, 4096, 128, 0, 0, 0, 0, True, True, 0), (16, 8200, 72, 0, 2, 1, 1, True, True, 0), (9, 1032, 2048, 0, 3, 0, 0, False, True, 0),
    (7, 65536, 24, 0, 1, 0, 1, True, False, 0), (5, 3080, 264, 3, 0, 1, 0, True, True, 2), (1, 72, 6000, 0, 3, 0, 1, True, True, 0),
    (16, 1032, 2056, 5, 2, 1, 0, True, True, 1), (16, 264, 4104, 40, 0, 0, 1, False, True, 0),
    (16, 4096, 4096, 0, 1, 0, 0, True, True, 0), (3, 2048, 22000, 0, 3, 0, 0, True, False, 0),
]
# the gradients' long contractions: outputs (input gradient) and rows (weight gradient)
SHARED_BACKWARD = [
    (40, 264, 4096, 0, 0, 0, 0, 0), (129, 1000, 2056, 0, 2, 1, 1, 0), (5001, 264, 136, 0, 3, 0, 1, 0), (4097, 72, 8, 0, 0, 1, 0, 0),
    (3000, 2048, 256, 0, 1, 0, 0, 0), (2500, 2056, 520, 0, 3, 0, 1, 0), (1152, 136, 1032, 0, 2, 0, 0, 0),
]


@pytest.mark.parametrize("R,K,N,E,act,gated,typ,bias,res,spare", SHARED, ids=["-".join(map(str, c)) for c in SHARED])
def test_forward_of_shared_tiles(B, R, K, N, E, act, gated, typ, bias, res, spare):
    _check_forward(B, Case(R, K, N, E, act, gated, typ, bias, res, R + K, spare))


@pytest.mark.parametrize("R,K,N,E,act,gated,typ,bias,res,spare", FORWARD, ids=["-".join(map(str, c)) for c in FORWARD])
def test_forward(B, R, K, N, E, act, gated, typ, bias, res, spare):
    _check_forward(B, Case(R, K, N, E, act, gated, typ, bias, res, R + K, spare))


class Grad:
    """Inputs of a gradient call and its outputs in 64 bits with their tolerances."""

    def __init__(self, c, seed):
        self.c, dt, u = c, TYPES[c.typ], HALF[c.typ]
        self.needs_z = c.gated or c.act != 3
        self.dout = _normal((c.R, c.N), seed + 5, dt)
        self.z = _normal((c.R, c.Nw), seed + 6, dt) if self.needs_z else None
        self.dout[c.used:] = float("nan")
        if self.z is not None:
            self.z[c.used:] = float("nan")
        n = c.used
        d = self.dout[:n].double()
        e_dz = torch.zeros(n, c.Nw, dtype=torch.float64, device="cuda")
        dz = d
        if self.needs_z:
            g = self.z[:n, :c.N].double()
            y, dy = _act(g, c.act), _act_grad(g, c.act)
            if c.gated:
                up = self.z[:n, c.N:].double()
                dz = torch.cat([d * up * dy, d * y], 1)
                e_dz = torch.cat([(d * up).abs(), d.abs()], 1)
            else:
                dz, e_dz = d * dy, d.abs()
            # the derivative's terms: |p| <= 1 and |z p (1 - p) v'| <= 1, each good to 2^-17, and y = z p
            e_dz = e_dz * 2 * ACT * (torch.cat([torch.ones_like(g), g.abs()], 1) if c.gated else 1)
        f = 1 if self.needs_z else 0
        e_op = (1 + u) * e_dz + f * (u * dz.abs() + SMALL[c.typ])  # dz as the products' operand
        E = len(c.off) - 1
        k = dict(dtype=torch.float64, device="cuda")
        self.dx, self.dw, self.db = torch.zeros(n, c.K, **k), torch.zeros(E, c.Nw, c.K, **k), torch.zeros(E, c.Nw, **k)
        self.e_dx, self.e_dw, self.e_db = torch.zeros_like(self.dx), torch.zeros_like(self.dw), torch.zeros_like(self.db)
        s_dx, s_dw = 0.0, 0.0
        for e in range(E):
            i, j = int(c.off[e]), int(c.off[e + 1])
            x, w, z, ez = c.x[i:j].double(), c.w[e].double(), dz[i:j], e_op[i:j]
            a, b = z.abs() @ w.abs(), z.abs().T @ x.abs()
            self.dx[i:j], self.dw[e], self.db[e] = z @ w, z.T @ x, z.sum(0)
            self.e_dx[i:j] = ez @ w.abs() + (c.Nw + 2) * T23 * a
            self.e_dw[e] = ez.T @ x.abs() + (j - i + 2) * T23 * b
            # 8 rows a thread (blocks of 64), eight threads, then every eighth of up to 1 + rows / 64 partial sums and
            # those eight: fewer than 26 + rows / 128 additions in a row
            self.e_db[e] = e_dz[i:j].sum(0) + (26 + (j - i) / 128) * T23 * z.abs().sum(0) + 1e-12
            s_dx, s_dw = s_dx + float(a.norm()) ** 2, s_dw + float(b.norm()) ** 2
        self.e_dx = (1 + u) * self.e_dx + u * self.dx.abs() + SMALL[c.typ]
        self.e_dw = (1 + u) * self.e_dw + u * self.dw.abs() + SMALL[c.typ]
        rel = u * (1.42 if f else 1) + 3 * ACT
        self.r_dx = rel + T23 * math.sqrt(c.Nw) * math.sqrt(s_dx) / max(float(self.dx.norm()), 1e-30)
        self.r_dw = rel + T23 * math.sqrt(c.R) * math.sqrt(s_dw) / max(float(self.dw.norm()), 1e-30)
        self.r_db = 3 * ACT + T23 * math.sqrt(c.R) * float(dz.norm()) * math.sqrt(c.R) / max(float(self.db.norm()), 1e-30)


def _run_backward(B, c, g, want=(True, True, True), stream=None):
    cfg = B.make_linear(c.R, c.K, c.N, max(c.E, 1), c.act, int(c.gated), c.typ)
    dx = torch.full((c.R, c.K), 7, dtype=TYPES[c.typ], device="cuda") if want[0] else None
    dw = torch.full(c.w.shape, 7, dtype=TYPES[c.typ], device="cuda") if want[1] else None
    db = torch.full((max(c.E, 1), c.Nw), 7, dtype=torch.float32, device="cuda") if want[2] else None
    ws = torch.full((B.moe_w4a16_linear_backward_workspace_bytes(cfg),), 255, dtype=torch.uint8, device="cuda")  # NaNs
    B.moe_w4a16_workspace_init(ws)
    B.moe_w4a16_linear_backward(cfg, c.x if want[1] else None, c.offd, c.w if want[0] else None, g.z, g.dout, dx, dw, db,
                                ws, stream)
    torch.cuda.synchronize()
    assert B.moe_w4a16_read_error(ws) == B.OK
    return dx, dw, db


# R, K, N, E, activation, gated, type, rows of no expert
BACKWARD = [
    (1, 8, 8, 0, 3, 0, 0, 0), (1, 64, 64, 0, 0, 0, 0, 0), (9, 72, 136, 0, 0, 1, 1, 0), (31, 136, 72, 0, 2, 0, 1, 0),
    (64, 128, 64, 0, 3, 0, 0, 0), (65, 264, 200, 0, 1, 1, 0, 0), (130, 1000, 520, 0, 0, 0, 1, 0), (777, 136, 264, 0, 2, 1, 0, 0),
    (1500, 520, 1032, 0, 1, 0, 0, 0), (4100, 264, 136, 0, 3, 0, 1, 0),
    (1, 64, 64, 3, 0, 0, 0, 0), (8, 136, 72, 8, 0, 1, 1, 3), (40, 64, 64, 7, 3, 0, 0, 5), (300, 264, 136, 128, 0, 1, 0, 0),
    (500, 72, 200, 256, 2, 0, 1, 40), (1000, 200, 264, 4, 1, 0, 0, 100), (3000, 136, 136, 9, 0, 1, 1, 999),
    (64, 64, 64, 1, 0, 0, 0, 63), (33, 64, 64, 4, 0, 0, 0, 33), (2000, 704, 72, 2, 3, 0, 1, 1),
]


@pytest.mark.parametrize("R,K,N,E,act,gated,typ,spare", BACKWARD, ids=["-".join(map(str, c)) for c in BACKWARD])
def test_backward(B, R, K, N, E, act, gated, typ, spare):
    c = Case(R, K, N, E, act, gated, typ, False, False, R + K + 1, spare)
    g = Grad(c, R + K + 1)
    dx, dw, db = _run_backward(B, c, g)
    _check(dx[:c.used], g.dx, g.e_dx, g.r_dx)
    _check(dw, g.dw, g.e_dw, g.r_dw)
    _check(db, g.db, g.e_db, g.r_db)
    assert bool((dx[c.used:] == 7).all())
    for n in range(3):  # each output alone gives the same bits
        alone = _run_backward(B, c, g, tuple(i == n for i in range(3)))
        assert torch.equal(alone[n], (dx, dw, db)[n])


@pytest.mark.parametrize("R,K,N,E,act,gated,typ,spare", SHARED_BACKWARD, ids=["-".join(map(str, c)) for c in SHARED_BACKWARD])
def test_backward_of_shared_tiles(B, R, K, N, E, act, gated, typ, spare):
    test_backward(B, R, K, N, E, act, gated, typ, spare)


def test_gradient_against_differences(B):
    """Central differences of sum(g out) over steps of the input, the weight and the bias,
    with the forward call in 16 bits: the quotient is off by the outputs' roundings,
    u sqrt(sum (g out)^2) for each of the two calls over 2 h (five times that is allowed),
    and by h^2 / 6 of the third derivative, at most 2 h^2 of the second term here."""
    for gated, act in ((0, 0), (1, 2), (0, 1), (1, 0)):
        R, K, N, h = 96, 64, 40, 0.25
        c = Case(R, K, N, 0, act, gated, 0, True, False, 11)
        g = _normal((R, N), 3, torch.float16)
        _, z = _run_forward(B, c)

        class G:
            pass

        G.z, G.dout = z, g
        dx, dw, db = _run_backward(B, c, G)

        def f():
            out, _ = _run_forward(B, c, save=False)
            return float((out.double() * g.double()).sum()), float((out.double() * g.double()).norm())

        for name, grad in (("x", dx), ("w", dw), ("b", db)):
            t = getattr(c, name)
            step = (_normal(t.shape, 5, torch.float64) * h / (16 if name == "b" else 64)).to(torch.float16).to(t.dtype)
            want = float((grad.double() * step.double()).sum())
            keep = t.clone()
            up, down = (keep.double() + step.double()).to(t.dtype), (keep.double() - step.double()).to(t.dtype)
            moved = (up.double() - down.double()) / 2  # what the rounded steps are
            want = float((grad.double() * moved.double()).sum())
            setattr(c, name, up)
            a, na = f()
            setattr(c, name, down)
            b, nb = f()
            setattr(c, name, keep)
            size = float((grad.double() * moved.double()).norm())
            tol = 5 * HALF[0] * (na + nb) / 2 + 2 * HALF[0] * size + 0.02 * abs(want) + 0.05 * size
            assert abs((a - b) / 2 - want) <= tol, (gated, act, name, (a - b) / 2, want, tol)


def _layer(B, x, lg, gu, bgu, dn, E, k, f, typ, dout=None):
    """route -> dispatch -> gate and up -> down -> combine with the residual, and back."""
    from w4a16_moe_expert_router_gb300 import runtime
    layer = runtime.Layer16(x.shape[0], x.shape[1], f, E, k, activation=0, type=typ)
    out = layer.forward(x, lg, gu, bgu, dn)
    if dout is None:
        return out.clone()
    return out.clone(), layer.backward(dout)


@pytest.mark.parametrize("T,d,f,E,k,typ", [(37, 256, 64, 8, 2, 0), (300, 264, 72, 16, 4, 1), (1, 128, 64, 4, 2, 0)])
def test_layer_forward_and_backward(B, T, d, f, E, k, typ):
    """The operators together, as a layer uses them, against autograd in 64 bits on the same
    routing.  Each stored intermediate (z, h, y, dz and the rows' gradients) rounds once to the
    type, u = 2^-11 or 2^-8 of its size and independent from element to element; the longest
    chain to a result passes eight of them, so its norm is off by at most 8 u."""
    dt, u = TYPES[typ], HALF[typ]
    x, lg = _normal((T, d), 1, dt), _normal((T, E), 2, torch.float32)
    gu, dn = _normal((E, 2 * f, d), 3, dt, d ** -0.5), _normal((E, d, f), 4, dt, f ** -0.5)
    bgu, dout = _normal((E, 2 * f), 5, torch.float32, 0.3), _normal((T, d), 6, dt)
    out, grads = _layer(B, x, lg, gu, bgu, dn, E, k, f, typ, dout)
    torch.cuda.synchronize()
    X, L, GU, BGU, DN = (t.double().detach().clone().requires_grad_() for t in (x, lg, gu, bgu, dn))
    val, idx = torch.topk(L, k, dim=1)
    w = torch.softmax(val, 1)
    y = X
    for r in range(k):
        z = torch.einsum("td,tnd->tn", X, GU[idx[:, r]]) + BGU[idx[:, r]]
        h = _act(z[:, :f], 0) * z[:, f:]
        y = y + w[:, r, None] * torch.einsum("tf,tdf->td", h, DN[idx[:, r]])
    y.backward(dout.double())
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())
    assert rel(out, y.detach()) <= 8 * u
    for name, want in (("x", X.grad), ("logits", L.grad), ("gate_up", GU.grad), ("gate_up_bias", BGU.grad), ("down", DN.grad)):
        assert rel(grads[name], want) <= 8 * u, (name, rel(grads[name], want), 8 * u)


def test_streams_and_a_captured_graph(B):
    """A captured forward and backward follow new inputs, and every run gives the same bits;
    two workspaces let two streams run at once."""
    c, c2 = (Case(300, 136, 72, 5, 0, 1, 1, True, True, s) for s in (1, 50))
    g = Grad(c, 2)
    first = _run_forward(B, c), _run_backward(B, c, g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    cfg = B.make_linear(c.R, c.K, c.N, c.E, 0, 1, 1)
    bufs = []
    for _ in streams:
        b = [torch.empty_like(t) for t in first[0] + first[1]]
        b += [torch.empty(B.moe_w4a16_linear_workspace_bytes(cfg), dtype=torch.uint8, device="cuda"),
              torch.empty(B.moe_w4a16_linear_backward_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")]
        B.moe_w4a16_workspace_init(b[5])
        B.moe_w4a16_workspace_init(b[6])
        bufs.append(b)

    def go(b, stream=None):
        B.moe_w4a16_linear(cfg, c.x, c.offd, c.w, c.b, c.res, b[0], b[1], b[5], stream)
        B.moe_w4a16_linear_backward(cfg, c.x, c.offd, c.w, g.z, g.dout, b[2], b[3], b[4], b[6], stream)

    torch.cuda.synchronize()
    for _ in range(5):
        for b, s in zip(bufs, streams):
            go(b, s)
    torch.cuda.synchronize()
    for b in bufs:
        assert all(torch.equal(x, y) for x, y in zip(b, first[0] + first[1]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(bufs[0])
    c.x.copy_(c2.x)
    c.offd.copy_(c2.offd)  # other rows for the experts: the launches read them on the device
    c.w.copy_(c2.w)
    graph.replay()
    torch.cuda.synchronize()
    go(bufs[1])
    torch.cuda.synchronize()
    assert not torch.equal(bufs[0][0], first[0][0])
    assert all(torch.equal(x, y) for x, y in zip(bufs[0][:5], bufs[1][:5]))  # not the workspaces


@pytest.mark.parametrize("R,K,N,E", [(40, 4096, 264, 0), (300, 2056, 1032, 0), (1, 4096, 128, 0), (16, 264, 4104, 40)])
def test_clusters_in_a_graph_beside_another_stream(B, R, K, N, E):
    """CTAs that share a tile or an item, in replayed graphs while another stream runs the same:
    the same bits every time."""
    c = Case(R, K, N, E, 0, 1, 1, True, True, R + 3)
    g = Grad(c, 4)
    want = _run_forward(B, c) + _run_backward(B, c, g)
    cfg = B.make_linear(R, K, N, max(E, 1), 0, 1, 1)
    streams, sets = [torch.cuda.Stream(), torch.cuda.Stream()], []

    def call(b):
        B.moe_w4a16_linear(cfg, c.x, c.offd, c.w, c.b, c.res, b[0], b[1], b[5])
        B.moe_w4a16_linear_backward(cfg, c.x, c.offd, c.w, g.z, g.dout, b[2], b[3], b[4], b[6])

    for _ in streams:
        b = [t.clone() for t in want] + [torch.empty(n, dtype=torch.uint8, device="cuda") for n in (
            B.moe_w4a16_linear_workspace_bytes(cfg), B.moe_w4a16_linear_backward_workspace_bytes(cfg))]
        B.moe_w4a16_workspace_init(b[5])
        B.moe_w4a16_workspace_init(b[6])
        sets.append(b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(sets[0])
        call(sets[0])
    for _ in range(3):
        for b in sets:
            for t in b[:5]:
                t.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(streams[0]):
            graph.replay()
        with torch.cuda.stream(streams[1]):
            call(sets[1])
            call(sets[1])
        torch.cuda.synchronize()
        for b in sets:
            assert all(torch.equal(t, w) for t, w in zip(b, want))
            assert B.moe_w4a16_read_error(b[5]) == B.OK and B.moe_w4a16_read_error(b[6]) == B.OK


def test_in_place_residual_and_infinities(B):
    """out may be the residual; an infinite row reaches its own outputs only, and an expert's
    weight gradient only from its own rows."""
    c = Case(200, 64, 72, 4, 3, 0, 0, True, True, 9)
    out, _ = _run_forward(B, c)
    cfg = B.make_linear(c.R, c.K, c.N, c.E, 3, 0, 0)
    same = c.res.clone()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    B.moe_w4a16_linear(cfg, c.x, c.offd, c.w, c.b, same, same, None, ws)
    torch.cuda.synchronize()
    assert torch.equal(same, out)
    e = int(np.argmax(np.diff(c.off)))
    row = int(c.off[e])  # the first row of its expert: behind the one before
    c.x[row] = float("inf")
    bad, _ = _run_forward(B, c)
    keep = torch.arange(c.R, device="cuda") != row
    assert torch.equal(bad[keep], out[keep]) and not bool(torch.isfinite(bad[row]).any())
    g = Grad(c, 3)
    _, dw, _ = _run_backward(B, c, g)
    finite = torch.isfinite(dw).flatten(1).all(1)
    assert [bool(v) for v in finite] == [i != e for i in range(c.E)]


@pytest.mark.parametrize("E", [0, 3])
def test_outputs_beyond_32_bits(B, E):
    """2^21 rows of 1032 outputs: elements past 2^31, bytes past 2^32, in the output, the saved z,
    the residual and dz; checked at the first, middle and last rows."""
    R, K, N = (1 << 21) + 5, 16, 1032
    dt, u = torch.bfloat16, HALF[1]
    x, w = _normal((R, K), 1, dt), _normal((max(E, 1), N, K), 2, dt, K ** -0.5)
    off = torch.tensor([0, 7, R - 100, R], dtype=torch.int32, device="cuda") if E else None
    res = torch.randn(R, N, device="cuda", dtype=dt)
    out, z = torch.empty_like(res), torch.empty_like(res)
    cfg = B.make_linear(R, K, N, max(E, 1), 2, 0, 1)
    ws = torch.empty(B.moe_w4a16_linear_backward_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
    B.moe_w4a16_workspace_init(ws)
    B.moe_w4a16_linear(cfg, x, off, w, None, res, out, z, ws)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    B.moe_w4a16_linear_backward(cfg, x, off, w, z, res, dx, dw, None, ws)
    torch.cuda.synchronize()
    assert B.moe_w4a16_read_error(ws) == B.OK
    for r, e in ((0, 0), (6, 0), (7, 1), (R // 2, 1), (R - 101, 1), (R - 100, 2), (R - 1, 2)):
        we = w[e if E else 0].double()
        S = x[r].double().abs() @ we.abs().T
        zz = x[r].double() @ we.T
        e_z = (K + 2) * T23 * S
        _check(z[r], zz, (1 + u) * e_z + u * zz.abs(), 1)
        y = _act(zz, 2) + res[r].double()
        _check(out[r], y, (1 + u) * (1.13 * e_z + ACT * zz.abs() + 1e-9) + (u + T23) * y.abs(), 1)
        g = z[r].double()
        dz = res[r].double() * _act_grad(g, 2)
        e_dz = (1 + u) * res[r].double().abs() * 2 * ACT + u * dz.abs()
        want = dz @ we
        tol = (1 + u) * (e_dz @ we.abs() + (N + 2) * T23 * (dz.abs() @ we.abs())) + u * want.abs()
        _check(dx[r], want, tol, 1)
    if E:  # the expert of the last hundred rows
        g, xs = z[R - 100:].double(), x[R - 100:].double()
        d = res[R - 100:].double()
        dz = d * _act_grad(g, 2)
        e_dz = (1 + u) * d.abs() * 2 * ACT + u * dz.abs()
        want = dz.T @ xs
        _check(dw[2], want, (1 + u) * (e_dz.T @ xs.abs() + 102 * T23 * (dz.abs().T @ xs.abs())) + u * want.abs(), 1)


def test_no_rows(B):
    cfg = B.make_linear(0, 64, 32, 3, 0, 0, 0)
    dw = torch.full((3, 32, 64), 7, dtype=torch.float16, device="cuda")
    db = torch.full((3, 32), 7, dtype=torch.float32, device="cuda")
    ws = torch.zeros(B.moe_w4a16_linear_backward_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    none = torch.empty(0, dtype=torch.float16, device="cuda")
    B.moe_w4a16_linear_backward(cfg, none, off, dw.clone(), none, none, None, dw, db, ws)
    torch.cuda.synchronize()
    assert bool((dw == 0).all()) and bool((db == 0).all())


@pytest.mark.parametrize("R,K,N", [(300, 256, 520), (300, 8200, 136), (3000, 256, 264), (5, 264, 72)])
def test_a_launch_before_that_outlasts_a_waits_limit(B, R, K, N):
    """Behind a launch of 2.4 s that lets the next one start at once (each wait in these kernels may last 2 s),
    the products' waits have not run out."""
    c = Case(R, K, N, 0, 3, 0, 1, True, True, R + 9)
    g = Grad(c, 4)
    want, (_, dw, _) = _run_forward(B, c), _run_backward(B, c, g, (False, True, False))
    cfg = B.make_linear(R, K, N, 1, 3, 0, 1)
    ws = [torch.empty(max(n, 256), dtype=torch.uint8, device="cuda") for n in (
        0, B.moe_w4a16_linear_workspace_bytes(cfg), B.moe_w4a16_linear_backward_workspace_bytes(cfg))]
    for w in ws:
        B.moe_w4a16_workspace_init(w)
    out, z, got = torch.zeros_like(want[0]), torch.zeros_like(want[1]), torch.zeros_like(dw)
    B.moe_w4a16_selftest_wait_timeout(ws[0], 1_200_000_000)
    B.moe_w4a16_linear(cfg, c.x, None, c.w, c.b, c.res, out, z, ws[1])
    B.moe_w4a16_selftest_wait_timeout(ws[0], 1_200_000_000)
    B.moe_w4a16_linear_backward(cfg, c.x, None, None, None, g.dout, None, got, None, ws[2])
    torch.cuda.synchronize()
    assert [B.moe_w4a16_read_error(w) for w in ws] == [B.ERR_TIMEOUT, B.OK, B.OK]
    assert torch.equal(out, want[0]) and torch.equal(z, want[1]) and torch.equal(got, dw)


@pytest.mark.parametrize("gated,act", [(0, 0), (1, 2), (0, 1), (1, 0)])
def test_gradient_against_differences_along_itself(B, gated, act):
    """Central differences of sum(g out) along the sign of each gradient, where the quotient is the sum of the
    gradient's magnitudes and not lost in the outputs' roundings.  It may differ from the gradient's product with the
    step by the roundings of the two calls' outputs (5 u |g out| each, over 2), by the quotient's own distance from the
    derivative, taken from the same quotient in 64 bits, and by the roundings of z, dz and the gradient: 8 u of the sum
    of magnitudes.  All of that is at most 3 % of the quotient."""
    R, K, N, u = 96, 64, 40, HALF[0]
    c = Case(R, K, N, 0, act, gated, 0, True, False, 11)
    g = _normal((R, N), 3, torch.float16)
    leaves = {n: getattr(c, n).double().requires_grad_() for n in ("x", "w", "b")}
    zz = leaves["x"] @ leaves["w"][0].T + leaves["b"]
    y = _act(zz[:, :N], act)
    ((y * zz[:, N:] if gated else y) * g.double()).sum().backward()

    class G:
        z, dout = _run_forward(B, c)[1], g

    def f():
        out, exact = _run_forward(B, c, save=False)[0].double() * g.double(), c.forward()[0] * g.double()
        return float(out.sum()), float(out.norm()), float(exact.sum())

    for name, grad in zip(("x", "w", "b"), _run_backward(B, c, G)):
        keep = getattr(c, name)
        step = torch.sign(leaves[name].grad).reshape(keep.shape) * (2.0 ** -7 if name == "x" else 2.0 ** -9 if name == "w" else 2.0 ** -5)
        up, down = (keep.double() + step).to(keep.dtype), (keep.double() - step).to(keep.dtype)
        moved = (up.double() - down.double()) / 2  # what the rounded steps are
        want, true = (float((t.double().reshape(moved.shape) * moved).sum()) for t in (grad, leaves[name].grad))
        setattr(c, name, up)
        a, na, a64 = f()
        setattr(c, name, down)
        b, nb, b64 = f()
        setattr(c, name, keep)
        tol = 5 * u * (na + nb) / 2 + abs((a64 - b64) / 2 - true) + 8 * u * float((grad.double().reshape(moved.shape) * moved).abs().sum())
        assert tol <= 0.03 * abs(want), (name, tol, want)
        assert abs((a - b) / 2 - want) <= tol, (name, (a - b) / 2, want, tol)


@pytest.mark.parametrize("E", [0, 3])
@pytest.mark.parametrize("gated", [0, 1])
def test_bias_gradient_of_more_than_two_million_rows(B, E, gated):
    """Above 2^21 rows the bias gradient's partial sums cover 256 rows each.  Whole numbers, whose sums stay below
    2^24, so that every addition in fp32 is exact: the sums are equal to those in 64 bits, the weight gradient to its
    one rounding, with and without the other outputs.  An expert without rows gets zeros, rows of none add nothing."""
    R, K, N = (1 << 21) + 300, 8, 24
    gen = torch.Generator(device="cuda").manual_seed(E + gated)

    def whole(most, *shape):
        return torch.randint(-most, most + 1, shape, generator=gen, device="cuda").to(torch.bfloat16)

    Nw = 2 * N if gated else N
    off = [0, 700001, 700001, R - 37] if E else [0, R]
    x, dout, z = whole(1, R, K), whole(4, R, N), whole(1, R, Nw) if gated else None
    for t in (x, dout) + ((z,) if gated else ()):
        t[off[-1]:] = float("nan")
    cfg = B.make_linear(R, K, N, max(E, 1), 3, gated, 1)
    offd = torch.tensor(off, dtype=torch.int32, device="cuda") if E else None
    ws = torch.full((B.moe_w4a16_linear_backward_workspace_bytes(cfg),), 255, dtype=torch.uint8, device="cuda")
    B.moe_w4a16_workspace_init(ws)

    def go(with_weight):
        dw = torch.full((max(E, 1), Nw, K), 7, dtype=torch.bfloat16, device="cuda") if with_weight else None
        db = torch.full((max(E, 1), Nw), 7, dtype=torch.float32, device="cuda")
        B.moe_w4a16_linear_backward(cfg, x if with_weight else None, offd, None, z, dout, None, dw, db, ws)
        torch.cuda.synchronize()
        assert B.moe_w4a16_read_error(ws) == B.OK
        return dw, db

    (dw, db), (_, alone) = go(True), go(False)
    assert torch.equal(db, alone)
    for e in range(len(off) - 1):
        d, rows = dout[off[e]:off[e + 1]].double(), x[off[e]:off[e + 1]].double()
        if gated:
            zz = z[off[e]:off[e + 1]].double()
            d = torch.cat([d * zz[:, N:], d * zz[:, :N]], 1)
        assert float(d.abs().sum(0).max() if len(d) else 0) < 2 ** 24
        assert torch.equal(db[e].double(), d.sum(0))
        assert torch.equal(dw[e], (d.T @ rows).to(torch.bfloat16))


def test_a_layer_on_another_stream_than_its_constructors(B):
    """A layer whose buffers take over memory that the constructor's stream still writes, used on another stream."""
    from w4a16_moe_expert_router_gb300 import runtime
    T, d, f, E, k, dt = 200, 264, 72, 8, 2, torch.bfloat16
    x, lg = _normal((T, d), 1, dt), _normal((T, E), 2, torch.float32)
    gu, dn, dout = _normal((E, 2 * f, d), 3, dt, d ** -0.5), _normal((E, d, f), 4, dt, f ** -0.5), _normal((T, d), 6, dt)
    out, grads = _layer(B, x, lg, gu, None, dn, E, k, f, 1, dout)
    want = [out] + [grads[n].clone() for n in sorted(grads)]
    torch.cuda.synchronize()
    busy = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in (1 << 20, 1 << 20, 1 << 24)]
    torch.cuda._sleep(100_000_000)
    for t in busy:
        t.fill_(255)
    del busy, t
    layer, other = runtime.Layer16(T, d, f, E, k, type=1), torch.cuda.Stream()
    out = layer.forward(x, lg, gu, None, dn, stream=other)
    grads = layer.backward(dout, stream=other)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip([out] + [grads[n] for n in sorted(grads)], want))
    assert all(B.moe_w4a16_read_error(layer.ws[i]) == B.OK for i in (0, 2))


def test_a_layer_without_tokens(B):
    from w4a16_moe_expert_router_gb300 import runtime
    none, gu, dn = (torch.ones(s, dtype=torch.float16, device="cuda") for s in ((0, 64), (4, 128, 64), (4, 64, 64)))
    layer = runtime.Layer16(0, 64, 64, 4, 2)
    out = layer.forward(none, torch.zeros(0, 4, device="cuda"), gu, None, dn)
    grads = layer.backward(none)
    torch.cuda.synchronize()
    assert out.shape == (0, 64) and bool((grads["gate_up"] == 0).all()) and bool((grads["down"] == 0).all())
