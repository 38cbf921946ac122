"""Token rows sorted by expert and back, with their gradients, against plain
64-bit forms.

Tolerances, with u the half step of the rows' type (2^-11 fp16, 2^-8 bf16, 2^-24
fp32) and v = 2^-24: the integers and the copied rows are equal.  A combined element
is a chain of k fused multiply-adds and one addition in fp32, each off by at most v
of a partial sum, all of which are at most S = sum |w row| + |res| (1 + k v): at most
(k + 1) v S (1 + 2^-20); the one rounding to the type adds u |out|, or half of fp16's
smallest step, 2^-25.  A weight's gradient adds at most n fused products in a thread, a
32nd of the row's, and at most 5 + 8 partial sums: (n + 13) v sum |dout row|.  A logit's gradient
w_r (dw_r - m), m the k-fold chain over w dw, takes w_r (e_r + e_m) from those errors
with e_m = sum_j w_j e_j + (k + 1) v sum_j |w_j dw_j|, and three roundings of its own,
for each time the token chose the expert.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

V = 2.0 ** -24
TYPES = {0: torch.float16, 1: torch.bfloat16, 2: torch.float32}
HALF = {0: 2.0 ** -11, 1: 2.0 ** -8, 2: 2.0 ** -24}
SMALL = {0: 2.0 ** -25, 1: 0.0, 2: 0.0}


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from w4a16_moe_expert_router_gb300 import build as libbuild
    libbuild.build()
    from w4a16_moe_expert_router_gb300 import binding
    return binding


def _ids(T, E, k, seed, kind):
    rng = np.random.default_rng(seed)
    if kind == "twice":  # a token may choose an expert more than once
        return rng.integers(0, E, (T, k)).astype(np.int32)
    idx = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    if kind == "drop":
        idx[rng.random((T, k)) < 0.2] = -1
        idx[rng.random((T, k)) < 0.05] = E
        idx[rng.random((T, k)) < 0.02] = 2 ** 31 - 1
        idx[rng.random((T, k)) < 0.02] = -2 ** 31
        idx[T - T // 4:] = -1
    elif kind == "none":
        idx[:] = -1
    elif kind == "one":
        idx[:] = E - 1
    return idx


def _places(idx, E):
    ids = idx.reshape(-1)
    order = [p for e in range(E) for p in np.nonzero(ids == e)[0]]
    counts = [int((ids == e).sum()) for e in range(E)]
    pos = np.full(ids.size, -1, np.int32)
    pos[order] = np.arange(len(order))
    plist = np.full(ids.size, -1, np.int32)
    plist[:len(order)] = order
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32), plist, pos.reshape(idx.shape)


def _normal(shape, seed, typ, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g, dtype=torch.float64) * scale).to(TYPES[typ]).cuda()


def _dispatch(B, cfg, idx, x, stream=None):
    T, E, k, d = cfg.tokens, cfg.experts, cfg.top_k, cfg.hidden
    out = dict(off=torch.full((E + 1,), -7, dtype=torch.int32, device="cuda"),
               lst=torch.full((T * k,), -7, dtype=torch.int32, device="cuda"),
               pos=torch.full((T, k), -7, dtype=torch.int32, device="cuda"),
               rows=torch.full((T * k, d), 7, dtype=x.dtype, device="cuda"))
    ws = torch.empty(B.moe_w4a16_dispatch_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
    B.moe_w4a16_dispatch(cfg, idx, x, out["off"], out["lst"], out["pos"], out["rows"], ws, stream)
    return out


CASES = [  # T, E, k, d, type, kind
    (1, 1, 1, 8, 0, "plain"), (1, 128, 8, 2048, 0, "plain"), (2, 3, 2, 64, 1, "twice"), (5, 256, 8, 200, 2, "drop"),
    (33, 24, 3, 1000, 1, "drop"), (304, 128, 8, 136, 0, "plain"), (305, 16, 8, 64, 1, "one"), (512, 128, 8, 72, 0, "drop"),
    (513, 128, 8, 72, 1, "drop"), (585, 256, 7, 40, 0, "twice"), (586, 9, 7, 40, 2, "plain"), (4096, 8, 1, 16, 0, "drop"),
    (4097, 8, 1, 16, 1, "one"), (1400, 4, 3, 2056, 0, "drop"), (2500, 31, 5, 64, 1, "none"), (20000, 128, 8, 16, 1, "twice"),
    (17, 8, 8, 8192, 2, "plain"), (3, 2, 2, 65536, 1, "drop"),
]
IDS = ["-".join(map(str, c)) for c in CASES]


@pytest.mark.parametrize("T,E,k,d,typ,kind", CASES, ids=IDS)
def test_dispatch_equals_the_definition(B, T, E, k, d, typ, kind):
    idx = _ids(T, E, k, T + d, kind)
    off, lst, pos = _places(idx, E)
    x = _normal((T, d), 1, typ)
    got = _dispatch(B, B.make_rows(T, E, k, d, typ), torch.from_numpy(idx).cuda(), x)
    torch.cuda.synchronize()
    assert np.array_equal(got["off"].cpu().numpy(), off)
    assert np.array_equal(got["lst"].cpu().numpy(), lst)
    assert np.array_equal(got["pos"].cpu().numpy(), pos)
    n = int(off[E])
    want = x[torch.from_numpy(lst[:n] // k).long().cuda()]
    assert torch.equal(got["rows"][:n], want)
    assert bool((got["rows"][n:] == 7).all())  # rows behind the last expert's stay as they were


def test_dispatch_gives_the_lists_of_route(B):
    from w4a16_moe_expert_router_gb300 import runtime, synth
    for tokens in (256, 700):
        wl = synth.Workload("r", tokens, 256, 64, 128, 8, 64, 64)
        buf = runtime.alloc_buffers(wl)
        B.moe_w4a16_route(buf.shape, runtime.to_device_f32(synth.make_logits(wl)), buf.routing, buf.workspace)
        got = _dispatch(B, B.make_rows(tokens, 128, 8, 256), buf.routing.topk_idx, _normal((tokens, 256), 2, 0))
        torch.cuda.synchronize()
        assert torch.equal(got["off"], buf.routing.expert_offsets)
        assert torch.equal(got["lst"], buf.routing.pair_list)


def _within(got, want, tol):
    got, want, tol = got.double().cpu(), want.cpu(), tol.cpu()
    assert bool(torch.isfinite(got).all())
    err = (got - want).abs()
    assert bool((err <= tol).all()), float((err / tol.clamp(min=1e-300)).max())


def _data(T, E, k, d, typ, kind):
    idx = _ids(T, E, k, 3 * T + d, kind)
    off, lst, pos = _places(idx, E)
    rows = _normal((T * k, d), 4, typ)
    rows[int(off[E]):] = float("nan")  # never read
    w = torch.softmax(torch.randn(T, k, generator=torch.Generator().manual_seed(5)), 1).cuda()
    p = torch.from_numpy(pos).cuda()
    there = (p >= 0)[:, :, None]
    v = torch.where(there, rows[p.clamp(min=0).long()].double(), torch.zeros((), device="cuda", dtype=torch.float64))
    return idx, p, rows, w, v


@pytest.mark.parametrize("T,E,k,d,typ,kind", CASES, ids=IDS)
def test_combine_and_dispatch_backward(B, T, E, k, d, typ, kind):
    idx, pos, rows, w, v = _data(T, E, k, d, typ, kind)
    cfg = B.make_rows(T, E, k, d, typ)
    res = _normal((T, d), 6, typ)
    for weights, residual in ((w, None), (w, res), (None, None), (None, res)):
        out = torch.full((T, d), float("nan"), dtype=TYPES[typ], device="cuda")
        if weights is None and residual is None:
            B.moe_w4a16_dispatch_backward(cfg, pos, rows, out)
        else:
            B.moe_w4a16_combine_rows(cfg, pos, weights, rows, residual, out)
        torch.cuda.synchronize()
        terms = v if weights is None else v * w.double()[:, :, None]
        want, mag = terms.sum(1), terms.abs().sum(1)
        if residual is not None:
            want, mag = want + residual.double(), mag + residual.double().abs()
        _within(out, want, HALF[typ] * want.abs() * 1.01 + (k + 1) * V * mag * 1.01 + SMALL[typ])


def test_combine_in_place_and_bad_places(B):
    """out may be the residual; places outside the rows add nothing and are not read."""
    T, E, k, d = 9, 4, 2, 72
    idx, pos, rows, w, v = _data(T, E, k, d, 0, "plain")
    cfg, res = B.make_rows(T, E, k, d, 0), _normal((T, d), 6, 0)
    out = torch.empty_like(res)
    B.moe_w4a16_combine_rows(cfg, pos, w, rows, res, out)
    same = res.clone()
    B.moe_w4a16_combine_rows(cfg, pos, w, rows, same, same)
    assert torch.equal(out, same)
    bad = pos.clone()
    bad[3, 0], bad[4, 1], bad[5, 0] = T * k, 2 ** 31 - 1, -2 ** 31
    zero = w.clone()
    zero[3, 0] = zero[4, 1] = zero[5, 0] = 0
    a, b = torch.empty_like(res), torch.empty_like(res)
    B.moe_w4a16_combine_rows(cfg, bad, w, rows, res, a)
    B.moe_w4a16_combine_rows(cfg, pos, zero, rows, res, b)
    assert torch.equal(a, b)


@pytest.mark.parametrize("T,E,k,d,typ,kind", CASES, ids=IDS)
def test_combine_backward(B, T, E, k, d, typ, kind):
    idx, pos, rows, w, v = _data(T, E, k, d, typ, kind)
    cfg, dout = B.make_rows(T, E, k, d, typ), _normal((T, d), 8, typ)
    di = torch.from_numpy(idx).cuda()
    gr = torch.full((T * k, d), 7, dtype=TYPES[typ], device="cuda")
    gw = torch.full((T, k), float("nan"), device="cuda")
    gl = torch.full((T, E), float("nan"), device="cuda")
    B.moe_w4a16_combine_rows_backward(cfg, di, pos, w, rows, dout, gr, gw, gl)
    torch.cuda.synchronize()
    D, W = dout.double(), w.double()
    there = pos >= 0
    prod = v * D[:, None, :]
    dw, per = prod.sum(2), 4 if typ == 2 else 8
    e_dw = (-(-d // per // 32) * per + 13) * V * prod.abs().sum(2) * 1.01
    _within(gw, dw, e_dw)
    want = (W[:, :, None] * D[:, None, :])
    tol = (HALF[typ] + V) * want.abs() * 1.01 + SMALL[typ]
    full, ftol = torch.full((T * k, d), 7.0, dtype=torch.float64, device="cuda"), torch.zeros(T * k, d, device="cuda", dtype=torch.float64)
    full[pos[there].long()], ftol[pos[there].long()] = want[there], tol[there]
    _within(gr, full, ftol)
    e_m = (W * e_dw).sum(1, keepdim=True) + (k + 1) * V * (W * dw).abs().sum(1, keepdim=True)
    m = (W * dw).sum(1, keepdim=True)
    sel = torch.where(there, W * (dw - m), 0 * dw)
    e_sel = torch.where(there, W * (e_dw + e_m) + 3 * V * W * (dw.abs() + m.abs()), 0 * dw) * 1.01
    dl, tl = torch.zeros(T, E, dtype=torch.float64, device="cuda"), torch.zeros(T, E, dtype=torch.float64, device="cuda")
    at = torch.where(there, di, torch.zeros_like(di)).long()
    dl.scatter_add_(1, at, sel)
    tl.scatter_add_(1, at, e_sel)
    if kind in ("twice", "one"):  # each addition of a second choice rounds once more
        tl.scatter_add_(1, at, k * V * sel.abs())
    _within(gl, dl, tl)
    # each output alone gives the same bits
    for n in range(3):
        alone = [None, None, None]
        alone[n] = torch.full_like((gr, gw, gl)[n], 7)
        B.moe_w4a16_combine_rows_backward(cfg, di if n == 2 else None, pos, w, rows, dout, *alone)
        assert torch.equal(alone[n], (gr, gw, gl)[n])


def test_gradients_against_differences(B):
    """<g, combine(x + h dx) - combine(x - h dx)> / 2h of the pair dispatch -> combine in fp32
    against the gradients' products: both maps are linear in x and in w, so the quotient is
    exact but for roundings, about 2^-24 sqrt(terms) relative to the magnitudes, over h = 1."""
    T, E, k, d = 21, 6, 3, 40
    cfg = B.make_rows(T, E, k, d, 2)
    idx = torch.from_numpy(_ids(T, E, k, 3, "drop")).cuda()
    x, dx, g = (_normal((T, d), s, 2) for s in (1, 2, 3))
    w = torch.softmax(torch.randn(T, k, generator=torch.Generator().manual_seed(4)), 1).cuda()
    dwt = torch.randn(T, k, generator=torch.Generator().manual_seed(5)).cuda()

    def f(x, w):
        dd = _dispatch(B, cfg, idx, x)
        out = torch.empty_like(x)
        B.moe_w4a16_combine_rows(cfg, dd["pos"], w, dd["rows"], None, out)
        return float((out.double() * g.double()).sum()), dd

    _, dd = f(x, w)
    gr, gw, gx = torch.zeros_like(dd["rows"]), torch.empty_like(w), torch.empty_like(x)
    B.moe_w4a16_combine_rows_backward(cfg, None, dd["pos"], w, dd["rows"], g, gr, gw, None)
    B.moe_w4a16_dispatch_backward(cfg, dd["pos"], gr, gx)
    for want, a, b, arg in ((float((gx.double() * dx.double()).sum()), (x + dx, w), (x - dx, w), dx),
                            (float((gw.double() * dwt.double()).sum()), (x, w + dwt), (x, w - dwt), dwt)):
        got = (f(*a)[0] - f(*b)[0]) / 2
        scale = float(g.double().abs().sum()) * float(x.double().abs().max() + dx.double().abs().max()) * k * 4
        assert abs(got - want) <= (k + 8) * V * scale


def test_two_streams_and_a_captured_graph(B):
    """The calls run on the stream they are given, repeat bit for bit, and a captured
    dispatch -> combine -> backward follows new inputs in its buffers."""
    T, E, k, d, typ = 700, 32, 8, 128, 1
    cfg = B.make_rows(T, E, k, d, typ)
    w = torch.softmax(torch.randn(T, k, generator=torch.Generator().manual_seed(5)), 1).cuda()
    idx, x = torch.from_numpy(_ids(T, E, k, 1, "drop")).cuda(), _normal((T, d), 1, typ)
    bufs = dict(off=torch.zeros(E + 1, dtype=torch.int32, device="cuda"),
                lst=torch.zeros(T * k, dtype=torch.int32, device="cuda"),
                pos=torch.zeros(T, k, dtype=torch.int32, device="cuda"),
                rows=torch.zeros(T * k, d, dtype=TYPES[typ], device="cuda"),
                out=torch.zeros(T, d, dtype=TYPES[typ], device="cuda"),
                gr=torch.zeros(T * k, d, dtype=TYPES[typ], device="cuda"),
                gw=torch.zeros(T, k, device="cuda"), gl=torch.zeros(T, E, device="cuda"),
                gx=torch.zeros(T, d, dtype=TYPES[typ], device="cuda"))
    ws = torch.empty(B.moe_w4a16_dispatch_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")

    def go(stream=None):
        b = bufs
        B.moe_w4a16_dispatch(cfg, idx, x, b["off"], b["lst"], b["pos"], b["rows"], ws, stream)
        B.moe_w4a16_combine_rows(cfg, b["pos"], w, b["rows"], x, b["out"], stream)
        B.moe_w4a16_combine_rows_backward(cfg, idx, b["pos"], w, b["rows"], b["out"], b["gr"], b["gw"], b["gl"], stream)
        B.moe_w4a16_dispatch_backward(cfg, b["pos"], b["gr"], b["gx"], stream)

    go()
    torch.cuda.synchronize()
    first = {n: t.clone() for n, t in bufs.items()}
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    go(other)
    other.synchronize()
    assert all(torch.equal(bufs[n], first[n]) for n in bufs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    idx2, x2 = torch.from_numpy(_ids(T, E, k, 9, "twice")).cuda(), _normal((T, d), 9, typ)
    idx.copy_(idx2)
    x.copy_(x2)
    graph.replay()
    torch.cuda.synchronize()
    replayed = {n: t.clone() for n, t in bufs.items()}
    for n in ("gr", "rows"):
        bufs[n].copy_(first[n])  # rows behind the last are left as they were
    go()
    torch.cuda.synchronize()
    assert all(torch.equal(bufs[n], replayed[n]) for n in bufs)


def test_rows_beyond_32_bits(B):
    """2^17 tokens top-8 of 2056 columns: the rows' last elements lie past 2^31, their bytes past 2^32."""
    T, E, k, d, typ = (1 << 17) + 3, 16, 8, 2056, 1
    cfg = B.make_rows(T, E, k, d, typ)
    g = torch.Generator(device="cuda").manual_seed(1)
    idx = torch.argsort(torch.rand(T, E, generator=g, device="cuda"), dim=1)[:, :k].int().contiguous()
    x = torch.randn(T, d, generator=g, device="cuda", dtype=torch.bfloat16)
    got = _dispatch(B, cfg, idx, x)
    torch.cuda.synchronize()
    order = torch.sort(idx.reshape(-1).long(), stable=True).indices
    assert torch.equal(got["lst"].long(), order)
    for part in torch.arange(T * k, device="cuda").split(1 << 17):
        assert torch.equal(got["rows"][part], x[order[part] // k])
    w = torch.rand(T, k, generator=g, device="cuda")
    out, gw = torch.empty_like(x), torch.empty_like(w)
    B.moe_w4a16_combine_rows(cfg, got["pos"], w, got["rows"], None, out)
    gr = torch.empty_like(got["rows"])
    B.moe_w4a16_combine_rows_backward(cfg, None, got["pos"], w, got["rows"], x, gr, gw, None)
    torch.cuda.synchronize()
    t = torch.tensor([0, T // 2, T - 1], device="cuda")
    want = x[t].double() * w[t].double().sum(1, keepdim=True)
    _within(out[t], want, (HALF[typ] + 9 * V) * want.abs() * 1.01)
    for r in range(k):
        want = w[t, r, None].double() * x[t].double()
        _within(gr[got["pos"][t, r].long()], want, (HALF[typ] + V) * want.abs() * 1.01)
        dw = (x[t].double() ** 2).sum(1)
        _within(gw[t, r], dw, (-(-d // 8 // 32) * 8 + 13) * V * dw * 1.01)


def test_no_tokens(B):
    cfg = B.make_rows(0, 5, 2, 64, 0)
    off = torch.full((6,), 3, dtype=torch.int32, device="cuda")
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    B.moe_w4a16_dispatch(cfg, e, torch.empty(0, 64, dtype=torch.float16, device="cuda"), off, e, e,
                         torch.empty(0, 64, dtype=torch.float16, device="cuda"),
                         torch.empty(16, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    assert bool((off == 0).all())


@pytest.mark.parametrize("T,E,k,d,typ,twice", [(5, 6, 3, 64, 2, False), (700, 32, 8, 200, 1, False), (33, 256, 8, 2056, 0, False),
                                               (260, 5, 2, 520, 2, False), (91, 9, 4, 72, 0, True), (64, 16, 1, 136, 1, False)])
def test_logit_gradients_of_dropped_choices(B, T, E, k, d, typ, twice):
    """Choices that full experts dropped, their ids still the router's: the kept weights are a
    softmax over all k chosen logits, so a dropped one has a gradient too.  Against autograd
    through softmax in 64 bits.  The kernel's weights are rounded to fp32, which adds v w
    (|dw| + 2 sum_j w_j |dw_j|) to the error of the formula in the heading."""
    idx = _ids(T, E, k, T, "twice" if twice else "plain")
    gone = np.random.default_rng(d).random((T, k)) < 0.3
    gone[0], gone[T - 1] = np.arange(k) == 0, True
    off, _, pos = _places(np.where(gone, -1, idx), E)
    pos[gone & (np.arange(k) % 2 == 1)] = T * k + 3  # any place outside the rows drops a pair
    rows, dout = _normal((T * k, d), 4, typ), _normal((T, d), 8, typ)
    rows[int(off[E]):] = float("nan")
    di, dp, kept = torch.from_numpy(idx).cuda(), torch.from_numpy(pos).cuda(), torch.from_numpy(~gone).cuda()
    logits = torch.randn(T, E, generator=torch.Generator().manual_seed(9), dtype=torch.float64).cuda().requires_grad_()
    w = torch.softmax(logits.gather(1, di.long()), 1)
    at = torch.where(kept, dp, torch.zeros_like(dp)).long()
    v = torch.where(kept[:, :, None], rows[at].double(), torch.zeros((), dtype=torch.float64, device="cuda"))
    prod = v * dout.double()[:, None, :]
    (w[:, :, None] * prod).sum().backward()
    gw, gl = torch.full((T, k), float("nan"), device="cuda"), torch.full((T, E), float("nan"), device="cuda")
    B.moe_w4a16_combine_rows_backward(B.make_rows(T, E, k, d, typ), di, dp, w.detach().float(), rows, dout, None, gw, gl)
    torch.cuda.synchronize()
    W, dw, per = w.detach(), prod.sum(2).abs(), 4 if typ == 2 else 8
    e_dw = (-(-d // per // 32) * per + 13) * V * prod.abs().sum(2)
    m = (W * dw).sum(1, keepdim=True)
    e_m = (W * e_dw).sum(1, keepdim=True) + (k + 1) * V * m
    tol = torch.zeros_like(logits).scatter_add_(1, di.long(), W * (e_dw + e_m) + (5 + (k if twice else 0)) * V * W * (dw + m))
    _within(gw, prod.sum(2), e_dw * 1.01)
    _within(gl, logits.grad, tol * 1.01)
    assert bool((gl[T - 1] == 0).all())  # all of a token's choices dropped
    if k > 1:
        assert float(gl[0, idx[0, 0]]) != 0  # one dropped, the others kept


def test_weights_of_dropped_choices_are_not_used(B):
    """Whatever lies in topk_w at a pair without an expert (padding that nobody wrote, infinities):
    the same bits as with zeros there, forwards and backwards."""
    T, E, k, d, typ = 70, 12, 4, 136, 1
    cfg = B.make_rows(T, E, k, d, typ)
    idx, pos, rows, w, _ = _data(T, E, k, d, typ, "drop")
    di, dout = torch.from_numpy(idx).cuda(), _normal((T, d), 8, typ)
    assert bool(((pos < 0).any(1) & (pos >= 0).any(1)).any())

    def go(w):
        out, gr = torch.empty_like(dout), torch.zeros_like(rows)
        gw, gl = torch.empty_like(w), torch.empty(T, E, device="cuda")
        B.moe_w4a16_combine_rows(cfg, pos, w, rows, None, out)
        B.moe_w4a16_combine_rows_backward(cfg, di, pos, w, rows, dout, gr, gw, gl)
        torch.cuda.synchronize()
        return out, gr, gw, gl

    want = go(torch.where(pos < 0, 0.0, w))
    for junk in (float("nan"), float("inf"), -1e30):
        assert all(torch.equal(a, b) for a, b in zip(go(torch.where(pos < 0, junk, w)), want))
