"""The whole layer for a few tokens against a plain 64-bit form.

Tolerances, u the half step of the tokens' type (2^-11 fp16, 2^-8 bf16), t = 2^-23 the step of fp32. Products of codes
and tokens are exact in fp32; the sums of a group's G products, of its zero-point's term, of the K / G groups and of
at most eight warps are each off by at most a step of a partial sum, at most A = sum (s q + |c|) |x| in all: (G + K / G
+ 12) t A. The activation changes by at most 1.13 times its argument's error and is good to 2^-17 of its value;
h is kept to 2^-22 of it (fp16, or 2^-25) or 2^-16 (bf16). The router's weights are good to 8 v, v = 2^-24, a
token's k shares and the warps' sums add (k + 12) v of the shares' magnitudes, and the one rounding to the type u of the
result, or half of fp16's smallest step. Those worst cases add up over a thousand terms, so the whole output is also held
to what they come to at random: its difference, over its norm, is at most u, the one rounding, plus 2^-14 (bf16: h's
2^-16, twice, and the activation) or 2^-15.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from w4a16_moe_expert_router_gb300 import synth  # noqa: E402

T23, V = 2.0 ** -23, 2.0 ** -24
TYPES = {0: torch.float16, 1: torch.bfloat16}
HALF = {0: 2.0 ** -11, 1: 2.0 ** -8}
SMALL = {0: 2.0 ** -25, 1: 0.0}
KEPT = {0: 2.0 ** -22, 1: 2.0 ** -16}
RANDOM = {0: 2.0 ** -15, 1: 2.0 ** -14}


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from w4a16_moe_expert_router_gb300 import build as libbuild
    libbuild.build()
    from w4a16_moe_expert_router_gb300 import binding
    return binding


def _weights(w, part, group, fmt):
    """Scale, code and offset of every weight [E][rows][cols]: w = s q + c."""
    q = torch.from_numpy(w[part + "_q"]).cuda()
    codes = torch.stack([q & 15, q >> 4], -1).reshape(*q.shape[:2], -1).double()
    s = torch.from_numpy(w[part + "_scale"].view(np.float16)).cuda().double().repeat_interleave(group, 2)
    z = torch.from_numpy(w[part + "_zero"].view(np.float16)).cuda().double().repeat_interleave(group, 2)
    return s * codes, z if fmt == 1 else -s * z


def _gelu(a, kind):
    if kind == 1:
        return a * torch.special.ndtr(a)
    return a * torch.sigmoid(1.5957691216057308 * (a + 0.044715 * a ** 3))


class Layer:
    def __init__(self, B, T, d, f, E, k, g1, g2, fmt, act, typ, seed=0, logits=None, residual=True, x_scale=1.0):
        from w4a16_moe_expert_router_gb300 import runtime
        self.B, self.typ, self.k = B, typ, k
        self.wl = synth.Workload("few", T, d, f, E, k, g1, g2, activation=act, format=fmt)
        w = synth.make_weights(self.wl, seed)
        self.host, self.shape = w, runtime.shape_of(self.wl)
        self.dev = runtime.upload_weights(self.wl, w)
        g = torch.Generator(device="cuda").manual_seed(seed + 1)
        new = lambda *shape: torch.randn(shape, generator=g, device="cuda", dtype=torch.float64)
        self.x = (new(T, d) * x_scale).to(TYPES[typ])
        self.logits = new(T, E).float() if logits is None else logits
        self.residual = new(T, d).to(TYPES[typ]) if residual else None

    def run(self, tokens=None, stream=None, out=None):
        B, sh = self.B, self.shape
        sel = slice(None) if tokens is None else tokens
        x, lg = self.x[sel].contiguous(), self.logits[sel].contiguous()
        res = None if self.residual is None else self.residual[sel].contiguous()
        T = x.shape[0]
        shape = B.make_shape(T, sh.hidden, sh.inter, sh.experts, sh.top_k, sh.group_gate_up, sh.group_down,
                             sh.activation, 0, sh.format)
        idx = torch.full((T, self.k), -7, dtype=torch.int32, device="cuda")
        tw = torch.full((T, self.k), -7.0, device="cuda")
        out = torch.full_like(x, 7) if out is None else out
        ws = torch.full((B.moe_w4a16_few_workspace_bytes(shape),), 255, dtype=torch.uint8, device="cuda")
        B.moe_w4a16_few(shape, self.typ, x, lg, self.dev.gate_up, self.dev.down, res, idx, tw, out, ws, stream)
        return idx, tw, out

    def want(self):
        """Choice, weights, output in 64 bits and what the output may be off by before its rounding."""
        wl, T = self.wl, self.x.shape[0]
        f, k, act = wl.inter, wl.top_k, wl.activation
        lg = self.logits.double()
        order = torch.argsort(lg, dim=1, descending=True, stable=True)[:, :k]
        tw = torch.softmax(torch.gather(lg, 1, order), 1)
        gq, gc = _weights(self.host, "gate_up", wl.group_gate_up, wl.format)
        dq, dc = _weights(self.host, "down", wl.group_down, wl.format)
        x = self.x.double()
        out, lim = torch.zeros_like(x), torch.zeros_like(x)
        n1 = (wl.group_gate_up + wl.hidden / wl.group_gate_up + 12) * T23
        n2 = (wl.group_down + f / wl.group_down + 12) * T23
        for r in range(k):
            e = order[:, r]
            a = torch.einsum("td,tnd->tn", x, gq[e] + gc[e])
            ea = n1 * torch.einsum("td,tnd->tn", x.abs(), gq[e] + gc[e].abs())
            act_g = _gelu(a[:, :f], act)
            h = act_g * a[:, f:]
            eh = 1.13 * ea[:, :f] * (a[:, f:].abs() + ea[:, f:]) + act_g.abs() * ea[:, f:] + \
                (KEPT[self.typ] + 2.0 ** -17) * h.abs() + (2.0 ** -25 if self.typ == 0 else 0.0)
            y = torch.einsum("tf,tdf->td", h, dq[e] + dc[e])
            ey = torch.einsum("tf,tdf->td", eh, (dq[e] + dc[e]).abs()) + \
                n2 * torch.einsum("tf,tdf->td", h.abs() + eh, dq[e] + dc[e].abs())
            out += tw[:, r, None] * y
            lim += tw[:, r, None] * (ey + (8 + k + 12) * V * y.abs())
        if self.residual is not None:
            out = out + self.residual.double()
            lim = lim + V * out.abs()
        return order, tw, out, lim

    def check(self, got):
        idx, tw, out = got
        w_idx, w_tw, w_out, lim = self.want()
        u = HALF[self.typ]
        assert torch.equal(idx.long(), w_idx)
        assert bool(((tw.double() - w_tw).abs() <= 8 * V * w_tw).all())
        err = (out.double() - w_out).abs()
        bound = lim + u * (w_out.abs() + lim) + SMALL[self.typ]
        assert bool((err <= bound).all()), float((err - bound).max())
        assert float((out.double() - w_out).norm() / w_out.norm()) <= u + RANDOM[self.typ]


CASES = [  # T, d, f, E, k, g1, g2, format, activation, type
    (1, 128, 64, 1, 1, 128, 64, 0, 0, 0), (1, 2048, 704, 128, 8, 64, 64, 0, 0, 0), (2, 256, 128, 8, 2, 64, 128, 1, 1, 1),
    (3, 384, 192, 5, 3, 32, 32, 2, 0, 0), (4, 1152, 448, 60, 3, 32, 64, 2, 1, 1), (5, 640, 320, 256, 8, 128, 64, 0, 0, 1),
    (7, 128, 1024, 129, 7, 32, 128, 1, 0, 0), (8, 2048, 704, 128, 8, 128, 64, 1, 0, 1), (9, 256, 64, 3, 3, 64, 32, 0, 1, 0),
    (16, 1024, 512, 128, 8, 64, 64, 0, 0, 0), (17, 512, 576, 31, 5, 128, 64, 2, 0, 1), (31, 256, 256, 7, 4, 64, 64, 0, 0, 0),
    (1, 4096, 192, 3, 2, 64, 32, 1, 0, 1), (2, 2048, 704, 128, 8, 64, 64, 2, 0, 0), (3, 256, 1600, 8, 2, 64, 64, 0, 0, 0),
    (12, 512, 2048, 6, 3, 128, 128, 1, 0, 1), (16, 2048, 704, 128, 8, 64, 64, 0, 0, 1), (20, 4096, 512, 48, 4, 64, 64, 0, 1, 0),
    (24, 2048, 256, 200, 8, 32, 32, 0, 0, 0), (32, 384, 128, 255, 8, 32, 128, 1, 1, 1), (32, 1280, 832, 16, 8, 64, 32, 0, 0, 0), (6, 8192, 128, 4, 2, 128, 64, 0, 0, 0),
]
IDS = ["-".join(map(str, c)) for c in CASES]


@pytest.mark.parametrize("residual", [False, True], ids=["", "residual"])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_few_matches_the_definition(B, case, residual):
    layer = Layer(B, *case, seed=sum(case), residual=residual)
    got = layer.run()
    layer.check(got)
    again = layer.run()
    assert all(torch.equal(a, b) for a, b in zip(got, again))  # the same bits in every run


@pytest.mark.parametrize("typ", [0, 1], ids=["fp16", "bf16"])
@pytest.mark.parametrize("T", [3, 9, 32])
def test_all_tokens_choose_the_same_experts(B, T, typ):
    logits = torch.full((T, 20), -3.0, device="cuda")
    logits[:, 11], logits[:, 4], logits[:, 19] = 2.0, 1.0, 1.5
    layer = Layer(B, T, 256, 192, 20, 3, 64, 64, 0, 0, typ, seed=T, logits=logits)
    layer.check(layer.run())


def test_equal_logits_go_to_the_lower_expert(B):
    logits = torch.zeros(4, 200, device="cuda")
    logits[1] = -0.0
    logits[2, 150:] = 1.0
    logits[3, ::2] = 5.0
    layer = Layer(B, 4, 256, 64, 200, 8, 64, 64, 0, 0, 0, logits=logits)
    got = layer.run()
    layer.check(got)
    assert got[0].tolist() == [list(range(8)), list(range(8)), list(range(150, 158)), list(range(0, 16, 2))]


@pytest.mark.parametrize("typ", [0, 1], ids=["fp16", "bf16"])
def test_a_token_does_not_depend_on_the_others(B, typ):
    layer = Layer(B, 32, 512, 320, 24, 4, 64, 64, 0, 0, typ)
    whole = layer.run()
    for tokens in (slice(0, 1), slice(5, 14), slice(31, 32), slice(8, 32)):
        part = layer.run(tokens)
        assert all(torch.equal(a[tokens], b) for a, b in zip(whole, part))
    # the sizes for which the layer's contraction is shared in several ways
    for d, f, E, k in ((2048, 704, 128, 8), (1152, 448, 60, 3), (384, 1600, 16, 2)):
        big = Layer(B, 32, d, f, E, k, 64, 64, 0, 0, typ, residual=False)
        whole_big = big.run()
        for tokens in (slice(0, 1), slice(3, 5), slice(7, 11), slice(0, 16), slice(1, 18)):
            assert all(torch.equal(a[tokens], b) for a, b in zip(whole_big, big.run(tokens)))
    layer.x[7] = float("inf")  # nor on what is no number there
    layer.x[8] = float("nan")
    broken = layer.run()
    keep = [t for t in range(32) if t not in (7, 8)]
    assert torch.equal(broken[2][keep], whole[2][keep])
    assert not bool(torch.isfinite(broken[2][7:9]).any())


def test_the_choice_is_that_of_route(B):
    from w4a16_moe_expert_router_gb300 import runtime
    layer = Layer(B, 32, 256, 64, 128, 8, 64, 64, 0, 0, 0)
    idx, tw, _ = layer.run()
    buf = runtime.alloc_buffers(layer.wl)
    B.moe_w4a16_route(buf.shape, layer.logits, buf.routing, buf.workspace)
    assert torch.equal(buf.routing.topk_idx, idx) and torch.equal(buf.routing.topk_w, tw)


def test_optional_outputs_and_a_residual_in_place(B):
    layer = Layer(B, 5, 256, 128, 8, 2, 64, 64, 0, 0, 0)
    _, _, want = layer.run()
    out = layer.residual.clone()
    ws = torch.empty(B.moe_w4a16_few_workspace_bytes(layer.shape), dtype=torch.uint8, device="cuda")
    B.moe_w4a16_few(layer.shape, 0, layer.x, layer.logits, layer.dev.gate_up, layer.dev.down, out, None, None, out, ws)
    assert torch.equal(out, want)


def test_streams_and_a_replayed_graph_with_new_inputs(B):
    layer = Layer(B, 6, 1024, 320, 32, 4, 64, 64, 0, 0, 0)
    other = Layer(B, 6, 1024, 320, 32, 4, 64, 64, 0, 0, 0, seed=0, x_scale=2.0)
    want, want_other = layer.run(), other.run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = layer.run()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    out = torch.zeros_like(layer.x)
    ws = torch.empty(B.moe_w4a16_few_workspace_bytes(layer.shape), dtype=torch.uint8, device="cuda")
    x, logits = layer.x.clone(), layer.logits.clone()
    graph = torch.cuda.CUDAGraph()
    call = lambda: B.moe_w4a16_few(layer.shape, 0, x, logits, layer.dev.gate_up, layer.dev.down, layer.residual, None,
                                   None, out, ws)
    call()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        for _ in range(3):
            call()
    for src, ref in ((other, want_other), (layer, want), (other, want_other)):
        x.copy_(src.x)
        logits.copy_(src.logits)
        layer.residual.copy_(src.residual)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref[2])


@pytest.mark.parametrize("case", [(1, 128, 64, 256, 8, 128, 64, 0, 0, 0), (1, 256, 64, 129, 3, 64, 32, 1, 1, 1),
                                  (4, 256, 128, 9, 8, 64, 64, 2, 0, 1), (2, 512, 2048, 200, 8, 64, 64, 0, 0, 0),
                                  (4, 8192, 64, 40, 6, 128, 64, 0, 0, 1)], ids=lambda c: "-".join(map(str, c)))
def test_few_tokens_over_many_and_few_experts(B, case):
    layer = Layer(B, *case, seed=sum(case))
    layer.check(layer.run())


@pytest.mark.parametrize("E", [5, 128, 200, 256])
def test_equal_logits_of_a_single_token(B, E):
    for k in (1, 4, 5):
        for logits in (torch.zeros(1, E), torch.arange(E).float()[None] // 3, -torch.arange(E).float()[None] % 4):
            layer = Layer(B, 1, 128, 64, E, k, 64, 64, 0, 0, 0, logits=logits.cuda().contiguous())
            layer.check(layer.run())


@pytest.mark.parametrize("T", [1, 3, 4, 13])
def test_logits_that_are_no_numbers_choose_in_bounds(B, T):
    """Their choice is unspecified; it is one of k experts of the layer, each once, and leaves other tokens alone."""
    layer = Layer(B, T, 256, 128, 40, 6, 64, 64, 0, 0, 1)
    want = layer.run()
    for value in (float("nan"), float("inf"), -float("inf")):
        for part in (slice(0, 40), slice(0, 37), slice(3, 9)):
            kept = layer.logits[T - 1].clone()
            layer.logits[T - 1, part] = value
            idx, _, out = layer.run()
            layer.logits[T - 1] = kept
            row = idx[T - 1].tolist()
            assert len(set(row)) == 6 and min(row) >= 0 and max(row) < 40
            assert torch.equal(out[:T - 1], want[2][:T - 1]) and torch.equal(idx[:T - 1], want[0][:T - 1])


def test_two_calls_at_once(B):
    """On two streams, each with a workspace of its own."""
    layers = [Layer(B, T, 1024, 320, 32, 4, 64, 64, 0, 0, 0, seed=T) for T in (1, 5)]
    want = [layer.run() for layer in layers]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(20):
        for layer, s in zip(layers, streams):
            with torch.cuda.stream(s):
                got.append(layer.run())
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % 2]))


@pytest.mark.parametrize("typ", [0, 1], ids=["fp16", "bf16"])
@pytest.mark.parametrize("d,f,E,k,fmt", [(512, 256, 200, 8, 0), (1024, 128, 196, 7, 1), (384, 384, 152, 8, 2), (256, 448, 128, 6, 0)])
def test_many_experts_of_a_small_layer(B, d, f, E, k, fmt, typ):
    """More items than one set of CTAs takes: the same bits as for a token alone."""
    layer = Layer(B, 32, d, f, E, k, 64, 64, fmt, 0, typ, seed=d)
    whole = layer.run()
    layer.check(whole)
    for tokens in (slice(0, 1), slice(3, 5), slice(7, 11), slice(0, 16), slice(1, 23)):
        assert all(torch.equal(a[tokens], b) for a, b in zip(whole, layer.run(tokens)))


@pytest.mark.parametrize("case", [(1, 8192, 8192, 2, 2, 128, 128, 0, 0, 0), (32, 128, 8192, 3, 2, 64, 32, 1, 0, 1),
                                  (32, 8192, 1024, 4, 4, 32, 32, 2, 0, 1), (3, 4096, 4096, 6, 2, 64, 64, 0, 1, 0),
                                  (32, 8192, 64, 9, 8, 32, 32, 0, 0, 0)], ids=lambda c: "-".join(map(str, c)))
def test_few_tokens_of_large_layers(B, case):
    layer = Layer(B, *case, seed=sum(case))
    whole = layer.run()
    layer.check(whole)
    assert all(torch.equal(a[:1], b) for a, b in zip(whole, layer.run(slice(0, 1))))


@pytest.mark.parametrize("typ", [0, 1], ids=["fp16", "bf16"])
@pytest.mark.parametrize("fmt", [0, 1, 2])
def test_tokens_of_one_sign(B, typ, fmt):
    """The sums of the tokens are as large as they get, and the zero-points take most of the products back."""
    for T, d, f, g in ((2, 2048, 704, 64), (8, 512, 256, 128), (5, 4096, 128, 32)):
        layer = Layer(B, T, d, f, 16, 4, g, min(g, 64), fmt, 0, typ, seed=T)
        layer.x = layer.x.abs() + 1
        layer.check(layer.run())
