"""The operators around the expert layer together, as a program uses them: a training step of two blocks with norms,
gates and clipping, and a step of a block for a few tokens, against plain 64-bit forms.

Tolerances: a tensor of the chain is rounded to the type (half a step u) at most twelve times on the way to a gradient of
the first block (rows, pre-activation, h, rows back, norm, and as many backwards); at random they add as their root, a
norm or a product passes them on with a factor of about one, and the gated activation with up to two: 12 u over a whole
tensor's norm. The gradients of gates and gammas are sums over rows of those, the clipped ones the same by a factor.
"""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from w4a16_moe_expert_router_gb300 import synth  # noqa: E402

HALF = {0: 2.0 ** -11, 1: 2.0 ** -8}
TYPES = {0: torch.float16, 1: torch.bfloat16}
EPS = 1e-6


@pytest.fixture(scope="module")
def rt():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from w4a16_moe_expert_router_gb300 import build as libbuild
    libbuild.build()
    from w4a16_moe_expert_router_gb300 import runtime
    return runtime


def _rms(v):
    return v / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)


def _gelu(a):
    return a * torch.sigmoid(math.sqrt(8 / math.pi) * (a + 0.044715 * a ** 3))


def _experts(u, idx, w, gate_up, down):
    f, y = down.shape[2], 0.0
    for r in range(idx.shape[1]):
        z = torch.einsum("td,tnd->tn", u, gate_up[idx[:, r]])
        y = y + w[:, r, None] * torch.einsum("tf,tdf->td", _gelu(z[:, :f]) * z[:, f:], down[idx[:, r]])
    return y


def _close(got, want, tol):
    assert float((got.double() - want).norm() / want.norm()) <= tol


@pytest.mark.parametrize("typ", [0, 1], ids=["fp16", "bf16"])
def test_a_training_step_of_two_blocks(rt, typ):
    from w4a16_moe_expert_router_gb300 import binding as B
    T, d, f, E, k, seq = 200, 256, 128, 16, 2, 77
    g = torch.Generator(device="cuda").manual_seed(5)
    rnd = lambda *s, scale=1.0, shift=0.0: torch.randn(s, generator=g, device="cuda") * scale + shift
    dt = TYPES[typ]
    x, dout, du = rnd(T, d).to(dt), rnd(T, d).to(dt), rnd(T, d).to(dt)
    gammas = [rnd(d, scale=0.1, shift=1.0) for _ in range(5)]  # before, and after and next of each block
    gates = [rnd(-(-T // seq), d, scale=0.3, shift=0.5) for _ in range(2)]
    gu = [rnd(E, 2 * f, d, scale=d ** -0.5).to(dt) for _ in range(2)]
    dn = [rnd(E, d, f, scale=f ** -0.5).to(dt) for _ in range(2)]
    logits = [rnd(T, E) for _ in range(2)]
    blocks = [rt.Block16(T, d, f, E, k, 0, typ, gate_rows=seq, residual_scale=0.5, eps=EPS) for _ in range(2)]
    # forwards: the second block takes what the first one's call left
    u0 = blocks[0].first_norm(x, gammas[0], torch.empty_like(x))
    h, u1 = blocks[0].forward(x, u0, logits[0], gu[0], None, dn[0], gammas[1], gates[0], gammas[2])
    out, u2 = blocks[1].forward(h, u1, logits[1], gu[1], None, dn[1], gammas[3], gates[1], gammas[4])
    # and back
    g1 = blocks[1].backward(dout, du)
    g0 = blocks[0].backward(g1["x"], g1["u"])
    grad_gamma, grad_x = torch.empty_like(gammas[0]), torch.empty_like(x)
    blocks[0].first_norm_backward(x, gammas[0], g0["x"], g0["u"], grad_x, grad_gamma)
    names = ("gate_up", "down", "gamma_post", "gate", "gamma_next")
    learned = [grad_gamma] + [q[n] for q in (g0, g1) for n in names]
    before = [t.clone() for t in learned]
    norm = float(blocks[0].clip(learned, 1.0))
    # the same in 64 bits on the routing that the blocks took
    X, GA, GT = x.double().requires_grad_(), [v.double().requires_grad_() for v in gammas], [v.double().requires_grad_() for v in gates]
    GU, DN = [v.double().requires_grad_() for v in gu], [v.double().requires_grad_() for v in dn]
    L = [v.double().requires_grad_() for v in logits]
    H, U = X, GA[0] * _rms(X)
    row = torch.arange(T, device="cuda") // seq
    for i in range(2):
        idx = blocks[i].layer.routing.topk_idx.long()
        w = torch.softmax(torch.gather(L[i], 1, idx), 1)
        y = _experts(U, idx, w, GU[i], DN[i])
        H = 0.5 * H + GT[i][row] * GA[1 + 2 * i] * _rms(y)
        U = GA[2 + 2 * i] * _rms(H)
    ((H * dout.double()).sum() + (U * du.double()).sum()).backward()
    u = HALF[typ]
    _close(out, H.detach(), 12 * u)
    _close(u2, U.detach(), 12 * u)
    _close(grad_x, X.grad, 12 * u)
    for q, i in ((g0, 0), (g1, 1)):
        _close(q["logits"], L[i].grad, 12 * u)
    want = [GA[0].grad] + [v for i in range(2) for v in (GU[i].grad, DN[i].grad, GA[1 + 2 * i].grad, GT[i].grad, GA[2 + 2 * i].grad)]
    total = math.sqrt(sum(float((v * v).sum()) for v in want))
    assert abs(norm - total) <= 12 * u * total and norm > 1.0
    for got, was, ref in zip(learned, before, want):
        _close(was, ref, 12 * u)
        _close(got, ref / total, 24 * u)
    assert B.moe_w4a16_read_error(blocks[0].layer.ws[2]) == B.OK


def test_a_step_replays_and_its_gradients_do_not_change(rt):
    """Forward, backward and clipping captured into a graph, and run eagerly: the same bits."""
    T, d, f, E, k = 130, 128, 64, 8, 2
    g = torch.Generator(device="cuda").manual_seed(6)
    rnd = lambda *s, scale=1.0, shift=0.0: torch.randn(s, generator=g, device="cuda") * scale + shift
    x, dout = rnd(T, d).half(), rnd(T, d).half()
    gu, dn, logits = rnd(E, 2 * f, d, scale=0.1).half(), rnd(E, d, f, scale=0.1).half(), rnd(T, E)
    post, pre, gate = rnd(d, scale=0.1, shift=1.0), rnd(d, scale=0.1, shift=1.0), rnd(1, d)
    block = rt.Block16(T, d, f, E, k, gate_rows=T)
    u, gx, gg = torch.empty_like(x), torch.empty_like(x), torch.empty_like(pre)

    def step():
        block.first_norm(x, pre, u)
        block.forward(x, u, logits, gu, None, dn, post, gate, None)
        q = block.backward(dout, None)
        block.first_norm_backward(x, pre, q["x"], q["u"], gx, gg)
        grads = [q["gate_up"], q["down"], q["gamma_post"], q["gate"], gg]
        block.clip(grads, 0.5)
        return [block.out, gx, block.grad_norm, *grads]

    first = [t.clone() for t in step()]
    again = [t.clone() for t in step()]
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for t in outs:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, outs))


@pytest.mark.parametrize("tokens", [1, 3, 16])
def test_a_block_for_a_few_tokens(rt, tokens):
    """Pre-norm and router of the W4A16 block, the whole layer, and the norm after it with the residual."""
    from w4a16_moe_expert_router_gb300 import binding as B
    from test_gpu_few import _weights
    wl = synth.Workload("few", tokens, 512, 320, 24, 4, 64, 64)
    host = synth.make_weights(wl)
    w, buf = rt.upload_weights(wl, host), rt.alloc_few(wl, tokens)
    x = rt.to_device_x(synth.make_x(wl))
    gamma, router = rt.to_device_f32(synth.make_gamma_pre(wl)), rt.to_device_x(synth.make_router(wl))
    post, gate = rt.to_device_f32(synth.make_gamma(wl)), torch.full((1, 512), 0.75, device="cuda")
    u, logits = torch.empty_like(x), torch.empty(tokens, 24, device="cuda")
    out, nxt = torch.empty_like(x), torch.empty_like(x)
    B.moe_w4a16_block_front(buf.shape, x, gamma, EPS, router, u, logits)
    y = rt.run_few(buf, u, logits, w)
    cfg = B.make_norm(tokens, 512, 0, tokens, 1.0, EPS)
    B.moe_w4a16_norm(cfg, x, y, post, gate, gamma, out, nxt)
    torch.cuda.synchronize()
    U = (gamma.double() * _rms(x.double()))
    idx = buf.topk_idx.long()
    W = torch.softmax(torch.gather(U @ router.double().T, 1, idx), 1)
    mats = [sum(_weights(host, part, 64, 0)) for part in ("gate_up", "down")]
    Y = _experts(U, idx, W, *mats)
    O = x.double() + 0.75 * post.double() * _rms(Y)
    _close(buf.topk_w, W, 12 * HALF[0])
    _close(out, O, 12 * HALF[0])
    _close(nxt, gamma.double() * _rms(O), 12 * HALF[0])
