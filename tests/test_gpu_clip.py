"""The norm over a list of tensors and their scaling, against 64-bit sums.

Tolerances, u the half step of a tensor's type (2^-11 fp16, 2^-8 bf16, 2^-24 fp32), v = 2^-24: an fp32 sum holds at
most 64 squares, eight chained and eight added, so a relative 16 v at most, the terms being positive; the root halves
it, and fp64 adds nothing that counts: 8 v and the last rounding, 9 v. The factor has one rounding more, a product one
of its own, and the rounding to the type u (half of fp16's smallest step).
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

V = 2.0 ** -24
HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
SMALL = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}
F16, B16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from w4a16_moe_expert_router_gb300 import build as libbuild
    libbuild.build()
    from w4a16_moe_expert_router_gb300 import binding
    return binding


def _tensors(sizes, types, seed=0, scale=1.0, pad=None):
    """Tensors of normal values; pad: each starts that many elements into a buffer of its own."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        off = 0 if pad is None else pad[i % len(pad)]
        whole = torch.full((n + off + 16,), 7.0, device="cuda", dtype=types[i % len(types)])
        whole[off:off + n] = torch.randn(n, generator=g, device="cuda") * scale
        out.append(whole[off:off + n])
    return out


def _clip(B, tensors, max_norm, outs=None, stream=None):
    lst = B.make_tensors(tensors, outs)
    norm = torch.full((1,), -7.0, device="cuda")
    ws = torch.full((B.moe_w4a16_clip_workspace_bytes(lst),), 255, dtype=torch.uint8, device="cuda")
    B.moe_w4a16_clip(lst, max_norm, norm, ws, stream)
    return norm


def _norm(tensors):
    return math.sqrt(math.fsum(float((t.double() ** 2).sum()) for t in tensors))


def _check(got, before, factor):
    for o, t in zip(got, before):
        ref = t.double() * factor
        lim = (11 * V + HALF[t.dtype]) * ref.abs() + SMALL[t.dtype]
        assert bool(((o.double() - ref).abs() <= lim).all())


SIZES = [[1], [0], [], [7, 0, 1, 8, 9, 15, 17], [16384, 16385, 8192, 8191], [1 << 20, 3], [100003, 5, 70001],
         list(range(1, 130)), [33] * 700]


@pytest.mark.parametrize("types", [[F16], [B16], [F32], [B16, F32, F16]], ids=["fp16", "bf16", "fp32", "mixed"])
@pytest.mark.parametrize("sizes", SIZES, ids=[str(i) for i in range(len(SIZES))])
@pytest.mark.parametrize("pad", [None, [1, 3, 0, 7]], ids=["aligned", "odd"])
def test_norm_and_scaling(B, sizes, types, pad):
    tensors = _tensors(sizes, types, 1, pad=pad)
    before = [t.clone() for t in tensors]
    want = _norm(tensors)
    for where in ("copy", "odd copy", "in place"):
        outs = None if where == "in place" else _tensors(sizes, types, 2, pad=pad if where == "copy" else [2, 5, 1])
        norm = _clip(B, tensors, 0.3 * want, outs)
        assert abs(float(norm) - want) <= 9 * V * want
        _check(tensors if outs is None else outs, before, 0.3 if want else 1.0)
        if outs is not None:
            assert all(torch.equal(a, b) for a, b in zip(tensors, before))
            for o in outs:  # what lies around an output stays as it was
                whole = o._base if o._base is not None else o
                off = o.storage_offset()
                assert bool((whole[:off] == 7).all()) and bool((whole[off + o.numel():] == 7).all())


@pytest.mark.parametrize("kind", ["below", "equal", "infinite bound"])
def test_below_the_bound_the_bits_stay(B, kind):
    tensors = _tensors([1000, 77, 9001], [B16, F32, F16], 3, pad=[0, 1, 3])
    before = [t.clone() for t in tensors]
    norm = _clip(B, tensors, math.inf)
    bound = {"below": 1.5 * float(norm), "equal": None, "infinite bound": math.inf}[kind]
    if bound is None:  # the norm itself: a list whose norm is known exactly
        tensors = [torch.full((16,), 2.0, device="cuda"), torch.full((12,), 3.0, device="cuda", dtype=F16),
                   torch.full((9,), 4.0, device="cuda", dtype=B16)]  # 64 + 108 + 144 + .. = 316 + 5
        tensors.append(torch.tensor([2.0, 2.0], device="cuda"))      # 8: 324 = 18^2
        before, bound = [t.clone() for t in tensors], 18.0
        norm = _clip(B, tensors, bound)
        assert float(norm) == 18.0
    outs = [torch.full_like(t, 7) for t in tensors]
    _clip(B, tensors, bound, outs)
    assert all(torch.equal(a, b) for a, b in zip(outs, before))
    _clip(B, tensors, bound)
    assert all(torch.equal(a, b) for a, b in zip(tensors, before))


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("dtype", [F16, B16, F32], ids=["fp16", "bf16", "fp32"])
def test_a_norm_that_is_no_number_scales_nothing(B, dtype, bad):
    tensors = _tensors([50, 40000], [dtype], 4)
    tensors[1][39999] = bad
    before = [t.clone() for t in tensors]
    norm = _clip(B, tensors, 1.0)
    assert math.isnan(float(norm)) if math.isnan(bad) else float(norm) == math.inf
    outs = [torch.zeros_like(t) for t in tensors]
    _clip(B, tensors, 1.0, outs)
    for a, b, c in zip(tensors, outs, before):
        view = torch.int32 if dtype is F32 else torch.int16
        assert torch.equal(a.view(view), c.view(view)) and torch.equal(b.view(view), c.view(view))


@pytest.mark.parametrize("dtype,scale", [(F32, 1e30), (F32, 1e-30), (B16, 1e25), (B16, 1e-25), (F32, 1e19), (F32, 2e-23),
                                         (F16, 6e4), (F16, 6e-8)])
def test_values_whose_squares_leave_fp32(B, dtype, scale):
    g = torch.Generator(device="cuda").manual_seed(5)
    v = (torch.rand(30011, generator=g, device="cuda", dtype=torch.float64) * scale).to(dtype)
    tensors = [v[1:], torch.zeros(5000, device="cuda", dtype=dtype), v[:9].clone()]
    before = [t.clone() for t in tensors]
    want = _norm(tensors)
    if want > 3e38:
        pytest.skip("the norm itself is out of range")
    outs = [torch.empty_like(t) for t in tensors]
    norm = _clip(B, tensors, 0.5 * want, outs)
    assert abs(float(norm) - want) <= 9 * V * want + 2.0 ** -150
    _check(outs, before, 0.5)


def test_zeros_and_a_bound_of_zero(B):
    tensors = [torch.zeros(3000, device="cuda"), torch.zeros(11, device="cuda", dtype=F16)]
    assert float(_clip(B, tensors, 0.0)) == 0.0 and not any(bool(t.any()) for t in tensors)
    tensors = _tensors([3000, 11], [F32, F16], 6)
    assert float(_clip(B, tensors, 0.0)) > 0 and not any(bool(t.any()) for t in tensors)


def test_tensors_that_only_count(B):
    tensors = _tensors([4000, 300], [F32], 7)
    before = [t.clone() for t in tensors]
    want = _norm(tensors)
    out = torch.empty_like(tensors[0])
    _clip(B, tensors, 0.25 * want, [out, None])
    _check([out], before[:1], 0.25)
    assert torch.equal(tensors[1], before[1])


def test_the_same_bits_in_every_run_and_in_a_replayed_graph(B):
    tensors = _tensors([123457, 99, 40000, 1], [B16, F32], 8, pad=[0, 3])
    outs = [torch.empty_like(t) for t in tensors]
    lst = B.make_tensors(tensors, outs)
    norm = torch.empty(1, device="cuda")
    ws = torch.empty(B.moe_w4a16_clip_workspace_bytes(lst), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    B.moe_w4a16_clip(lst, 1.0, norm, ws, side)
    side.synchronize()
    first, first_norm = [o.clone() for o in outs], norm.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.moe_w4a16_clip(lst, 1.0, norm, ws)
    for o in outs:
        o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(norm, first_norm) and all(torch.equal(a, b) for a, b in zip(outs, first))
    tensors[0].mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    want = _norm(tensors)
    assert abs(float(norm) - want) <= 9 * V * want


def test_an_element_past_32_bits_of_offset(B):
    n = (1 << 32) + 5  # bf16: 8.6 GB
    t = torch.zeros(n, device="cuda", dtype=B16)
    t[n - 1] = 3.0
    t[0] = 4.0
    assert float(_clip(B, [t], 2.5)) == 5.0
    assert float(t[n - 1]) == 1.5 and float(t[0]) == 2.0


@pytest.mark.parametrize("count", [64, 65, 640, 641, 1300])
def test_lists_of_views_of_one_buffer(B, count):
    """Tensors end to end, wherever that puts them, scaled in place; the list is as long as a launch takes, or longer."""
    g = torch.Generator().manual_seed(count)
    sizes = torch.randint(0, 3000, (count,), generator=g).tolist()
    flat = torch.randn(sum(sizes) + 2, device="cuda").to(B16)
    before = flat.clone()
    tensors = list(torch.split(flat[1:-1], sizes))
    want = _norm([before[1:-1]])
    norm = _clip(B, tensors, 0.5 * want)
    assert abs(float(norm) - want) <= 9 * V * want
    _check([flat[1:-1]], [before[1:-1]], 0.5)
    assert float(flat[0]) == float(before[0]) and float(flat[-1]) == float(before[-1])


def test_a_list_of_nothing(B):
    for tensors in ([], [torch.empty(0, device="cuda")] * 3, [torch.empty(0, device="cuda")] * 700):
        assert float(_clip(B, tensors, 1.0)) == 0.0


def test_two_calls_at_once(B):
    """On two streams, each with a workspace of its own."""
    lists = [_tensors([90001, 7, 300], [B16, F32], 11), _tensors([5, 1000], [F32], 12)]
    outs = [[torch.empty_like(t) for t in lst] for lst in lists]
    want = [(_clip(B, lst, 0.5, out).clone(), [o.clone() for o in out]) for lst, out in zip(lists, outs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in lists]
    got = []
    for _ in range(10):
        for lst, s in zip(lists, streams):
            with torch.cuda.stream(s):
                new = [torch.empty_like(t) for t in lst]
                got.append((_clip(B, lst, 0.5, new), new))
    torch.cuda.synchronize()
    for i, (norm, new) in enumerate(got):
        assert torch.equal(norm, want[i % 2][0]) and all(torch.equal(a, b) for a, b in zip(new, want[i % 2][1]))
