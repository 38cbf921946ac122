"""Host-only tests of the operators around the layer (the whole layer for a few tokens, the norms around a block,
gradient clipping): configurations, pointers and workspaces are checked before a GPU is touched."""
import ctypes
import math
import os
import subprocess

import pytest

from w4a16_moe_expert_router_gb300 import binding as B
from w4a16_moe_expert_router_gb300 import build as libbuild

torch = pytest.importorskip("torch")
P = 4096  # an aligned address that no call here reads


@pytest.fixture(scope="session", autouse=True)
def built_library():
    libbuild.build()
    return B.lib()


# ------------------------------------------------------------------ a few tokens

FEW = dict(tokens=4, hidden=256, inter=128, experts=8, top_k=2, group_gate_up=64, group_down=64, activation=0,
           reduction=0, format=0)


def _few(type=0, ws_bytes=1 << 30, cfg=None, **null):
    """The call on stand-in addresses; null[name] replaces one.  Only calls that are refused are made: the addresses
    are no memory."""
    a = {n: P for n in ("x", "logits", "gate_up", "down", "res", "idx", "w", "out", "ws")}
    a.update(null)
    shape = B.make_shape(**{**FEW, **(cfg or {})})
    weights = B.Weights(a["gate_up"], a["down"])
    return B.lib().moe_w4a16_few(ctypes.byref(shape), type, a["x"], a["logits"], ctypes.byref(weights), a["res"],
                                 a["idx"], a["w"], a["out"], a["ws"], ws_bytes, None)


@pytest.mark.parametrize("bad", [dict(tokens=-1), dict(tokens=33), dict(hidden=192), dict(hidden=8320), dict(inter=96),
                                 dict(experts=257), dict(top_k=9, experts=16), dict(top_k=9), dict(group_gate_up=16),
                                 dict(group_down=128, inter=192), dict(activation=2), dict(format=3)])
def test_few_shapes_refused(bad):
    assert _few(cfg=bad) == B.ERR_SHAPE
    assert B.moe_w4a16_few_workspace_bytes(B.make_shape(**{**FEW, **bad})) == 0


def test_few_arguments_refused():
    assert _few(type=2) == _few(type=-1) == B.ERR_SHAPE
    for n in ("x", "logits", "gate_up", "down", "out", "ws"):
        assert _few(**{n: None}) == B.ERR_NULL, n
    for n in ("x", "logits", "gate_up", "down", "res", "idx", "w", "out", "ws"):
        assert _few(**{n: P + 8}) == B.ERR_ALIGN, n
    need = B.moe_w4a16_few_workspace_bytes(B.make_shape(**FEW))
    pair = 2 * 128 * 2 + 128 // 8 * 4  # (hi, lo) x f in 16 bits, sums of eight columns
    more = B.moe_w4a16_few_workspace_bytes(B.make_shape(**{**FEW, "tokens": 5}))
    assert more - need == 2 * pair and need > 4 * 2 * pair  # and the lists
    assert _few(ws_bytes=need - 1) == B.ERR_WORKSPACE
    none = {n: None for n in ("x", "logits", "gate_up", "down", "res", "idx", "w", "out", "ws")}
    assert _few(cfg=dict(tokens=0), **none) == B.OK


# ------------------------------------------------------------------------- norms

NORM = dict(rows=16, hidden=64, type=0, gate_rows=4, residual_scale=1.0, eps=1e-6)


def _norm_calls(cfg=None, ws_bytes=1 << 30, **null):
    L, c = B.lib(), ctypes.byref(B.make_norm(**{**NORM, **(cfg or {})}))
    a = {n: P for n in ("x", "y", "post", "gate", "pre", "out", "u", "go", "gu", "gx", "gy", "gpost", "ggate", "gpre", "ws")}
    a.update(null)
    return {
        "forward": lambda: L.moe_w4a16_norm(c, a["x"], a["y"], a["post"], a["gate"], a["pre"], a["out"], a["u"], None),
        "backward": lambda: L.moe_w4a16_norm_backward(c, a["y"], a["post"], a["gate"], a["out"], a["pre"], a["go"],
                                                      a["gu"], a["gx"], a["gy"], a["gpost"], a["ggate"], a["gpre"],
                                                      a["ws"], ws_bytes, None),
    }


@pytest.mark.parametrize("bad,status", [
    (dict(rows=-1), B.ERR_SHAPE), (dict(rows=(1 << 22) + 1), B.ERR_SHAPE), (dict(hidden=0), B.ERR_SHAPE),
    (dict(hidden=12), B.ERR_SHAPE), (dict(hidden=8200), B.ERR_SHAPE), (dict(type=3), B.ERR_SHAPE),
    (dict(type=-1), B.ERR_SHAPE), (dict(gate_rows=-1), B.ERR_SHAPE), (dict(gate_rows=(1 << 22) + 1), B.ERR_SHAPE),
    (dict(gate_rows=0), B.ERR_SHAPE),  # a gate is given
    (dict(residual_scale=math.inf), B.ERR_VALUE), (dict(residual_scale=math.nan), B.ERR_VALUE),
    (dict(eps=-1e-9), B.ERR_VALUE), (dict(eps=math.inf), B.ERR_VALUE), (dict(eps=math.nan), B.ERR_VALUE),
])
def test_norm_configurations_refused(bad, status):
    assert {call() for call in _norm_calls(bad).values()} == {status}
    if bad != dict(gate_rows=0):
        assert B.moe_w4a16_norm_backward_workspace_bytes(B.make_norm(**{**NORM, **bad})) == 0


def test_norm_pointers_refused():
    fwd = lambda **kw: _norm_calls(**kw)["forward"]()
    bwd = lambda **kw: _norm_calls(**kw)["backward"]()
    assert fwd(x=None, y=None, post=None, gate=None) == B.ERR_NULL        # nothing to norm
    assert fwd(out=None, u=None, pre=None) == B.ERR_NULL                  # nothing wanted
    assert fwd(y=None, gate=None) == fwd(y=None, post=None) == B.ERR_NULL  # y's weights without y
    assert fwd(pre=None) == fwd(u=None) == B.ERR_NULL                     # u and its weight go together
    for n in ("x", "y", "post", "gate", "pre", "out", "u"):
        assert fwd(**{n: P + 8}) == B.ERR_ALIGN, n
    assert bwd(go=None, gu=None, gpre=None) == B.ERR_NULL                 # no gradient arrives
    assert bwd(gx=None, gy=None, gpost=None, ggate=None, gpre=None) == B.ERR_NULL
    assert bwd(out=None) == bwd(pre=None) == B.ERR_NULL                   # grad_u needs both
    assert bwd(gu=None) == B.ERR_NULL                                     # grad_gamma_pre needs grad_u
    assert bwd(post=None) == bwd(gate=None) == B.ERR_NULL                 # a gradient of what is not there
    assert bwd(y=None) == bwd(ws=None) == B.ERR_NULL
    assert bwd(y=None, gpost=None, ggate=None) == B.ERR_NULL              # grad_y through the norm
    for n in ("y", "post", "gate", "pre", "out", "go", "gu", "gx", "gy", "gpost", "ggate", "gpre", "ws"):
        assert bwd(**{n: P + 8}) == B.ERR_ALIGN, n
    need = B.moe_w4a16_norm_backward_workspace_bytes(B.make_norm(**NORM))
    assert need > 0 and bwd(ws_bytes=need - 1) == B.ERR_WORKSPACE


def test_norm_without_rows_is_a_no_op():
    none = {n: None for n in ("x", "y", "post", "gate", "pre", "out", "u")}
    assert _norm_calls(dict(rows=0), **none)["forward"]() == B.OK


# ---------------------------------------------------------------------- clipping

def _clip(tensors, count=None, max_norm=1.0, norm=P, ws=P, ws_bytes=1 << 30):
    arr = (B.Tensor * max(len(tensors), 1))(*tensors)
    n = len(tensors) if count is None else count
    return B.lib().moe_w4a16_clip(ctypes.addressof(arr), n, max_norm, norm, ws, ws_bytes, None)


def test_clip_arguments_refused():
    t = B.Tensor(P, P, 8, 0)
    assert _clip([t], count=-1) == _clip([t], count=65537) == B.ERR_SHAPE
    assert B.moe_w4a16_clip_workspace_bytes(-1) == B.moe_w4a16_clip_workspace_bytes(65537) == 0
    assert B.lib().moe_w4a16_clip(None, 1, 1.0, P, P, 1 << 30, None) == B.ERR_NULL
    assert _clip([t], norm=None) == _clip([t], ws=None) == B.ERR_NULL
    assert _clip([t], max_norm=-1.0) == _clip([t], max_norm=math.nan) == B.ERR_VALUE
    assert _clip([t], norm=P + 2) == _clip([t], ws=P + 8) == B.ERR_ALIGN
    for bad in (B.Tensor(P, P, 8, 3), B.Tensor(P, P, 8, -1), B.Tensor(P, P, -1, 0), B.Tensor(P, P, (1 << 34) + 1, 0)):
        assert _clip([t, bad]) == B.ERR_SHAPE
    assert _clip([t, B.Tensor(None, P, 8, 0)]) == B.ERR_NULL
    for bad in (B.Tensor(P + 1, P, 8, 0), B.Tensor(P, P + 1, 8, 1), B.Tensor(P + 2, P, 8, 2), B.Tensor(P, P + 2, 8, 2)):
        assert _clip([t, bad]) == B.ERR_ALIGN
    for n in (0, 1, 640, 641, 65536):
        need = B.moe_w4a16_clip_workspace_bytes(n)
        assert need == 608 * 8 * max(1, -(-n // 640))
        assert _clip([t] * n, ws_bytes=need - 1) == B.ERR_WORKSPACE


def test_tensor_lists_refused(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(B, "_CONTEXT", None)
    norm, ws = torch.zeros(1), torch.zeros(8192, dtype=torch.uint8)

    def refused(make):
        with pytest.raises(B.MoeW4A16Error) as e:
            make()
        return e.value.status

    a = torch.zeros(4, 6)
    assert refused(lambda: B.make_tensors([a, a.long()])) == B.ERR_SHAPE
    assert refused(lambda: B.make_tensors([a.t()])) == B.ERR_SHAPE            # strided
    assert refused(lambda: B.make_tensors([a], [a.half()])) == B.ERR_SHAPE    # another type
    assert refused(lambda: B.make_tensors([a], [a[:3]])) == B.ERR_SHAPE       # another size
    assert refused(lambda: B.make_tensors([a, a], [a])) == B.ERR_SHAPE
    assert refused(lambda: B.moe_w4a16_clip([a], 1.0, norm, ws, 0)) == B.ERR_DEVICE  # on the host
    lst = B.make_tensors([a, torch.zeros(0, dtype=torch.float16), a.bfloat16()], [None, None, a.bfloat16()])
    assert [s.count for s in lst.array] == [24, 0, 24] and [s.type for s in lst.array] == [2, 0, 1]
    assert [bool(s.out) for s in lst.array] == [False, False, True]
    monkeypatch.setattr(B, "_CONTEXT", None)


def test_structs_match_the_header(tmp_path):
    structs = {"moe_w4a16_norm_cfg": B.Norm, "moe_w4a16_tensor": B.Tensor}
    lines = ['#include <stddef.h>', '#include <stdio.h>', '#include "moe_w4a16.h"', "int main(void) {",
             '  printf("few tokens %d\\n", MOE_W4A16_FEW_TOKENS);']
    for cname, cls in structs.items():
        lines.append(f'  printf("{cname} size %zu\\n", sizeof({cname}));')
        lines += [f'  printf("{cname} {f} %zu\\n", offsetof({cname}, {f}));' for f, _ in cls._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["  return 0;\n}"]))
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.run(["gcc", "-std=c11", "-I", include, str(src), "-o", str(exe)], check=True)
    got = {}
    for ln in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines():
        name, field, val = ln.split()
        got[(name, field)] = int(val)
    assert got[("few", "tokens")] == B.FEW_TOKENS
    for cname, cls in structs.items():
        assert got[(cname, "size")] == ctypes.sizeof(cls)
        assert all(got[(cname, f)] == getattr(cls, f).offset for f, _ in cls._fields_)


def test_a_blocks_buffers_are_ready_for_any_stream(monkeypatch):
    """Its own buffers are allocated before those of its layer, whose constructor ends when the stream has."""
    from w4a16_moe_expert_router_gb300 import runtime
    seen, empty = [], torch.empty

    class Stream:
        def synchronize(self):
            seen.append("synchronize")

    monkeypatch.setattr(B, "moe_w4a16_workspace_init", lambda ws, stream=None: None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream())
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch, "empty", lambda *a, **k: seen.append("empty") or empty(*a, **k))
    runtime.Block16(4, 64, 64, 4, 2, gate_rows=3, device="cpu")
    assert seen.count("synchronize") == 1 and seen[-1] == "synchronize"


def test_layer16_without_its_residual(monkeypatch):
    """The layer adds x and its gradient only where it was asked to."""
    from w4a16_moe_expert_router_gb300 import runtime
    seen = []
    for name in [n for n in vars(B) if n.startswith("moe_w4a16_") and not n.endswith("_bytes")]:
        monkeypatch.setattr(B, name, lambda *a, name=name: seen.append((name, a)))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    layer = runtime.Layer16(4, 64, 64, 4, 2, device="cpu")
    x, dout = object(), object()
    for residual in (True, False):
        seen.clear()
        layer.forward(x, None, None, None, None, None, residual)
        layer.backward(dout)
        rows = [a for n, a in seen if n == "moe_w4a16_combine_rows"]
        assert [a[4] for a in rows] == ([x, dout] if residual else [None, None])
