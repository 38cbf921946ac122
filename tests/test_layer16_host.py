"""Host-only tests of the 16-bit layer's operators: configurations, pointers and
workspaces are checked before a GPU is touched, and the binding refuses tensors
of another type, size, layout or device than the call reads."""
import ctypes
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


ROWS = dict(tokens=16, experts=8, top_k=2, hidden=64, type=0)


def _rows(**kw):
    return B.make_rows(**{**ROWS, **kw})


def _row_calls(cfg, ws_bytes=1 << 30, **null):
    """Each row call on stand-in addresses; null[name] replaces one.  Only calls that are
    refused are made: the addresses are no memory."""
    L, c = B.lib(), ctypes.byref(cfg)
    a = {n: P for n in ("idx", "x", "off", "list", "pos", "rows", "ws", "w", "res", "out", "gx", "gr", "gw", "gl", "go")}
    a.update(null)
    return {
        "dispatch": lambda: L.moe_w4a16_dispatch(c, a["idx"], a["x"], a["off"], a["list"], a["pos"], a["rows"], a["ws"],
                                                 ws_bytes, None),
        "dispatch_backward": lambda: L.moe_w4a16_dispatch_backward(c, a["pos"], a["rows"], a["gx"], None),
        "combine": lambda: L.moe_w4a16_combine_rows(c, a["pos"], a["w"], a["rows"], a["res"], a["out"], None),
        "combine_backward": lambda: L.moe_w4a16_combine_rows_backward(c, a["idx"], a["pos"], a["w"], a["rows"], a["go"],
                                                              a["gr"], a["gw"], a["gl"], None),
    }


@pytest.mark.parametrize("bad", [
    dict(tokens=-1), dict(experts=0), dict(experts=257), dict(top_k=0), dict(top_k=9, experts=16),
    dict(experts=4, top_k=5), dict(hidden=0), dict(hidden=4), dict(hidden=68), dict(hidden=65544), dict(type=3),
    dict(type=-1), dict(tokens=(1 << 21) + 1),
])
def test_row_configurations_refused(bad):
    cfg = _rows(**bad)
    assert B.moe_w4a16_dispatch_workspace_bytes(cfg) == 0
    assert {call() for call in _row_calls(cfg).values()} == {B.ERR_SHAPE}


@pytest.mark.parametrize("name,calls", [
    ("idx", {"dispatch"}), ("x", {"dispatch"}), ("off", {"dispatch"}), ("list", {"dispatch"}), ("ws", {"dispatch"}),
    ("pos", {"dispatch", "dispatch_backward", "combine", "combine_backward"}),
    ("rows", {"dispatch", "dispatch_backward", "combine", "combine_backward"}),
    ("gx", {"dispatch_backward"}), ("w", {"combine_backward"}), ("out", {"combine"}),
    ("go", {"combine_backward"}),
])
def test_row_pointers_refused(name, calls):
    for call in calls:
        assert _row_calls(_rows(), **{name: None})[call]() == B.ERR_NULL, call
        assert _row_calls(_rows(), **{name: P + 8})[call]() == B.ERR_ALIGN, call


def test_row_optional_pointers():
    for name in ("res", "w"):
        assert _row_calls(_rows(), **{name: P + 8})["combine"]() == B.ERR_ALIGN
    for name in ("gr", "gw", "gl"):
        assert _row_calls(_rows(), **{name: P + 8})["combine_backward"]() == B.ERR_ALIGN
    assert _row_calls(_rows(), gr=None, gw=None, gl=None)["combine_backward"]() == B.ERR_NULL
    assert _row_calls(_rows(), idx=None)["combine_backward"]() == B.ERR_NULL  # grad_logits needs the ids


def test_dispatch_workspace():
    assert B.moe_w4a16_dispatch_workspace_bytes(_rows(tokens=2048)) == 16           # 4096 pairs: one chunk
    big = _rows(tokens=2049)                                                        # 4098 pairs in chunks of 512
    assert B.moe_w4a16_dispatch_workspace_bytes(big) == (9 + 1) * 8 * 4
    assert B.moe_w4a16_dispatch_workspace_bytes(_rows(tokens=1000, top_k=7)) == (14 + 1) * 8 * 4  # chunks of 504
    assert _row_calls(big, ws_bytes=(9 + 1) * 8 * 4 - 1)["dispatch"]() == B.ERR_WORKSPACE


def test_no_tokens_is_a_no_op():
    none = {n: None for n in ("idx", "x", "list", "pos", "rows", "ws", "w", "out", "gx", "go", "gr", "gw", "gl")}
    got = _row_calls(_rows(tokens=0), **none)
    assert got["dispatch_backward"]() == got["combine"]() == got["combine_backward"]() == B.OK
    assert _row_calls(_rows(tokens=0), off=None)["dispatch"]() == B.ERR_NULL  # the offsets are written all the same
    assert _row_calls(_rows(tokens=0), off=P + 4)["dispatch"]() == B.ERR_ALIGN


LINEAR = dict(rows=16, inp=64, out=32, groups=4, activation=0, gated=0, type=0)


def _linear(**kw):
    return B.make_linear(**{**LINEAR, **kw})


def _linear_calls(cfg, ws_bytes=1 << 30, **null):
    """Both product calls on stand-in addresses; only calls that are refused are made."""
    L, c = B.lib(), ctypes.byref(cfg)
    a = {n: P for n in ("x", "off", "weight", "bias", "res", "out", "z", "ws", "go", "gx", "gw", "gb")}
    a.update(null)
    return {
        "forward": lambda: L.moe_w4a16_linear(c, a["x"], a["off"], a["weight"], a["bias"], a["res"], a["out"], a["z"],
                                              a["ws"], ws_bytes, None),
        "backward": lambda: L.moe_w4a16_linear_backward(c, a["x"], a["off"], a["weight"], a["z"], a["go"], a["gx"],
                                                        a["gw"], a["gb"], a["ws"], ws_bytes, None),
    }


@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(rows=(1 << 22) + 1), dict(inp=0), dict(inp=12), dict(inp=65544), dict(out=0), dict(out=20),
    dict(out=65544), dict(groups=0), dict(groups=257), dict(activation=-1), dict(activation=4), dict(gated=2),
    dict(gated=-1), dict(type=2), dict(type=-1),
])
def test_linear_configurations_refused(bad):
    cfg = _linear(**bad)
    assert B.moe_w4a16_linear_workspace_bytes(cfg) == B.moe_w4a16_linear_backward_workspace_bytes(cfg) == 0
    assert {call() for call in _linear_calls(cfg).values()} == {B.ERR_SHAPE}


@pytest.mark.parametrize("name,calls", [
    ("x", {"forward", "backward"}), ("weight", {"forward", "backward"}), ("off", {"forward", "backward"}),
    ("out", {"forward"}), ("ws", {"forward", "backward"}), ("z", {"backward"}), ("go", {"backward"}),
])
def test_linear_pointers_refused(name, calls):
    for call in calls:
        assert _linear_calls(_linear(), **{name: None})[call]() == B.ERR_NULL, call
        assert _linear_calls(_linear(), **{name: P + 8})[call]() == B.ERR_ALIGN, call


def test_linear_optional_pointers_and_workspace():
    for name in ("bias", "res", "z"):
        assert _linear_calls(_linear(), **{name: P + 8})["forward"]() == B.ERR_ALIGN
    for name in ("gx", "gw", "gb"):
        assert _linear_calls(_linear(), **{name: P + 8})["backward"]() == B.ERR_ALIGN
    assert _linear_calls(_linear(), gx=None, gw=None, gb=None)["backward"]() == B.ERR_NULL
    assert _linear_calls(_linear(activation=3, gated=1), z=None)["backward"]() == B.ERR_NULL
    assert _linear_calls(_linear(), ws_bytes=255)["forward"]() == B.ERR_WORKSPACE
    # header, dz [16][64] in 16 bits, partial sums of 1 + 4 row blocks of 64 columns
    need = B.moe_w4a16_linear_backward_workspace_bytes(_linear(gated=1))
    assert need == 256 + 16 * 64 * 2 + 5 * 64 * 4
    assert _linear_calls(_linear(gated=1), ws_bytes=need - 1)["backward"]() == B.ERR_WORKSPACE


def test_linear_without_rows_is_a_no_op():
    none = {n: None for n in ("x", "off", "weight", "bias", "res", "out", "z", "ws")}
    assert _linear_calls(_linear(rows=0), **none)["forward"]() == B.OK


def test_binding_refuses_tensors_it_cannot_pass_on(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(B, "_CONTEXT", None)
    cfg = _rows()
    good = dict(pos=torch.zeros(16, 2, dtype=torch.int32), w=torch.zeros(16, 2),
                rows=torch.zeros(32, 64, dtype=torch.float16), out=torch.zeros(16, 64, dtype=torch.float16))

    def call(**kw):
        a = {**good, **kw}
        with pytest.raises(B.MoeW4A16Error) as e:
            B.moe_w4a16_combine_rows(cfg, a["pos"], a["w"], a["rows"], None, a["out"], stream=0)
        return e.value.status

    assert call() == B.ERR_DEVICE                                                # all on the host
    assert call(pos=torch.zeros(16, 2, dtype=torch.int64)) == B.ERR_SHAPE
    assert call(pos=torch.zeros(15, 2, dtype=torch.int32)) == B.ERR_SHAPE
    assert call(pos=torch.zeros(2, 16, dtype=torch.int32).t()) == B.ERR_SHAPE    # strided
    assert call(pos=P, w=torch.zeros(16, 2, dtype=torch.float16)) == B.ERR_SHAPE
    assert call(pos=P, w=P, rows=torch.zeros(32, 64)) == B.ERR_SHAPE
    monkeypatch.setattr(B, "_CONTEXT", None)


def test_structs_match_the_header(tmp_path):
    structs = {"moe_w4a16_rows": B.Rows, "moe_w4a16_linear_cfg": B.Linear}
    lines = ['#include <stddef.h>', '#include <stdio.h>', '#include "moe_w4a16.h"', "int main(void) {"]
    name = lambda f: {"inp": "in"}.get(f, f)  # a keyword in Python
    for cname, cls in structs.items():
        lines.append(f'  printf("{cname} size %zu\\n", sizeof({cname}));')
        lines += [f'  printf("{cname} {f} %zu\\n", offsetof({cname}, {name(f)}));' for f, _ in cls._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["  return 0;\n}"]))
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.run(["gcc", "-std=c11", "-I", include, str(src), "-o", str(exe)], check=True)
    got = {}
    for ln in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines():
        name, field, val = ln.split()
        got[(name, field)] = int(val)
    for cname, cls in structs.items():
        assert got[(cname, "size")] == ctypes.sizeof(cls)
        assert all(got[(cname, f)] == getattr(cls, f).offset for f, _ in cls._fields_)


@pytest.mark.parametrize("capturing", [False, True])
def test_a_layers_buffers_are_ready_for_any_stream(monkeypatch, capturing):
    """The constructor ends when its stream has: what it took over and cleared is done before a call on another
    stream.  A stream that is being captured cannot be waited for."""
    from w4a16_moe_expert_router_gb300 import runtime
    seen = []

    class Stream:
        def synchronize(self):
            seen.append("synchronize")

    monkeypatch.setattr(B, "moe_w4a16_workspace_init", lambda ws, stream=None: seen.append("init"))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream())
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing)
    runtime.Layer16(4, 64, 64, 4, 2, device="cpu")
    assert seen == ["init", "init"] + ([] if capturing else ["synchronize"])
