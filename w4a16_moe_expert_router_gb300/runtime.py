"""Device-side plumbing around the C ABI: buffers allocated with PyTorch,
weights uploaded in the prepared layout, and the route + forward call pair.

Nothing here computes any part of the layer; it only allocates, copies and
calls the binding.
"""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np
import torch

from . import binding as B
from .synth import Workload


def shape_of(wl: Workload, tokens: int | None = None) -> B.Shape:
    return B.make_shape(wl.tokens if tokens is None else tokens, wl.hidden, wl.inter, wl.experts, wl.top_k,
                        wl.group_gate_up, wl.group_down, wl.activation, wl.reduction, wl.format)


@dataclass
class PreparedWeights:
    gate_up: torch.Tensor  # uint8, prepared stream
    down: torch.Tensor

    @property
    def nbytes(self) -> int:
        return self.gate_up.numel() + self.down.numel()


def prepare_host(wl: Workload, w: dict) -> tuple[np.ndarray, np.ndarray]:
    """Canonical numpy weights -> the two prepared streams (host)."""
    sh = shape_of(wl, 1)
    gu = B.moe_w4a16_prepare(sh, B.GATE_UP, w["gate_up_q"], w["gate_up_scale"], w["gate_up_zero"])
    dn = B.moe_w4a16_prepare(sh, B.DOWN, w["down_q"], w["down_scale"], w["down_zero"])
    return gu, dn


def upload_weights(wl: Workload, w: dict, device="cuda") -> PreparedWeights:
    gu, dn = prepare_host(wl, w)
    return PreparedWeights(torch.from_numpy(gu).to(device), torch.from_numpy(dn).to(device))


@dataclass
class Buffers:
    """Per-canvas device buffers: routing, workspace and output."""
    shape: B.Shape
    routing: B.RoutingBuffers
    workspace: torch.Tensor
    out: torch.Tensor


def alloc_buffers(wl: Workload, tokens: int | None = None, device="cuda", stream=None) -> Buffers:
    sh = shape_of(wl, tokens)
    T, k, E = sh.tokens, sh.top_k, sh.experts
    routing = B.RoutingBuffers(
        topk_idx=torch.empty((T, k), dtype=torch.int32, device=device),
        topk_w=torch.empty((T, k), dtype=torch.float32, device=device),
        expert_offsets=torch.empty((E + 1,), dtype=torch.int32, device=device),
        pair_list=torch.empty((max(T * k, 1),), dtype=torch.int32, device=device),
    )
    ws = torch.empty((B.moe_w4a16_workspace_bytes(sh),), dtype=torch.uint8, device=device)
    B.moe_w4a16_workspace_init(ws, stream)
    out = torch.empty((T, wl.hidden), dtype=torch.float16, device=device)
    return Buffers(sh, routing, ws, out)


def run_layer(buf: Buffers, x: torch.Tensor, logits: torch.Tensor, w: PreparedWeights,
              gamma: torch.Tensor | None = None, eps: float = 1e-6, out: torch.Tensor | None = None,
              stream=None) -> torch.Tensor:
    """Route the canvas, then run the experts and the combine; returns the output tensor."""
    o = buf.out if out is None else out
    B.moe_w4a16_route(buf.shape, logits, buf.routing, buf.workspace, stream)
    B.moe_w4a16_forward(buf.shape, x, buf.routing, w.gate_up, w.down, gamma, eps, o, buf.workspace, stream)
    return o


def run_block(buf: Buffers, x: torch.Tensor, gamma_pre: torch.Tensor, router_w: torch.Tensor, w: PreparedWeights,
              eps: float = 1e-6, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The MoE block: pre-norm, router projection, routing, experts, combine plus the residual."""
    o = buf.out if out is None else out
    B.moe_w4a16_block(buf.shape, x, gamma_pre, eps, router_w, buf.routing, w.gate_up, w.down, o, buf.workspace,
                      stream)
    return o


def to_device_u16(a: np.ndarray, device="cuda") -> torch.Tensor:
    """fp16 bit patterns (uint16) as an fp16 device tensor."""
    return torch.from_numpy(np.ascontiguousarray(a).view(np.float16)).to(device)


def to_device_x(x_bits: np.ndarray, device="cuda") -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(x_bits).view(np.float16)).to(device)


def to_device_f32(a: np.ndarray, device="cuda") -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(device)


class Layer16:
    """The expert layer in 16 bits with gradients: the buffers of one batch and the call
    sequence route -> dispatch -> gate and up -> down -> combine (with the residual), and
    back.  ``backward`` belongs to the last ``forward``; both leave their results in the
    layer's buffers.  The calls take any stream, one after the other: their order over several
    streams is the caller's.  Nothing is recorded by autograd.

    Rows are fp16 (type 0) or bf16 (type 1); gate_up [E][2f][d] with an fp32 bias
    [E][2f] or None, down [E][d][f], router logits fp32 [T][E].
    """

    def __init__(self, tokens: int, hidden: int, inter: int, experts: int, top_k: int, activation: int = 0,
                 type: int = 0, device="cuda"):
        T, d, f, E, k = tokens, hidden, inter, experts, top_k
        dt = (torch.float16, torch.bfloat16)[type]
        # the routing call takes a layer shape; only its tokens, experts and top_k matter to it
        self.shape = B.make_shape(T, 128, 64, E, k, 32, 32)
        self.rows = B.make_rows(T, E, k, d, type)
        self.up = B.make_linear(T * k, d, f, E, activation, 1, type)
        self.dn = B.make_linear(T * k, f, d, E, 3, 0, type)

        def new(*shape, dtype=dt):
            return torch.empty(shape, dtype=dtype, device=device)

        i32, f32 = torch.int32, torch.float32
        self.routing = B.RoutingBuffers(new(T, k, dtype=i32), new(T, k, dtype=f32), new(E + 1, dtype=i32),
                                        new(T * k, dtype=i32))
        self.pair_pos = new(T, k, dtype=i32)
        self.x_rows, self.z, self.h, self.y = new(T * k, d), new(T * k, 2 * f), new(T * k, f), new(T * k, d)
        self.out = new(T, d)
        self.grad_y, self.grad_h, self.grad_rows, self.grad_x = new(T * k, d), new(T * k, f), new(T * k, d), new(T, d)
        self.grad_w, self.grad_logits = new(T, k, dtype=f32), new(T, E, dtype=f32)
        self.grad_gate_up, self.grad_down = new(E, 2 * f, d), new(E, d, f)
        self.grad_bias = new(E, 2 * f, dtype=f32)
        self.ws = [new(max(n, 256), dtype=torch.uint8) for n in (
            B.moe_w4a16_workspace_bytes(self.shape), B.moe_w4a16_dispatch_workspace_bytes(self.rows),
            max(B.moe_w4a16_linear_workspace_bytes(self.up), B.moe_w4a16_linear_backward_workspace_bytes(self.up),
                B.moe_w4a16_linear_backward_workspace_bytes(self.dn)))]
        B.moe_w4a16_workspace_init(self.ws[0])
        B.moe_w4a16_workspace_init(self.ws[2])
        # memory that the buffers took over may still be in use on this stream, and the workspaces' start is
        # cleared on it: done before another stream gets a call (a captured constructor keeps to its graph)
        if not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream().synchronize()

    def forward(self, x, logits, gate_up, gate_up_bias, down, stream=None) -> torch.Tensor:
        """out = x + sum_r w_r expert_r(x) for every token."""
        r = self.routing
        self.saved = (gate_up, gate_up_bias, down)
        B.moe_w4a16_route(self.shape, logits, r, self.ws[0], stream)
        B.moe_w4a16_dispatch(self.rows, r.topk_idx, x, r.expert_offsets, r.pair_list, self.pair_pos, self.x_rows,
                             self.ws[1], stream)
        B.moe_w4a16_linear(self.up, self.x_rows, r.expert_offsets, gate_up, gate_up_bias, None, self.h, self.z,
                           self.ws[2], stream)
        B.moe_w4a16_linear(self.dn, self.h, r.expert_offsets, down, None, None, self.y, None, self.ws[2], stream)
        B.moe_w4a16_combine_rows(self.rows, self.pair_pos, r.topk_w, self.y, x, self.out, stream)
        return self.out

    def backward(self, grad_out, stream=None) -> dict:
        """Gradients of the last forward: x (the residual's included), logits, gate_up,
        gate_up_bias (where there is a bias) and down."""
        r, (gate_up, bias, down) = self.routing, self.saved
        B.moe_w4a16_combine_rows_backward(self.rows, r.topk_idx, self.pair_pos, r.topk_w, self.y, grad_out, self.grad_y,
                                          self.grad_w, self.grad_logits, stream)
        B.moe_w4a16_linear_backward(self.dn, self.h, r.expert_offsets, down, None, self.grad_y, self.grad_h,
                                    self.grad_down, None, self.ws[2], stream)
        B.moe_w4a16_linear_backward(self.up, self.x_rows, r.expert_offsets, gate_up, self.z, self.grad_h,
                                    self.grad_rows, self.grad_gate_up, None if bias is None else self.grad_bias,
                                    self.ws[2], stream)
        # dispatch's gradient with the residual's added: the rows back with weights of one
        B.moe_w4a16_combine_rows(self.rows, self.pair_pos, None, self.grad_rows, grad_out, self.grad_x, stream)
        out = {"x": self.grad_x, "logits": self.grad_logits, "gate_up": self.grad_gate_up, "down": self.grad_down}
        if bias is not None:
            out["gate_up_bias"] = self.grad_bias
        return out
