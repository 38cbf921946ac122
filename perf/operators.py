"""Cases for measuring the operators of the 16-bit expert layer with gradients.

A case is one call of one operator:

  dispatch       tokens sorted by expert: expert offsets, pair list, each pair's row, and the rows copied in that order
  dispatch_grad  its gradient: every token's gradient is the sum over its pairs' rows
  combine        rows back to their tokens, weighted by the router, with the residual added
  combine_grad   its gradient: rows, router weights and router logits
  linear         act(x W^T + b) (gated: act(x Wg^T + bg) * (x Wu^T + bu)) + residual, one weight for all rows or one
                 per expert on rows sorted by expert
  linear_grad    its gradient: input, weight and bias

With ``own`` false an operator is computed in its plain form: elementary torch operations in 32 bits, rounded once at
the end.  With ``own`` true ``run`` makes the calls of the library's binding.
"""
import math

import torch

own = False

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
TYPE_CODES = {"fp16": 0, "bf16": 1, "fp32": 2}
BYTES = {"fp16": 2, "bf16": 2, "fp32": 4}
ACT_CODES = {"gelu": 0, "gelu_erf": 1, "silu": 2, "none": 3}


def _rows(name, op, dtype, tokens, experts, top_k, hidden, skew=0.0, drop=0.0, residual=False):
    return {"name": name, "op": op, "dtype": dtype, "tokens": tokens, "experts": experts, "top_k": top_k,
            "hidden": hidden, "skew": skew, "drop": drop, "residual": residual}


def _linear(name, op, dtype, rows, inp, out, experts=0, act="none", gated=False, bias=True, residual=False,
            save=False, skew=0.0):
    return {"name": name, "op": op, "dtype": dtype, "rows": rows, "in": inp, "out": out, "experts": experts,
            "act": act, "gated": gated, "bias": bias, "residual": residual, "save": save, "skew": skew}


def listed():
    return [
        # one token of a generation loop: 8 of 128 experts; latency only
        _rows("dispatch one token", "dispatch", "fp16", 1, 128, 8, 2048),
        # a training batch of the 128-expert layer, unevenly loaded
        _rows("dispatch 16384 tokens", "dispatch", "bf16", 16384, 128, 8, 2048, skew=1.1),
        # the gradient of a batch in 32 bits whose last tokens are padding and whose full experts dropped pairs
        _rows("dispatch gradient padded", "dispatch_grad", "fp32", 4099, 128, 8, 2048, skew=1.1, drop=0.1),
        # one 256-token canvas back to its tokens, on to the residual stream
        _rows("combine canvas", "combine", "fp16", 256, 128, 8, 2048, residual=True),
        # the gradient of a training batch of odd length, down to the router's logits
        _rows("combine gradient", "combine_grad", "bf16", 8191, 128, 8, 2048, skew=1.1, drop=0.05),
        # a dense projection of one token: its time is the weight's way from memory
        _linear("linear one token", "linear", "fp16", 1, 2048, 4096, residual=True),
        # a ragged batch through a projection whose sizes fit no tile
        _linear("linear ragged", "linear", "fp16", 777, 1000, 2056, act="silu", residual=True),
        # the wide projection of a dense feed-forward block in training: keeps what its gradient needs
        _linear("linear 8192 rows", "linear", "bf16", 8192, 2048, 8192, act="gelu", save=True),
        # the gate and up projections of all 128 experts on one 256-token canvas (16 rows an expert)
        _linear("experts canvas gated", "linear", "fp16", 2048, 2048, 704, experts=128, act="gelu", gated=True,
                bias=False),
        # the down projections of a training batch, 32768 rows unevenly over 128 experts
        _linear("experts down skewed", "linear", "bf16", 32768, 704, 2048, experts=128, bias=False, skew=0.1),
        # the gradient of a dense projection
        _linear("linear gradient", "linear_grad", "fp16", 4096, 2048, 2048, act="gelu_erf"),
        # the gradient of the experts' gate and up projections in a training batch
        _linear("experts gradient gated", "linear_grad", "bf16", 16384, 2048, 704, experts=128, act="gelu", gated=True,
                skew=0.1),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["dispatch", "dispatch_grad", "combine", "combine_grad", "linear", "linear", "linear_grad"])
    if not op.startswith("linear"):
        dtype = rng.choice(["fp16", "bf16", "bf16", "fp32"])
        experts = _log_int(rng, 4, 256)
        top_k = rng.randint(1, min(8, experts))
        hidden = 8 * _log_int(rng, 8, 512)
        tokens = _log_int(rng, 1, 16384)
        tokens = max(1, min(tokens, (1 << 28) // (top_k * hidden * BYTES[dtype] // 2)))
        c = _rows("", op, dtype, tokens, experts, top_k, hidden, skew=rng.choice([0.0, 1.1]),
                  drop=rng.choice([0.0, 0.0, 0.1]), residual=op == "combine" and rng.random() < 0.5)
    else:
        dtype = rng.choice(["fp16", "bf16"])
        gated = rng.random() < 0.4
        inp, out = 8 * _log_int(rng, 8, 512), 8 * _log_int(rng, 8, 512)
        experts = rng.choice([0, 0, _log_int(rng, 2, 128)])
        rows = _log_int(rng, 1, 16384)
        rows = max(1, min(rows, int(4e10) // (inp * out * (2 if gated else 1))))
        if experts:
            experts = max(1, min(experts, (1 << 28) // (inp * out * (2 if gated else 1))))
        act = rng.choice(["gelu", "gelu_erf", "silu"] + ([] if gated else ["none"]))
        fwd = op == "linear"
        c = _linear("", op, dtype, rows, inp, out, experts=experts, act=act, gated=gated, bias=rng.random() < 0.7,
                    residual=fwd and rng.random() < 0.5, save=fwd and rng.random() < 0.3,
                    skew=rng.choice([0.0, 0.1]) if experts else 0.0)
    del c["name"]
    return c


# ------------------------------------------------------------------- inputs


def _router(g, tokens, experts, top_k, skew, drop):
    """The router's choice: expert ids [T][k] (-1: the pair is dropped) and the softmax over the k chosen logits.
    The last tokens are padding (all their pairs dropped), half as many pairs again were dropped singly."""
    logits = torch.randn(tokens, experts, generator=g, device="cuda")
    if skew:
        logits = logits - skew * torch.log(torch.arange(1, experts + 1, device="cuda", dtype=torch.float32))
    val, idx = torch.topk(logits, top_k, dim=1)
    idx, w = idx.to(torch.int32), torch.softmax(val, 1)
    if drop:
        gone = torch.rand(tokens, top_k, generator=g, device="cuda") < drop / 2
        gone[tokens - int(tokens * drop):] = True
        idx = torch.where(gone, torch.full_like(idx, -1), idx)
    return idx.contiguous(), w.contiguous()


def _places(idx, experts):
    """Offsets, pair list and row of each pair of a choice of experts."""
    top_k = idx.shape[1]
    ids = idx.reshape(-1).long()
    there = (ids >= 0) & (ids < experts)
    key = torch.where(there, ids, torch.full_like(ids, experts))
    sorted_key, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(sorted_key, torch.arange(experts + 1, device=ids.device))
    at = torch.arange(ids.numel(), device=ids.device)
    kept = at < offsets[experts]
    pair_list = torch.where(kept, order, torch.full_like(order, -1))
    pos = torch.empty_like(order)
    pos[order] = at
    pos = torch.where(there, pos, torch.full_like(pos, -1))
    return offsets.to(torch.int32), pair_list.to(torch.int32), pos.to(torch.int32).reshape(-1, top_k), order, kept


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = TYPES[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dtype).mul_(scale)

    s = {"case": case}
    if not case["op"].startswith("linear"):
        T, E, k, d = case["tokens"], case["experts"], case["top_k"], case["hidden"]
        s["idx"], s["w"] = _router(g, T, E, k, case["skew"], case["drop"])
        s["offsets"], s["pair_list"], s["pos"], _, kept = _places(s["idx"], E)
        if case["op"] == "dispatch":
            s["x"] = normal(T, d)
        else:
            s["rows"] = normal(T * k, d)
        if case["residual"]:
            s["residual"] = normal(T, d)
        if case["op"] == "combine_grad":
            s["dout"] = normal(T, d)
        if own:
            from w4a16_moe_expert_router_gb300 import binding as B
            s["B"] = B
            s["cfg"] = B.make_rows(T, E, k, d, TYPE_CODES[case["dtype"]])
            if case["op"] == "dispatch":
                s["out"] = {"offsets": torch.zeros(E + 1, dtype=torch.int32, device="cuda"),
                            "pair_list": torch.zeros(T * k, dtype=torch.int32, device="cuda"),
                            "pos": torch.zeros(T, k, dtype=torch.int32, device="cuda"),
                            "rows": torch.zeros(T * k, d, dtype=dt, device="cuda")}
                s["ws"] = torch.empty(B.moe_w4a16_dispatch_workspace_bytes(s["cfg"]), dtype=torch.uint8, device="cuda")
            elif case["op"] == "combine_grad":
                s["out"] = {"rows": torch.zeros(T * k, d, dtype=dt, device="cuda"), "w": torch.empty_like(s["w"]),
                            "logits": torch.empty(T, E, dtype=torch.float32, device="cuda")}
            else:
                s["out"] = torch.empty(T, d, dtype=dt, device="cuda")
        return s
    R, K, N, E = case["rows"], case["in"], case["out"], case["experts"]
    Nw = 2 * N if case["gated"] else N
    if E:
        logits = torch.randn(R, E, generator=g, device="cuda")
        if case["skew"]:
            logits = logits - case["skew"] * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
        ids = torch.sort(logits.argmax(1)).values
        s["offsets"] = torch.searchsorted(ids, torch.arange(E + 1, device="cuda")).to(torch.int32)
        s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())  # rows of the fullest expert
    s["x"] = normal(R, K)
    s["weight"] = normal(max(E, 1), Nw, K, scale=K ** -0.5)
    if case["bias"]:
        s["bias"] = normal(max(E, 1), Nw, scale=0.5, dtype=torch.float32)
    if case["residual"]:
        s["residual"] = normal(R, N)
    if case["op"] == "linear_grad":
        s["dout"] = normal(R, N)
        if case["gated"] or case["act"] != "none":
            s["preact"] = normal(R, Nw)
    if own:
        from w4a16_moe_expert_router_gb300 import binding as B
        s["B"] = B
        s["cfg"] = B.make_linear(R, K, N, max(E, 1), ACT_CODES[case["act"]], int(case["gated"]),
                                 TYPE_CODES[case["dtype"]])
        if case["op"] == "linear":
            s["out"] = {"out": torch.empty(R, N, dtype=dt, device="cuda")}
            if case["save"]:
                s["out"]["preact"] = torch.empty(R, Nw, dtype=dt, device="cuda")
            need = B.moe_w4a16_linear_workspace_bytes(s["cfg"])
        else:
            s["out"] = {"x": torch.empty_like(s["x"]), "weight": torch.empty_like(s["weight"])}
            if case["bias"]:
                s["out"]["bias"] = torch.empty_like(s["bias"])
            need = B.moe_w4a16_linear_backward_workspace_bytes(s["cfg"])
        s["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda")
        B.moe_w4a16_workspace_init(s["ws"])
    return s


# ---------------------------------------------------------- the two forms


def run(s):
    return _own(s) if own else _PLAIN[s["case"]["op"]](s)


def _own(s):
    B, cfg, op, out = s["B"], s["cfg"], s["case"]["op"], s["out"]
    if op == "dispatch":
        B.moe_w4a16_dispatch(cfg, s["idx"], s["x"], out["offsets"], out["pair_list"], out["pos"], out["rows"], s["ws"])
    elif op == "dispatch_grad":
        B.moe_w4a16_dispatch_backward(cfg, s["pos"], s["rows"], out)
    elif op == "combine":
        B.moe_w4a16_combine_rows(cfg, s["pos"], s["w"], s["rows"], s.get("residual"), out)
    elif op == "combine_grad":
        B.moe_w4a16_combine_rows_backward(cfg, s["idx"], s["pos"], s["w"], s["rows"], s["dout"], out["rows"], out["w"],
                                          out["logits"])
    elif op == "linear":
        B.moe_w4a16_linear(cfg, s["x"], s.get("offsets"), s["weight"], s.get("bias"), s.get("residual"), out["out"],
                           out.get("preact"), s["ws"])
    else:
        B.moe_w4a16_linear_backward(cfg, s["x"], s.get("offsets"), s["weight"], s.get("preact"), s["dout"], out["x"],
                                    out["weight"], out.get("bias"), s["ws"])
    return out


def _plain_dispatch(s):
    x, idx, E, k = s["x"], s["idx"], s["case"]["experts"], s["case"]["top_k"]
    offsets, pair_list, pos, order, kept = _places(idx, E)
    rows = torch.where(kept[:, None], x[order // k], torch.zeros((), dtype=x.dtype, device=x.device))
    return {"offsets": offsets, "pair_list": pair_list, "pos": pos, "rows": rows}


def _pair_rows(s):
    """The row of every pair in 32 bits [T][k][d], zeros for a dropped one."""
    pos, there = s["pos"].clamp(min=0).long(), (s["pos"] >= 0)[:, :, None]
    return torch.where(there, s["rows"][pos].float(), torch.zeros((), device=pos.device))


def _plain_dispatch_grad(s):
    return _pair_rows(s).sum(1).to(s["rows"].dtype)


def _plain_combine(s):
    out = (_pair_rows(s) * s["w"][:, :, None]).sum(1)
    if "residual" in s:
        out = out + s["residual"].float()
    return out.to(s["rows"].dtype)


def _plain_combine_grad(s):
    k, rows, w = s["case"]["top_k"], s["rows"], s["w"]
    pair = s["pair_list"].clamp(min=0).long()
    there = (s["pair_list"] >= 0)[:, None]
    dout = s["dout"].float()
    drows = torch.where(there, w.reshape(-1)[pair][:, None] * dout[pair // k], torch.zeros((), device=w.device))
    dw = (_pair_rows(s) * dout[:, None, :]).sum(2)
    dsel = w * (dw - (w * dw).sum(1, keepdim=True))
    dlogits = torch.zeros(w.shape[0], s["case"]["experts"], device=w.device)
    dsel = torch.where(s["idx"] >= 0, dsel, torch.zeros((), device=w.device))
    dlogits.scatter_add_(1, s["idx"].clamp(min=0).long(), dsel)
    return {"rows": drows.to(rows.dtype), "w": dw, "logits": dlogits}


def _act(a, kind):
    """The activation and its derivative in 32 bits."""
    if kind == "none":
        return a, torch.ones_like(a)
    if kind == "silu":
        p = torch.sigmoid(a)
        return a * p, p * (1 + a * (1 - p))
    if kind == "gelu_erf":
        c = 0.5 * (1 + torch.erf(a * math.sqrt(0.5)))
        return a * c, c + a * torch.exp(-0.5 * a * a) * (1 / math.sqrt(2 * math.pi))
    r = math.sqrt(2 / math.pi)
    p = torch.sigmoid(2 * r * (a + 0.044715 * a * a * a))
    return a * p, p + a * p * (1 - p) * (2 * r) * (1 + 3 * 0.044715 * a * a)


def _spread(s, v):
    """Rows [R][c] dealt to their experts: [E][most][c] with zeros behind an expert's rows (dense: [1][R][c])."""
    if "offsets" not in s:
        return v[None].float()
    at, there = _slots(s)
    return torch.where(there[:, :, None], v[at].float(), torch.zeros((), device=v.device))


def _slots(s):
    first, last = s["offsets"][:-1, None].long(), s["offsets"][1:, None].long()
    at = first + torch.arange(s["most"], device=first.device)
    there = at < last
    return torch.where(there, at, torch.zeros_like(at)), there


def _back(s, v):
    """The inverse of _spread."""
    if "offsets" not in s:
        return v[0]
    row = torch.arange(s["case"]["rows"], device=v.device)
    expert = torch.searchsorted(s["offsets"][1:].long(), row, right=True)
    return v[expert, row - s["offsets"].long()[expert]]


def _plain_linear(s):
    c, dt = s["case"], s["x"].dtype
    z = _back(s, torch.bmm(_spread(s, s["x"]), s["weight"].float().transpose(1, 2)) + (
        s["bias"][:, None, :] if "bias" in s else 0.0))
    a = z[:, :c["out"]]
    y = _act(a, c["act"])[0]
    if c["gated"]:
        y = y * z[:, c["out"]:]
    if "residual" in s:
        y = y + s["residual"].float()
    out = {"out": y.to(dt)}
    if c["save"]:
        out["preact"] = z.to(dt)
    return out


def _plain_linear_grad(s):
    c, dt = s["case"], s["x"].dtype
    dz = s["dout"].float()
    if "preact" in s:
        z = s["preact"].float()
        y, dy = _act(z[:, :c["out"]], c["act"])
        dz = torch.cat([dz * z[:, c["out"]:] * dy, dz * y], 1) if c["gated"] else dz * dy
    dz = _spread(s, dz)
    out = {"x": _back(s, torch.bmm(dz, s["weight"].float())).to(dt),
           "weight": torch.bmm(dz.transpose(1, 2), _spread(s, s["x"])).to(dt)}
    if "bias" in s:
        out["bias"] = dz.sum(1)
    return out


_PLAIN = {"dispatch": _plain_dispatch, "dispatch_grad": _plain_dispatch_grad, "combine": _plain_combine,
          "combine_grad": _plain_combine_grad, "linear": _plain_linear, "linear_grad": _plain_linear_grad}


# ------------------------------------------------------------------- work


def work(case):
    b = BYTES[case["dtype"]]
    if not case["op"].startswith("linear"):
        T, E, k, d = case["tokens"], case["experts"], case["top_k"], case["hidden"]
        padded = int(T * case["drop"])
        pairs = (T - padded) * k * (1 - case["drop"] / 2)  # kept
        tokens, moved = T * d * b, pairs * d * b
        if case["op"] == "dispatch":
            return {"bytes": tokens + moved + 12 * T * k + 4 * (E + 1), "flops": 0}
        if case["op"] == "combine_grad":
            return {"bytes": tokens + 2 * moved + 16 * T * k + 4 * T * E, "flops": 3 * pairs * d}
        return {"bytes": moved + tokens * (2 if case["residual"] else 1) + 8 * T * k, "flops": 2 * pairs * d}
    R, K, N, E = case["rows"], case["in"], case["out"], case["experts"]
    Nw = 2 * N if case["gated"] else N
    used = E * (1 - (1 - 1 / E) ** R) if E else 1  # experts with rows, evenly loaded
    weight = max(used, 1) * Nw * K * b
    bias = max(E, 1) * Nw * 4 if case["bias"] else 0
    if case["op"] == "linear":
        rows = R * (K + N * (2 if case["residual"] else 1) + (Nw if case["save"] else 0)) * b
        return {"bytes": rows + weight + bias, "flops": 2 * R * K * Nw}
    needs_z = case["gated"] or case["act"] != "none"
    rows = R * (2 * K + N + (Nw if needs_z else 0)) * b
    return {"bytes": rows + weight + max(E, 1) * Nw * K * b + bias, "flops": 4 * R * K * Nw}


# --------------------------------------------------- the definition in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "dispatch":
        return {"offsets": None, "pair_list": None, "pos": None, "rows": _exact_rows(s)}
    if op.startswith("linear"):
        return _exact_linear(s)
    T, k, d = case["tokens"], case["top_k"], case["hidden"]
    rows = s["rows"].double()
    if op == "combine_grad":
        dout, w = s["dout"].double(), s["w"].double()
        drows = torch.zeros_like(rows)
        dw = torch.zeros(T, k, dtype=torch.float64, device="cuda")
        dl = torch.zeros(T, case["experts"], dtype=torch.float64, device="cuda")
        for r in range(k):
            t = torch.nonzero(s["pos"][:, r] >= 0).flatten()
            p = s["pos"][t, r].long()
            drows[p] = w[t, r, None] * dout[t]
            dw[t, r] = torch.einsum("td,td->t", rows[p], dout[t])
        for r in range(k):  # d softmax: w_r (1 - w_r) for its own logit, -w_r w_j for another's
            t = torch.nonzero(s["pos"][:, r] >= 0).flatten()
            jac = -w[t, r, None] * w[t]
            jac[:, r] += w[t, r]
            dl[t, s["idx"][t, r].long()] += torch.einsum("tj,tj->t", jac, dw[t])
        return {"rows": drows, "w": dw, "logits": dl}
    out = s["residual"].double() if "residual" in s else torch.zeros(T, d, dtype=torch.float64, device="cuda")
    for r in range(k):
        t = torch.nonzero(s["pos"][:, r] >= 0).flatten()
        v = rows[s["pos"][t, r].long()]
        out[t] += v * s["w"][t, r, None].double() if op == "combine" else v
    return out


def _exact_rows(s):
    """Expert after expert, the tokens that chose it."""
    idx, at = s["idx"], 0
    rows = torch.zeros(idx.numel(), s["case"]["hidden"], dtype=torch.float64, device="cuda")
    for e in range(s["case"]["experts"]):
        t = torch.nonzero(idx == e)[:, 0]
        rows[at:at + t.numel()] = s["x"][t].double()
        at += t.numel()
    return rows


def _exact_act(a, kind):
    if kind == "none":
        return a
    if kind == "silu":
        return a / (1 + torch.exp(-a))
    if kind == "gelu_erf":
        return 0.5 * a * torch.special.erfc(-a / math.sqrt(2))
    return 0.5 * a * (1 + torch.tanh(math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3)))


def _exact_linear(s):
    c, grad = s["case"], s["case"]["op"] == "linear_grad"
    N, E = c["out"], max(c["experts"], 1)
    offsets = s["offsets"].tolist() if "offsets" in s else [0, c["rows"]]
    f64 = {"dtype": torch.float64, "device": "cuda"}
    R, K, Nw = c["rows"], c["in"], s["weight"].shape[1]
    if grad:
        out = {"x": torch.zeros(R, K, **f64), "weight": torch.zeros(E, Nw, K, **f64)}
        if c["bias"]:
            out["bias"] = torch.zeros(E, Nw, **f64)
    else:
        out = {"out": torch.zeros(R, N, **f64)}
        if c["save"]:
            out["preact"] = torch.zeros(R, Nw, **f64)
    for e in range(E):
        i, j = offsets[e], offsets[e + 1]
        if i == j:
            continue
        x, w = s["x"][i:j].double(), s["weight"][e].double()
        if grad:
            dz = s["dout"][i:j].double()
            if "preact" in s:
                z = s["preact"][i:j].double().requires_grad_()
                with torch.enable_grad():
                    y = _exact_act(z[:, :N], c["act"])
                    y = y * z[:, N:] if c["gated"] else y
                    dz = torch.autograd.grad(y, z, dz)[0]
            out["x"][i:j] = dz @ w
            out["weight"][e] = dz.T @ x
            if c["bias"]:
                out["bias"][e] = dz.sum(0)
        else:
            z = x @ w.T
            if c["bias"]:
                z = z + s["bias"][e].double()
            y = _exact_act(z[:, :N], c["act"])
            y = y * z[:, N:] if c["gated"] else y
            out["out"][i:j] = y + s["residual"][i:j].double() if c["residual"] else y
            if c["save"]:
                out["preact"][i:j] = z
    return out
