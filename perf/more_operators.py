"""Cases for measuring the operators around the expert layer: the whole layer for a few tokens, the norms around a
block, and the gradients' norm with clipping.

A case is one call of one operator:

  few        the whole W4A16 layer for a few tokens: router's choice, experts and weighted sum, with the residual added
  norm       v = rms(y) gamma_post, out = scale x + gate v, u = rms(out) gamma_pre: what stands between two blocks
  norm_grad  its gradient: x, y, both gammas and the gate
  clip       the norm over a list of gradients, and the gradients scaled down to a bound

With ``own`` false an operator is computed in its plain form: elementary torch operations in 32 bits, rounded once at
the end.  With ``own`` true ``run`` makes the calls of the library's binding.
"""
import math
from concurrent.futures import ThreadPoolExecutor

import numpy as np
import torch

own = False

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
TYPE_CODES = {"fp16": 0, "bf16": 1, "fp32": 2}
BYTES = {"fp16": 2, "bf16": 2, "fp32": 4}
FORMATS = {"zero": 0, "affine": 1, "symmetric": 2}
EPS = 1e-6


def _few(name, dtype, tokens, hidden, inter, experts, top_k, groups=(64, 64), fmt="zero", act="gelu", residual=False):
    return {"name": name, "op": "few", "dtype": dtype, "tokens": tokens, "hidden": hidden, "inter": inter,
            "experts": experts, "top_k": top_k, "group_gate_up": groups[0], "group_down": groups[1], "format": fmt,
            "act": act, "residual": residual}


def _norm(name, op, dtype, rows, hidden, form="both", gate_rows=0, scale=1.0):
    """form: "pre" (the norm before a block alone), "post" (norm, gate and residual after it) or "both" (the norm
    after a block with the next block's); gate_rows: rows that share a row of the gate, 0 without a gate."""
    return {"name": name, "op": op, "dtype": dtype, "rows": rows, "hidden": hidden, "form": form,
            "gate_rows": gate_rows, "scale": scale}


def _clip(name, dtypes, sizes, ratio, in_place=False, flat=False):
    """sizes: "AxB+C..." elements of the tensors; dtypes: their types in turn; ratio: the bound as a part of the
    norm that is expected; flat: the tensors lie end to end in one buffer per type, wherever that puts them."""
    return {"name": name, "op": "clip", "dtypes": dtypes, "sizes": sizes, "ratio": ratio, "in_place": in_place,
            "flat": flat}


def _many(count, lo, hi, seed):
    """count sizes between lo and hi, spread over their logarithm."""
    rng = np.random.default_rng(seed)
    return "+".join(str(int(round(math.exp(v)))) for v in rng.uniform(math.log(lo), math.log(hi), count))


def listed():
    return [
        # one token of a generation loop: 8 of 128 experts, their weights' way from memory
        _few("layer one token", "fp16", 1, 2048, 704, 128, 8),
        # a few requests decoded together in a bf16 model, affine weights
        _few("layer four tokens", "bf16", 4, 2048, 704, 128, 8, groups=(128, 64), fmt="affine", residual=True),
        # a small batch: most of its pairs meet different experts
        _few("layer 16 tokens", "fp16", 16, 2048, 704, 128, 8),
        # a layer whose sizes fit no tile: an odd number of experts, contractions that end in half a stage
        _few("layer ragged", "bf16", 7, 1152, 448, 60, 3, groups=(32, 64), fmt="symmetric", act="gelu_erf",
             residual=True),
        # between two blocks while one token is generated; latency only
        _norm("norm one row", "norm", "fp16", 1, 2048),
        # between two blocks of a training batch, with a learned gate per column
        _norm("norm 16384 rows", "norm", "bf16", 16384, 2048, gate_rows=16384),
        # after a block of a padded batch in 32 bits: a gate row per sequence, the residual scaled
        _norm("norm ragged", "norm", "fp32", 4099, 1000, form="post", gate_rows=300, scale=0.5),
        # the gradient of the training batch's
        _norm("norm gradient 16384 rows", "norm_grad", "bf16", 16384, 2048, gate_rows=16384),
        # the gradient with a gate row per sequence, sizes that fit no tile
        _norm("norm gradient ragged", "norm_grad", "fp16", 5003, 1000, gate_rows=300, scale=0.5),
        # the gradients of one 16-bit expert layer and its router, clipped into the optimizer's buffers
        _clip("clip expert layer", "bf16,bf16,fp32,fp32", "128x1408x2048+128x2048x704+128x1408+128x2048", 0.4),
        # many tensors of a whole model, one after the other in flat buffers: a step that stays below the bound
        _clip("clip many below bound", "bf16,fp32,bf16", _many(400, 30, 400000, 7), 2.0, in_place=True, flat=True),
        # a handful of small tensors (norms, biases, a router): latency only
        _clip("clip few small", "fp32", "2048+2048+1408+128x256+1", 0.7),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["few", "few", "norm", "norm", "norm_grad", "norm_grad", "clip", "clip"])
    if op == "few":
        experts = _log_int(rng, 4, 256)
        hidden, inter = 128 * _log_int(rng, 2, 32), 64 * _log_int(rng, 2, 32)
        experts = max(4, min(experts, (128 * 2048 * 704) // (hidden * inter)))
        top_k = rng.randint(1, min(8, experts))
        tokens = _log_int(rng, 1, 32)
        tokens = max(1, min(tokens, (16 * 8 * 2048 * 704) // (hidden * inter * top_k)))
        c = _few("", rng.choice(["fp16", "bf16"]), tokens, hidden, inter, experts, top_k,
                 groups=(rng.choice([32, 64, 128]), rng.choice([32, 64] + ([128] if inter % 128 == 0 else []))),
                 fmt=rng.choice(["zero", "affine", "symmetric"]), act=rng.choice(["gelu", "gelu_erf"]),
                 residual=rng.random() < 0.5)
    elif op == "clip":
        kinds = rng.choice(["fp16", "bf16", "fp32", "bf16,fp32", "fp16,bf16,fp32"])
        flat = rng.random() < 0.5
        count, top = _log_int(rng, 1, 500 if flat else 40), _log_int(rng, 16, 1 << 24)
        sizes = [_log_int(rng, 1, top) for _ in range(count)]
        while sum(sizes) > 1 << 28:
            sizes.pop()
        in_place = rng.random() < 0.3
        c = _clip("", kinds, "+".join(map(str, sizes)), 2.0 if in_place else rng.choice([0.1, 0.4, 2.0]), in_place,
                  flat=flat)
    else:
        dtype = rng.choice(["fp16", "bf16", "bf16", "fp32"])
        hidden = 8 * _log_int(rng, 8, 1024)
        rows = max(1, min(_log_int(rng, 1, 16384), (1 << 26) // (hidden * BYTES[dtype])))
        form = rng.choice(["pre", "post", "both", "both"])
        gate_rows = 0 if form == "pre" else rng.choice([0, rows, rng.randint(1, rows), 1])
        c = _norm("", op, dtype, rows, hidden, form, gate_rows, scale=rng.choice([1.0, 0.5]))
        if form == "pre":
            c["scale"] = 1.0
    del c["name"]
    return c


# ------------------------------------------------------------------- inputs


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": case}
    if own:
        from w4a16_moe_expert_router_gb300 import binding as B
        s["B"] = B
    {"few": _prepare_few, "clip": _prepare_clip}.get(case["op"], _prepare_norm)(s, case, g)
    return s


def _uniform(g, shape, lo, hi, dtype):
    return torch.rand(shape, generator=g, device="cuda").mul_(hi - lo).add_(lo).to(dtype)


def _prepare_few(s, c, g):
    T, d, f, E, k = c["tokens"], c["hidden"], c["inter"], c["experts"], c["top_k"]
    g1, g2, dt = c["group_gate_up"], c["group_down"], TYPES[c["dtype"]]
    s["x"] = torch.randn(T, d, generator=g, device="cuda", dtype=dt)
    s["logits"] = torch.randn(T, E, generator=g, device="cuda")
    if c["residual"]:
        s["residual"] = torch.randn(T, d, generator=g, device="cuda", dtype=dt)
    for part, rows, cols, group in (("gate_up", 2 * f, d, g1), ("down", d, f, g2)):
        s[part + "_q"] = torch.randint(0, 256, (E, rows, cols // 2), generator=g, device="cuda", dtype=torch.uint8)
        s[part + "_s"] = _uniform(g, (E, rows, cols // group), 0.005, 0.02, torch.float16)
        z = _uniform(g, (E, rows, cols // group), 6.0, 9.0, torch.float16)
        if c["format"] == "affine":
            z = (-z.float() * s[part + "_s"].float()).half()
        elif c["format"] == "symmetric":
            z = torch.full_like(z, 8.0)
        s[part + "_z"] = z
    if own:
        B = s["B"]
        make = lambda experts: B.make_shape(T, d, f, experts, min(k, experts), g1, g2,
                                            0 if c["act"] == "gelu" else 1, 0, FORMATS[c["format"]])
        s["shape"], one = make(E), make(1)
        for part, which in (("gate_up", B.GATE_UP), ("down", B.DOWN)):
            q, sc, z = (s.pop(part + "_q").cpu().numpy(), s.pop(part + "_s").cpu().numpy().view(np.uint16),
                        s.pop(part + "_z").cpu().numpy().view(np.uint16))
            with ThreadPoolExecutor(16) as pool:  # an expert's stream depends on that expert alone
                s[part] = torch.from_numpy(np.concatenate(list(pool.map(
                    lambda e: B.moe_w4a16_prepare(one, which, q[e:e + 1], sc[e:e + 1], z[e:e + 1]), range(E))))).cuda()
        s["ws"] = torch.empty(B.moe_w4a16_few_workspace_bytes(s["shape"]), dtype=torch.uint8, device="cuda")
        s["out"] = {"idx": torch.empty(T, k, dtype=torch.int32, device="cuda"),
                    "w": torch.empty(T, k, dtype=torch.float32, device="cuda"), "out": torch.empty_like(s["x"])}


def _prepare_norm(s, c, g):
    R, d, dt, form, gr = c["rows"], c["hidden"], TYPES[c["dtype"]], c["form"], c["gate_rows"]

    def rows(scale=1.0):
        return torch.randn(R, d, generator=g, device="cuda", dtype=dt).mul_(scale)

    def gamma():
        return torch.randn(d, generator=g, device="cuda").mul_(0.1).add_(1.0)

    if form != "pre":
        s["y"], s["gamma_post"] = rows(3.0), gamma()
        if gr:
            s["gate"] = torch.randn(-(-R // gr), d, generator=g, device="cuda").mul_(0.3).add_(0.5)
    if form != "post":
        s["gamma_pre"] = gamma()
    if c["op"] == "norm":
        s["x"] = rows(2.0)
    else:
        s["stream"], s["dout"] = rows(2.0), rows()  # the residual stream after the block, and its gradient
        if form != "post":
            s["du"] = rows()
    if own:
        B = s["B"]
        s["cfg"] = B.make_norm(R, d, TYPE_CODES[c["dtype"]], gr, c["scale"], EPS)
        like = lambda: torch.empty(R, d, dtype=dt, device="cuda")
        if c["op"] == "norm":
            s["out"] = {}
            if form != "pre":
                s["out"]["out"] = like()
            if form != "post":
                s["out"]["u"] = like()
        else:
            s["ws"] = torch.empty(B.moe_w4a16_norm_backward_workspace_bytes(s["cfg"]), dtype=torch.uint8,
                                  device="cuda")
            s["out"] = {"x": like()}
            if form != "pre":
                s["out"]["y"], s["out"]["gamma_post"] = like(), torch.empty_like(s["gamma_post"])
                if gr:
                    s["out"]["gate"] = torch.empty_like(s["gate"])
            if form != "post":
                s["out"]["gamma_pre"] = torch.empty_like(s["gamma_pre"])


def _clip_shapes(c):
    kinds = c["dtypes"].split(",")
    return [(tuple(int(v) for v in t.split("x")), kinds[i % len(kinds)]) for i, t in enumerate(c["sizes"].split("+"))]


def _clip_tensors(c):
    """The tensors of a list, new, one by one or end to end in one buffer per type; and what holds them all: the
    tensors themselves or the buffers."""
    shapes = _clip_shapes(c)
    if not c["flat"]:
        tensors = [torch.empty(shape, dtype=TYPES[kind], device="cuda") for shape, kind in shapes]
        return tensors, tensors
    flat, at, tensors = {}, {}, []
    for shape, kind in shapes:
        flat[kind] = flat.get(kind, 0) + math.prod(shape)
    flat = {kind: torch.empty(n, dtype=TYPES[kind], device="cuda") for kind, n in flat.items()}
    for shape, kind in shapes:
        n, i = math.prod(shape), at.get(kind, 0)
        tensors.append(flat[kind][i:i + n].view(shape))
        at[kind] = i + n
    return tensors, list(flat.values())


def _prepare_clip(s, c, g):
    s["grads"], s["held"] = _clip_tensors(c)
    square = 0.0
    for i, t in enumerate(s["grads"]):
        std = 0.01 * (1 + i % 7)  # layers differ in the size of their gradients
        t.normal_(0.0, std, generator=g)
        square += t.numel() * std * std
    s["max_norm"] = c["ratio"] * math.sqrt(square)
    if own:
        B = s["B"]
        outs, s["out"] = (s["grads"], s["held"]) if c["in_place"] else _clip_tensors(c)
        s["list"] = B.make_tensors(s["grads"], outs)
        s["norm"] = torch.empty(1, device="cuda")
        s["ws"] = torch.empty(B.moe_w4a16_clip_workspace_bytes(s["list"]), dtype=torch.uint8, device="cuda")


# ---------------------------------------------------------- the two forms


def run(s):
    return _own(s) if own else _PLAIN[s["case"]["op"]](s)


def _own(s):
    B, op, out = s["B"], s["case"]["op"], s.get("out")
    if op == "few":
        code = TYPE_CODES[s["case"]["dtype"]]
        B.moe_w4a16_few(s["shape"], code, s["x"], s["logits"], s["gate_up"], s["down"], s.get("residual"), out["idx"],
                        out["w"], out["out"], s["ws"])
    elif op == "norm":
        B.moe_w4a16_norm(s["cfg"], s["x"], s.get("y"), s.get("gamma_post"), s.get("gate"), s.get("gamma_pre"),
                         out.get("out"), out.get("u"))
    elif op == "norm_grad":
        B.moe_w4a16_norm_backward(s["cfg"], s.get("y"), s.get("gamma_post"), s.get("gate"), s["stream"],
                                  s.get("gamma_pre"), s["dout"], s.get("du"), out["x"], out.get("y"),
                                  out.get("gamma_post"), out.get("gate"), out.get("gamma_pre"), s["ws"])
    else:
        B.moe_w4a16_clip(s["list"], s["max_norm"], s["norm"], s["ws"])
        out = {"norm": s["norm"], "grads": out}
    return out


def _weights(s, part, experts):
    """Weights of some experts in 32 bits [n][rows][cols]."""
    q, sc, z = s[part + "_q"][experts], s[part + "_s"][experts].float(), s[part + "_z"][experts].float()
    codes = torch.stack([q & 15, q >> 4], -1).float()
    codes = codes.reshape(*q.shape[:2], sc.shape[2], -1)
    sc, z = sc[..., None], z[..., None]
    w = codes * sc + z if s["case"]["format"] == "affine" else (codes - z) * sc
    return w.reshape(*q.shape[:2], -1)


def _plain_few(s):
    c, x = s["case"], s["x"]
    T, f, k = c["tokens"], c["inter"], c["top_k"]
    val, idx = torch.sort(s["logits"], dim=1, descending=True, stable=True)
    val, idx = val[:, :k], idx[:, :k]
    w = torch.exp(val - val[:, :1])
    w = w / w.sum(1, keepdim=True)
    used, at = torch.unique(idx, return_inverse=True)
    out = torch.zeros(x.shape, device="cuda")
    step = 16  # experts at a time
    a = torch.empty(T, k, 2 * f, device="cuda")
    for i in range(0, used.numel(), step):
        z = torch.einsum("td,end->ten", x.float(), _weights(s, "gate_up", used[i:i + step]))
        here = (at >= i) & (at < i + step)
        a = torch.where(here[:, :, None], torch.gather(z, 1, (at - i).clamp(0, z.shape[1] - 1)[:, :, None].expand(
            T, k, 2 * f)), a)
    g, u = a[:, :, :f], a[:, :, f:]
    if c["act"] == "gelu":
        h = 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g))) * u
    else:
        h = 0.5 * g * (1 + torch.erf(g * math.sqrt(0.5))) * u
    for i in range(0, used.numel(), step):
        wd = _weights(s, "down", used[i:i + step])
        n = wd.shape[0]
        share = torch.where(((at >= i) & (at < i + n))[:, :, None], w[:, :, None] * h, torch.zeros((), device="cuda"))
        rows = torch.zeros(T, n, f, device="cuda").scatter_add_(1, (at - i).clamp(0, n - 1)[:, :, None].expand(T, k, f),
                                                                share)
        out = out + torch.einsum("tef,edf->td", rows, wd)
    if "residual" in s:
        out = out + s["residual"].float()
    return {"idx": idx.to(torch.int32), "w": w, "out": out.to(x.dtype)}


def _rows_gate(s):
    """The gate of every row, or None."""
    if "gate" not in s:
        return None
    return s["gate"][torch.arange(s["case"]["rows"], device="cuda") // s["case"]["gate_rows"]]


def _inverse_rms(v):
    return torch.rsqrt((v * v).mean(1, keepdim=True) + EPS)


def _plain_norm(s):
    c, dt = s["case"], s["x"].dtype
    out = c["scale"] * s["x"].float()
    res = {}
    if "y" in s:
        y = s["y"].float()
        v = y * _inverse_rms(y) * s["gamma_post"]
        gate = _rows_gate(s)
        out = out + (v if gate is None else gate * v)
        res["out"] = out.to(dt)
    if "gamma_pre" in s:
        res["u"] = (out * _inverse_rms(out) * s["gamma_pre"]).to(dt)
    return res


def _plain_norm_grad(s):
    c, dt = s["case"], s["stream"].dtype
    g = s["dout"].float()
    res = {}
    if "gamma_pre" in s:
        out, du = s["stream"].float(), s["du"].float()
        r = _inverse_rms(out)
        n, dn = out * r, du * s["gamma_pre"]
        g = g + r * (dn - n * (dn * n).mean(1, keepdim=True))
        res["gamma_pre"] = (du * n).sum(0)
    res["x"] = (c["scale"] * g).to(dt)
    if "y" in s:
        y, gate = s["y"].float(), _rows_gate(s)
        r = _inverse_rms(y)
        m = y * r
        dv = g if gate is None else gate * g
        dm = dv * s["gamma_post"]
        res["y"] = (r * (dm - m * (dm * m).mean(1, keepdim=True))).to(dt)
        res["gamma_post"] = (dv * m).sum(0)
        if gate is not None:
            group = torch.arange(c["rows"], device="cuda") // c["gate_rows"]
            res["gate"] = torch.zeros_like(s["gate"]).index_add_(0, group, g * m * s["gamma_post"])
    return res


def _plain_clip(s):
    square = torch.zeros((), dtype=torch.float64, device="cuda")
    for t in s["grads"]:
        v = t.double()
        square = square + (v * v).sum()
    norm = torch.sqrt(square)
    factor = torch.where(torch.isfinite(norm) & (norm > s["max_norm"]), s["max_norm"] / norm, torch.ones_like(norm))
    factor = factor.float()
    return {"norm": norm.float().reshape(1), "grads": [(t.float() * factor).to(t.dtype) for t in s["held"]]}


_PLAIN = {"few": _plain_few, "norm": _plain_norm, "norm_grad": _plain_norm_grad, "clip": _plain_clip}


# ------------------------------------------------------------------- work


def work(case):
    op = case["op"]
    if op == "few":
        T, d, f, E, k = case["tokens"], case["hidden"], case["inter"], case["experts"], case["top_k"]
        used = E * (1 - (1 - k / E) ** T)  # distinct experts chosen, evenly loaded
        expert = 3 * d * f // 2 + 8 * f * (d // case["group_gate_up"]) + 4 * d * (f // case["group_down"])
        rows = T * d * BYTES[case["dtype"]] * (3 if case["residual"] else 2) + T * E * 4 + 8 * T * k
        return {"bytes": used * expert + rows, "flops": 6 * T * k * d * f}
    if op == "clip":
        elements = [(math.prod(shape), BYTES[kind]) for shape, kind in _clip_shapes(case)]
        b = sum(n * w for n, w in elements)
        return {"bytes": b if case["in_place"] else 2 * b, "flops": 3 * sum(n for n, _ in elements)}
    R, d, form, gr = case["rows"], case["hidden"], case["form"], case["gate_rows"]
    if op == "norm":
        moved = {"pre": 2, "post": 3, "both": 4}[form]
    else:
        moved = {"pre": 4, "post": 4, "both": 6}[form]
    vectors = 4 * d * (2 if form == "both" else 1) + (4 * d * -(-R // gr) if gr else 0)
    if op == "norm_grad":
        vectors *= 2
    return {"bytes": moved * R * d * BYTES[case["dtype"]] + vectors, "flops": 5 * moved * R * d}


# --------------------------------------------------- the definition in 64 bits


def exact(case, seed):
    global own
    kept, own = own, False  # the inputs alone, without the library's handles
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    return {"few": _exact_few, "norm": _exact_norm, "norm_grad": _exact_norm_grad, "clip": _exact_clip}[case["op"]](s)


def _exact_matrix(s, part, e):
    q = s[part + "_q"][e].long()
    codes = torch.zeros(q.shape[0], 2 * q.shape[1], dtype=torch.float64, device="cuda")
    codes[:, 0::2] = (q % 16).double()
    codes[:, 1::2] = (q // 16).double()
    per = codes.shape[1] // s[part + "_s"].shape[2]
    sc = s[part + "_s"][e].double().repeat_interleave(per, 1)
    z = s[part + "_z"][e].double().repeat_interleave(per, 1)
    return sc * codes + z if s["case"]["format"] == "affine" else sc * (codes - z)


def _exact_few(s):
    c = s["case"]
    T, f, k = c["tokens"], c["inter"], c["top_k"]
    logits, x = s["logits"].double().cpu().numpy(), s["x"].double()
    idx = [sorted(range(c["experts"]), key=lambda e: (-logits[t, e], e))[:k] for t in range(T)]
    sel = torch.tensor([[logits[t, e] for e in idx[t]] for t in range(T)], dtype=torch.float64, device="cuda")
    w = torch.softmax(sel, 1)
    out = s["residual"].double() if "residual" in s else torch.zeros_like(x)
    for e in sorted({e for row in idx for e in row}):
        pairs = [(t, r) for t in range(T) for r in range(k) if idx[t][r] == e]
        t = torch.tensor([p[0] for p in pairs], device="cuda")
        r = torch.tensor([p[1] for p in pairs], device="cuda")
        z = x[t] @ _exact_matrix(s, "gate_up", e).T
        gate, up = z[:, :f], z[:, f:]
        if c["act"] == "gelu":
            h = gate * torch.sigmoid(math.sqrt(8 / math.pi) * (gate + 0.044715 * gate ** 3)) * up
        else:
            h = gate * torch.special.ndtr(gate) * up
        out[t] += w[t, r, None] * (h @ _exact_matrix(s, "down", e).T)
    return {"idx": None, "w": w, "out": out}


def _exact_gate(s):
    if "gate" not in s:
        return 1.0
    return s["gate"].double().repeat_interleave(s["case"]["gate_rows"], 0)[:s["case"]["rows"]]


def _exact_rms(v):
    return torch.sqrt((v ** 2).sum(1, keepdim=True) / v.shape[1] + EPS)


def _exact_norm(s):
    x, res = s["x"].double() * s["case"]["scale"], {}
    if "y" in s:
        y = s["y"].double()
        x = x + _exact_gate(s) * (s["gamma_post"].double() * (y / _exact_rms(y)))
        res["out"] = x
    if "gamma_pre" in s:
        res["u"] = s["gamma_pre"].double() * (x / _exact_rms(x))
    return res


def _exact_norm_grad(s):
    """Through autograd, from the definition of the forward step."""
    c, res = s["case"], {}
    with torch.enable_grad():
        # the stream that the next norm reads is given, so its gradient is taken there
        stream = s["stream"].double().requires_grad_()
        loss = (stream * s["dout"].double()).sum()
        if "gamma_pre" in s:
            gamma_pre = s["gamma_pre"].double().requires_grad_()
            u = gamma_pre * (stream / _exact_rms(stream))
            loss = loss + (u * s["du"].double()).sum()
            dstream, res["gamma_pre"] = torch.autograd.grad(loss, (stream, gamma_pre))
        else:
            dstream, = torch.autograd.grad(loss, stream)
        res["x"] = c["scale"] * dstream
        if "y" in s:
            leaves = [s["y"].double().requires_grad_(), s["gamma_post"].double().requires_grad_()]
            v = leaves[1] * (leaves[0] / _exact_rms(leaves[0]))
            if "gate" in s:
                leaves.append(s["gate"].double().requires_grad_())
                v = v * leaves[2].repeat_interleave(c["gate_rows"], 0)[:c["rows"]]
            grads = torch.autograd.grad((v * dstream).sum(), leaves)
            res["y"], res["gamma_post"] = grads[:2]
            if "gate" in s:
                res["gate"] = grads[2]
    return res


def _exact_clip(s):
    norm = math.sqrt(math.fsum(float(torch.linalg.vector_norm(t.double())) ** 2 for t in s["grads"]))
    factor = min(1.0, s["max_norm"] / norm) if norm else 1.0
    return {"norm": torch.tensor([norm], dtype=torch.float64, device="cuda"),
            "grads": [t.double() * factor for t in s["held"]]}
