"""The gradient of an MoE block's token path, and the layer norm: what each case runs, in plain torch and through the
library.

Five operators:

  ln        r = residual + x;  y = (r - mean(r)) / sqrt(var(r) + eps) * w + b, with optional E4M3 rows of the same
            values and one power-of-two scale per row (moe_add_layernorm);
  norm_bwd  the gradient of that norm, or of the RMS norm, at r: xh = (r - mean) rstd (RMS: r rstd), g = dy w,
            dr = dstream + rstd (g - mean(g) - xh mean(g xh)) (RMS: without mean(g)), dweight = sum over rows of dy xh,
            dbias = sum over rows of dy (moe_add_layernorm_bwd, moe_add_rmsnorm_bwd);
  combine   the gradient of the weighted combine out[t] = sum_j w[t,j] y[row(t,j)] + sigmoid(x[t] . ws) ysh[t]:
            dy[row(t,j)] = w[t,j] dout[t], dw[t,j] = y[row(t,j)] . dout[t], and of the gated shared expert dysh, the
            gate's logit dz and dws (moe_finalize_bwd);
  permute   the gradient of the rows sorted by expert, xp[row(t,j)] = w[t,j] x[t] (or x[t]):
            dx[t] = add[t] + sum_j w[t,j] dxp[row(t,j)] + dz[t] ws,  dw[t,j] = x[t] . dxp[row(t,j)] (moe_permute_bwd);
  route     the gradient of the routing weights w[t,j] = softmax(l[t])[id(t,j)], with or without division by their sum,
            with respect to the logits l (moe_route_bwd).

A pair (t, j) whose expert this rank does not hold has row -1: it adds nothing, and its dw is 0.
"""
import math

import torch

own = False

EPS = 1e-5


def _ln(name, T, H, f32, q8):
    return {"name": name, "op": "ln", "T": T, "H": H, "f32": f32, "q8": q8}


def _norm_bwd(name, T, H, rms, f32, stream):
    return {"name": name, "op": "norm_bwd", "T": T, "H": H, "rms": rms, "f32": f32, "stream": stream}


def _combine(name, T, H, E, k, gated, local):
    return {"name": name, "op": "combine", "T": T, "H": H, "E": E, "k": k, "gated": gated, "local": local}


def _permute(name, T, H, E, k, on_input, add, gated, local):
    return {"name": name, "op": "permute", "T": T, "H": H, "E": E, "k": k, "on_input": on_input, "add": add,
            "gated": gated, "local": local}


def _route(name, T, E, k, renorm):
    return {"name": name, "op": "route", "T": T, "E": E, "k": k, "renorm": renorm}


def listed():
    return [
        # one token in front of a 64-expert layer: latency
        _ln("ln_t1_h2048", 1, 2048, False, False),
        # the prompt of the large layer, its residual stream kept in 32 bits, rows for the 8-bit experts
        _ln("ln_t8192_h7168_f32_q8", 8192, 7168, True, True),
        # an odd number of tokens and a width that is no power of two
        _norm_bwd("ln_bwd_t777_h1408", 777, 1408, False, False, False),
        # a training step of the 60-expert layer, its stream and the stream's gradient in 32 bits
        _norm_bwd("ln_bwd_t4096_h2048_f32", 4096, 2048, False, True, True),
        # a training step of the largest layer
        _norm_bwd("rms_bwd_t16384_h7168", 16384, 7168, True, False, True),
        # a few tokens of the 64-expert layer: latency
        _combine("combine_t8_h2048_e64", 8, 2048, 64, 6, False, -1),
        # the 60-expert layer with its gated shared expert
        _combine("combine_t4096_h2048_e60_gated", 4096, 2048, 60, 4, True, -1),
        # the largest layer
        _combine("combine_t16384_h7168_e256", 16384, 7168, 256, 8, False, -1),
        # the 60-expert layer with its weights applied at the experts' input
        _permute("permute_t4096_h2048_e60_on_input", 4096, 2048, 60, 4, True, "", False, -1),
        # the large layer on a rank that holds half of its experts, added to the router's gradient in 32 bits
        _permute("permute_t8191_h7168_e256_local", 8191, 7168, 256, 8, False, "f32", False, 128),
        # the routing weights of the 60-expert layer (not renormalised) and of the largest layer
        _route("route_t4096_e60", 4096, 60, 4, False),
        _route("route_t16384_e256_renorm", 16384, 256, 8, True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ln", "norm_bwd", "norm_bwd", "combine", "permute", "route"])
    if op in ("ln", "norm_bwd"):
        H = 8 * _log(rng, 8, 1024)
        c = {"op": op, "T": _log(rng, 1, min(16384, 8192 * 7168 // H)), "H": H, "f32": rng.random() < 0.4}
        if op == "ln":
            c["q8"] = rng.random() < 0.5
        else:
            c["rms"], c["stream"] = rng.random() < 0.5, rng.random() < 0.6
        return c
    k = rng.randint(1, 8)
    E = max(2 * k, _log(rng, 8, 512))
    if op == "route":
        return {"op": op, "T": _log(rng, 1, 16384), "E": E, "k": k, "renorm": rng.random() < 0.5}
    H = 64 * _log(rng, 1, 112)
    c = {"op": op, "T": _log(rng, 1, min(16384, 16384 * 8 * 7168 // (2 * k * H))), "H": H, "E": E, "k": k,
         "gated": rng.random() < 0.4, "local": E // 2 if rng.random() < 0.3 else -1}
    if op == "permute":
        c["on_input"], c["add"] = rng.random() < 0.5, rng.choice(["", "bf16", "f32"])
    return c


# ------------------------------------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rows(T, H, g, std=1.0):
    return (torch.randn(T, H, generator=g, device="cuda") * std).to(torch.bfloat16)


def _stream(T, H, g, f32):
    r = torch.randn(T, H, generator=g, device="cuda") * 4.0 + 0.5  # a residual stream is wider than what one layer
    r[:, H // 3] *= 30.0                            # adds, off zero, and has a channel far larger than the rest
    return r if f32 else r.to(torch.bfloat16)


def _vec(H, g, mean, std):
    return (mean + std * torch.randn(H, generator=g, device="cuda")).to(torch.bfloat16)


def _tables(s, T, E, k, local, g):
    """The routing of a step, as moe_route and moe_permute leave it: k experts a token, pairs grouped by expert, pairs
    of experts that this rank does not hold dropped (row -1, weight 0)."""
    score, ids = torch.randn(T, E, generator=g, device="cuda").topk(k, dim=1)
    S = local if local >= 0 else E
    key = torch.where(ids < S, ids, S).reshape(-1)
    order = torch.argsort(key, stable=True)
    row = torch.empty_like(order)
    row[order] = torch.arange(T * k, device="cuda")
    keep = (key < S).reshape(T, k)
    s["pair_row"] = torch.where(keep, row.reshape(T, k), -1).to(torch.int32).contiguous()
    s["topk_w"] = torch.where(keep, torch.softmax(score, dim=1), 0.0).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    T = c["T"]
    s = {"op": c["op"], "T": T}
    empty = lambda *shape, dtype=torch.bfloat16: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    if c["op"] == "ln":
        H = c["H"]
        s["x"], s["residual"] = _rows(T, H, g), _stream(T, H, g, c["f32"])
        s["w"], s["b"] = _vec(H, g, 1.0, 0.2), _vec(H, g, 0.0, 0.2)
        s["residual_out"], s["y"] = torch.empty_like(s["residual"]), torch.empty_like(s["x"])
        s["q"] = empty(T, H, dtype=torch.uint8) if c["q8"] else None
        s["scale"] = empty(T, dtype=torch.float32) if c["q8"] else None
        return s
    if c["op"] == "norm_bwd":
        H = c["H"]
        s["rms"] = c["rms"]
        s["r"] = _stream(T, H, g, c["f32"])
        s["dy"] = _rows(T, H, g, 0.01)
        s["w"] = _vec(H, g, 1.0, 0.2)
        s["dstream"] = (torch.randn(T, H, generator=g, device="cuda") * 0.01).to(s["r"].dtype) if c["stream"] else None
        s["dr"] = torch.empty_like(s["r"])
        s["dx"] = empty(T, H) if c["f32"] else None
        s["dweight"] = empty(H, dtype=torch.float32)
        s["dbias"] = None if c["rms"] else empty(H, dtype=torch.float32)
        s["ws"] = torch.zeros(4096 + 2560 * H, dtype=torch.uint8, device="cuda")
        return s
    k, E = c["k"], c["E"]
    if c["op"] == "route":
        logits = torch.randn(T, E, generator=g, device="cuda") * 1.5
        top, ids = logits.topk(k, dim=1)
        s["renorm"] = c["renorm"]
        s["ids"] = ids.to(torch.int32)
        s["logits"] = None if c["renorm"] else logits
        s["topk_w"] = torch.softmax(top, dim=1) if c["renorm"] else torch.softmax(logits, dim=1).gather(1, ids)
        s["dtopk_w"] = torch.randn(T, k, generator=g, device="cuda")
        s["dlogits"] = empty(T, E, dtype=torch.float32)
        s["ws"] = torch.zeros(4096, dtype=torch.uint8, device="cuda")
        return s
    H = c["H"]
    _tables(s, T, E, k, c["local"], g)
    s["gated"] = c["gated"]
    s["gate_w"] = _vec(H, g, 0.0, 0.02) if c["gated"] else None
    s["ws"] = torch.zeros(4096 + 2560 * H, dtype=torch.uint8, device="cuda")
    if c["op"] == "combine":
        s["dout"] = _rows(T, H, g, 0.01)
        s["y"] = _rows(T * k, H, g)
        s["x"] = _rows(T, H, g) if c["gated"] else None
        s["ysh"] = _rows(T, H, g) if c["gated"] else None
        s["dy"] = torch.zeros(T * k, H, dtype=torch.bfloat16, device="cuda")
        s["dtopk_w"] = empty(T, k, dtype=torch.float32)
        s["dysh"] = empty(T, H) if c["gated"] else None
        s["dz"] = empty(T, dtype=torch.float32) if c["gated"] else None
        s["dgate_w"] = empty(H, dtype=torch.float32) if c["gated"] else None
        return s
    s["dxp"] = _rows(T * k, H, g, 0.01)
    s["x"] = _rows(T, H, g) if c["on_input"] else None
    s["add"] = None
    if c["add"]:
        s["add"] = torch.randn(T, H, generator=g, device="cuda") * 0.01
        s["add"] = s["add"].to(torch.bfloat16) if c["add"] == "bf16" else s["add"]
    s["dz"] = torch.randn(T, generator=g, device="cuda") * 0.05 if c["gated"] else None
    s["dx"] = empty(T, H)
    s["dtopk_w"] = empty(T, k, dtype=torch.float32) if c["on_input"] else None
    return s


# ------------------------------------------------------------------------------------------------ plain forms

def _plain_ln(s):
    r = s["residual"].float() + s["x"].float()
    d = r - r.mean(dim=1, keepdim=True)
    y = d * torch.rsqrt(d.square().mean(dim=1, keepdim=True) + EPS) * s["w"].float() + s["b"].float()
    out = {"residual": r.to(s["residual"].dtype), "y": y.to(torch.bfloat16)}
    if s["q"] is not None:
        m, e = torch.frexp(y.abs().amax(dim=1))  # amax = m 2^e, 1/2 <= m < 1; 448 = 0.875 2^9
        e = torch.clamp(e - 9 + (m > 0.875).to(e.dtype), min=-126)
        scale = torch.ldexp(torch.ones_like(m), e)
        out["q"] = (y / scale[:, None]).to(torch.float8_e4m3fn)
        out["scale"] = scale
    return out


def _plain_norm_bwd(s):
    r, dy = s["r"].float(), s["dy"].float()
    d = r if s["rms"] else r - r.mean(dim=1, keepdim=True)
    rstd = torch.rsqrt(d.square().mean(dim=1, keepdim=True) + EPS)
    xh = d * rstd
    g = dy * s["w"].float()
    dr = g - xh * (g * xh).mean(dim=1, keepdim=True)
    if not s["rms"]:
        dr = dr - g.mean(dim=1, keepdim=True)
    dr = dr * rstd
    if s["dstream"] is not None:
        dr = dr + s["dstream"].float()
    out = {"dr": dr.to(s["r"].dtype), "dweight": (dy * xh).sum(dim=0)}
    if s["dx"] is not None:
        out["dx"] = dr.to(torch.bfloat16)
    if not s["rms"]:
        out["dbias"] = dy.sum(dim=0)
    return out


def _plain_combine(s):
    T, k = s["pair_row"].shape
    H = s["dout"].shape[1]
    dout = s["dout"].float()
    row = s["pair_row"].long()
    keep = row >= 0
    dy = torch.zeros(T * k + 1, H, dtype=torch.bfloat16, device=dout.device)  # the last row takes what is dropped
    dtopk_w = torch.empty(T, k, device=dout.device)
    for j in range(k):
        dy[torch.where(keep[:, j], row[:, j], T * k)] = (s["topk_w"][:, j, None] * dout).to(torch.bfloat16)
        dtopk_w[:, j] = (s["y"][row[:, j].clamp(min=0)].float() * dout).sum(dim=1) * keep[:, j]
    out = {"dy": dy[:T * k], "dtopk_w": dtopk_w}
    if s["gated"]:
        x, ysh = s["x"].float(), s["ysh"].float()
        gate = torch.sigmoid(x @ s["gate_w"].float())
        dz = gate * (1.0 - gate) * (dout * ysh).sum(dim=1)
        out["dysh"] = (gate[:, None] * dout).to(torch.bfloat16)
        out["dz"] = dz
        out["dgate_w"] = dz @ x
    return out


def _plain_permute(s):
    T, k = s["pair_row"].shape
    row = s["pair_row"].long()
    keep = row >= 0
    dx = torch.zeros(s["dx"].shape, device=row.device) if s["add"] is None else s["add"].float()
    out = {}
    if s["x"] is not None:
        x = s["x"].float()
        out["dtopk_w"] = torch.empty(T, k, device=row.device)
    for j in range(k):
        d = s["dxp"][row[:, j].clamp(min=0)].float()
        if s["x"] is not None:
            out["dtopk_w"][:, j] = (x * d).sum(dim=1) * keep[:, j]
            dx = dx + torch.where(keep[:, j], s["topk_w"][:, j], 0.0)[:, None] * d
        else:
            dx = dx + keep[:, j, None] * d
    if s["gated"]:
        dx = dx + s["dz"][:, None] * s["gate_w"].float()
    out["dx"] = dx.to(torch.bfloat16)
    return out


def _plain_route(s):
    ids, w, dw = s["ids"].long(), s["topk_w"], s["dtopk_w"]
    c = (w * dw).sum(dim=1, keepdim=True)
    if s["renorm"]:
        dl = torch.zeros(s["dlogits"].shape, device=w.device)
        return {"dlogits": dl.scatter_add_(1, ids, w * (dw - c))}
    e = torch.exp(s["logits"] - s["logits"].amax(dim=1, keepdim=True))
    p = e / e.sum(dim=1, keepdim=True)
    return {"dlogits": (-c * p).scatter_add_(1, ids, w * dw)}


_PLAIN = {"ln": _plain_ln, "norm_bwd": _plain_norm_bwd, "combine": _plain_combine, "permute": _plain_permute,
          "route": _plain_route}


def run(state):
    s = state
    if not own:
        return _PLAIN[s["op"]](s)
    import serving_router_gate_gb300 as moe
    if s["op"] == "ln":
        moe.moe_add_layernorm(s["x"], s["residual"], s["w"], s["b"], EPS, s["residual_out"], s["y"], s["q"], s["scale"])
        out = {"residual": s["residual_out"], "y": s["y"]}
        if s["q"] is not None:
            out["q"] = s["q"].view(torch.float8_e4m3fn)
            out["scale"] = s["scale"]
        return out
    if s["op"] == "norm_bwd":
        if s["rms"]:
            moe.moe_add_rmsnorm_bwd(s["dy"], s["r"], s["w"], EPS, s["dstream"], s["dr"], s["dx"], s["dweight"], s["ws"])
        else:
            moe.moe_add_layernorm_bwd(s["dy"], s["r"], s["w"], EPS, s["dstream"], s["dr"], s["dx"], s["dweight"],
                                      s["dbias"], s["ws"])
        return {n: s[n] for n in ("dr", "dweight", "dx", "dbias") if s[n] is not None}
    if s["op"] == "combine":
        moe.moe_finalize_bwd(s["dout"], s["y"], s["pair_row"], s["topk_w"], s["ysh"], s["x"], s["gate_w"], s["dy"],
                             s["dtopk_w"], s["dysh"], s["dz"], s["dgate_w"], s["ws"])
        return {n: s[n] for n in ("dy", "dtopk_w", "dysh", "dz", "dgate_w") if s[n] is not None}
    if s["op"] == "permute":
        moe.moe_permute_bwd(s["dxp"], s["pair_row"], None if s["x"] is None else s["topk_w"], s["x"], s["add"], s["dz"],
                            s["gate_w"], s["dx"], s["dtopk_w"], s["ws"])
        return {n: s[n] for n in ("dtopk_w", "dx") if s[n] is not None}
    moe.moe_route_bwd(s["ids"], s["topk_w"], s["dtopk_w"], s["logits"], s["renorm"], s["dlogits"], s["ws"])
    return {"dlogits": s["dlogits"]}


# ----------------------------------------------------------------------------------------------- work, 64-bit values

def work(case):
    c = case
    T = c["T"]
    if c["op"] == "ln":
        H, sb = c["H"], 4 if c["f32"] else 2
        return {"bytes": T * H * (4 + 2 * sb + (1 if c["q8"] else 0)) + 4 * H + (4 * T if c["q8"] else 0),
                "flops": 9 * T * H}
    if c["op"] == "norm_bwd":
        H, sb = c["H"], 4 if c["f32"] else 2
        return {"bytes": T * H * (2 + sb * (3 if c["stream"] else 2) + (2 if c["f32"] else 0)) + 2 * H
                + 4 * H * (1 if c["rms"] else 2), "flops": 14 * T * H}
    k, E = c["k"], c["E"]
    if c["op"] == "route":
        return {"bytes": T * (4 * E * (1 if c["renorm"] else 2) + 12 * k),
                "flops": T * (E * (1 if c["renorm"] else 6) + 6 * k)}
    H = c["H"]
    P = T * k * (c["local"] / E if c["local"] >= 0 else 1.0)  # kept pairs, on average
    if c["op"] == "combine":
        return {"bytes": 2 * T * H + 4 * P * H + 12 * T * k + ((6 * T * H + 4 * T + 6 * H) if c["gated"] else 0),
                "flops": 3 * P * H + (7 * T * H if c["gated"] else 0)}
    add = {"": 0, "bf16": 2, "f32": 4}[c["add"]]
    return {"bytes": 2 * P * H + T * H * (2 + add + (2 if c["on_input"] else 0)) + T * k * (12 if c["on_input"] else 4)
            + ((4 * T + 2 * H) if c["gated"] else 0),
            "flops": P * H * (4 if c["on_input"] else 1) + T * H * ((1 if add else 0) + (2 if c["gated"] else 0))}


def _exact_e4m3(v):
    """v rounded to the nearest E4M3 value, ties to even (|v| <= 448)."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), torch.clamp(e - 1, min=-6) - 3)
    return torch.round(v / step) * step


def _exact_norm(r, w, b, rms):
    """The norm's definition in 64 bits, on rows that may carry gradients."""
    var = (r * r).mean(dim=1) if rms else torch.var(r, dim=1, unbiased=False)
    shift = 0.0 if rms else r.mean(dim=1, keepdim=True)
    y = (r - shift) / torch.sqrt(var + EPS)[:, None] * w
    return y if b is None else y + b


def _leaf(t):
    return t.double().requires_grad_()


def exact(case, seed):
    """Forward formulas in 64 bits; gradients by differentiating them, some rows at a time."""
    s = prepare(case, seed)
    T = s["T"]
    if s["op"] == "ln":
        r = s["residual"].double() + s["x"].double()
        y = _exact_norm(r, s["w"].double(), s["b"].double(), False)
        out = {"residual": r, "y": y}
        if s["q"] is not None:
            amax = y.abs().max(dim=1).values
            e = torch.ceil(torch.log2(amax / 448.0)).clamp(min=-126)
            e = torch.where(amax <= 448.0 * torch.exp2(e - 1), e - 1, e)
            e = torch.where(amax > 448.0 * torch.exp2(e), e + 1, e)
            e = e.clamp(min=-126)
            out["q"] = _exact_e4m3(y * torch.exp2(-e)[:, None])
            out["scale"] = torch.exp2(e)
        return out
    if s["op"] == "norm_bwd":
        w = _leaf(s["w"])
        b = None if s["rms"] else torch.zeros_like(w).requires_grad_()
        dr = []
        for i in range(0, T, 2048):
            r = _leaf(s["r"][i:i + 2048])
            y = _exact_norm(r, w, b, s["rms"])
            y.backward(s["dy"][i:i + 2048].double())
            dr.append(r.grad if s["dstream"] is None else r.grad + s["dstream"][i:i + 2048].double())
        dr = torch.cat(dr)
        out = {"dr": dr, "dweight": w.grad}
        if s["dx"] is not None:
            out["dx"] = dr
        if b is not None:
            out["dbias"] = b.grad
        return out
    if s["op"] == "route":
        dl = []
        for i in range(0, T, 4096):
            ids = s["ids"][i:i + 4096].long()
            if s["renorm"]:  # the logits only matter up to a shift of the chosen ones: their weights' logarithms
                lg = torch.zeros(s["dlogits"][i:i + 4096].shape, dtype=torch.float64, device=ids.device)
                lg = lg.scatter(1, ids, s["topk_w"][i:i + 4096].double().log()).requires_grad_()
                w = torch.softmax(lg.gather(1, ids), dim=1)
            else:
                lg = _leaf(s["logits"][i:i + 4096])
                w = torch.softmax(lg, dim=1).gather(1, ids)
            w.backward(s["dtopk_w"][i:i + 4096].double())
            dl.append(lg.grad)
        return {"dlogits": torch.cat(dl)}
    k = s["pair_row"].shape[1]
    H = case["H"]
    step = max(1, 2 ** 27 // (k * H))
    gw = _leaf(s["gate_w"]) if s["gated"] else None
    if s["op"] == "combine":
        out = {"dy": torch.zeros(T * k, H, dtype=torch.float64, device="cuda"),
               "dtopk_w": torch.zeros(T, k, dtype=torch.float64, device="cuda")}
        dysh, dz = [], []
        for i in range(0, T, step):
            row = s["pair_row"][i:i + step].long()
            live = (row >= 0).nonzero()
            y, w = _leaf(s["y"][row[live[:, 0], live[:, 1]]]), _leaf(s["topk_w"][i:i + step])
            o = torch.zeros(row.shape[0], H, dtype=torch.float64, device="cuda")
            o = o.index_add(0, live[:, 0], y * w[live[:, 0], live[:, 1]][:, None])
            if gw is not None:
                ysh = _leaf(s["ysh"][i:i + step])
                z = (s["x"][i:i + step].double() * gw).sum(dim=1)
                z.retain_grad()
                o = o + ysh / (1.0 + torch.exp(-z))[:, None]
            o.backward(s["dout"][i:i + step].double())
            out["dy"][row[live[:, 0], live[:, 1]]] = y.grad
            out["dtopk_w"][i:i + step] = w.grad
            if gw is not None:
                dysh.append(ysh.grad)
                dz.append(z.grad)
        if gw is not None:
            out["dysh"], out["dz"], out["dgate_w"] = torch.cat(dysh), torch.cat(dz), gw.grad
        return out
    dx, dw = [], []
    for i in range(0, T, step):
        row = s["pair_row"][i:i + step].long()
        live = (row >= 0).nonzero()
        x = torch.zeros(row.shape[0], H, dtype=torch.float64, device="cuda") if s["x"] is None else s["x"][i:i + step]
        x = _leaf(x)
        xp = x[live[:, 0]]
        if s["x"] is not None:
            w = _leaf(s["topk_w"][i:i + step])
            xp = xp * w[live[:, 0], live[:, 1]][:, None]
        xp.backward(s["dxp"][row[live[:, 0], live[:, 1]]].double())
        d = x.grad
        if s["add"] is not None:
            d = d + s["add"][i:i + step].double()
        if gw is not None:
            d = d + torch.outer(s["dz"][i:i + step].double(), gw.detach())
        dx.append(d)
        if s["x"] is not None:
            dw.append(w.grad)
    out = {"dx": torch.cat(dx)}
    if dw:
        out["dtopk_w"] = torch.cat(dw)
    return out
