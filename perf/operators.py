"""The operators around and inside one MoE block at decode: what each case runs, in plain torch and through the library.

Three operators:

  norm     r' = r + x;  y = bf16(r' * rsqrt(mean(r'^2) + eps) * w), with optional E4M3 rows of the same values and one
           power-of-two scale per row (moe_add_rmsnorm);
  matvec   y[m] = x[m] W^T for a few rows x and a matrix of 4-bit weights, W[n][k] = s[n][k / group] * c[n][k],
           c in -8..7 (moe_matvec_w4);
  experts  the routed experts (and a shared expert) on such weights: per kept pair (t, j) of a token and an expert slot,
           y = W2 h, h = silu(W1_gate x) * (W1_up x); out[t] = sum_j w[t][j] y[t][j] + sigmoid(x . w_s) shared(x)
           (moe_forward_w4).

The packed weights hold eight elements in each 32-bit word (little-endian): element 2i in nibble i, element 2i + 1 in
nibble i + 4, each as c + 8.
"""
import math

import torch

own = False

EPS = 1e-6


def _norm(name, T, H, f32, q8):
    return {"name": name, "op": "norm", "T": T, "H": H, "f32": f32, "q8": q8}


def _matvec(name, M, N, K, group):
    return {"name": name, "op": "matvec", "M": M, "N": N, "K": K, "group": group}


def _experts(name, T, H, I, E, k, group, I_sh, gated, local):
    return {"name": name, "op": "experts", "T": T, "H": H, "I": I, "E": E, "k": k, "group": group, "I_sh": I_sh,
            "gated": gated, "local": local}


def listed():
    return [
        # one token between the attention and a 64-expert layer: latency
        _norm("norm_t1_h2048", 1, 2048, False, False),
        # a decode batch on the large layer, its residual stream kept in 32 bits, rows for the 8-bit experts
        _norm("norm_t32_h7168_f32_q8", 32, 7168, True, True),
        # an odd number of tokens and a width that is no power of two
        _norm("norm_t777_h1408_q8", 777, 1408, False, True),
        # the prompt of the largest layer, with 8-bit rows
        _norm("norm_t16384_h7168_q8", 16384, 7168, False, True),
        # one token through a square projection of the 64-expert layer: latency
        _matvec("matvec_m1_2048x2048", 1, 2048, 2048, 128),
        # one token through a vocabulary-sized projection
        _matvec("matvec_m1_65536x7168", 1, 65536, 7168, 128),
        # a decode batch through one expert-sized matrix, smaller groups
        _matvec("matvec_m8_4096x7168_g64", 8, 4096, 7168, 64),
        # odd numbers of rows and outputs, the smallest groups
        _matvec("matvec_m13_5633x1408_g32", 13, 5633, 1408, 32),
        # the 64-expert layer with its shared experts: one token, and a batch
        _experts("experts_t1_h2048_e64", 1, 2048, 1408, 64, 6, 128, 5632, False, -1),
        _experts("experts_t32_h2048_e64", 32, 2048, 1408, 64, 6, 128, 5632, False, -1),
        # the 60-expert layer with its gated shared expert, smaller groups, an odd batch
        _experts("experts_t7_h2048_e60_g64", 7, 2048, 1408, 60, 4, 64, 5632, True, -1),
        # the large layer: a batch of eight tokens over 256 experts
        _experts("experts_t8_h7168_e256", 8, 7168, 2048, 256, 8, 128, 0, False, -1),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _steps(rng, step, lo, hi):
    """A multiple of step, spread over the logarithm of lo..hi steps; 1536 and 3072 give way to the next one."""
    v = step * _log(rng, lo, hi)
    return v + step if v in (1536, 3072) else v


def draw(rng):
    op = rng.choice(["norm", "matvec", "experts"])
    if op == "norm":
        H = _steps(rng, 8, 8, 1024)
        return {"op": "norm", "T": _log(rng, 1, min(16384, 16384 * 7168 // H)), "H": H, "f32": rng.random() < 0.4,
                "q8": rng.random() < 0.6}
    group = rng.choice([32, 64, 128])
    if op == "matvec":
        K = _steps(rng, group, 1, 16384 // group)
        return {"op": "matvec", "M": _log(rng, 1, 32), "N": _log(rng, 1, min(65536, 65536 * 7168 // K)), "K": K,
                "group": group}
    H = _steps(rng, 128, 1, 56)
    I = _steps(rng, 128, 1, 16)
    k = rng.randint(1, 8)
    E = max(k, _log(rng, 4, min(256, 256 * 7168 * 2048 // (H * I))))
    T = _log(rng, 1, 64)
    while T > 1 and T * k * H * I > 64 * 7168 * 2048:
        T = max(1, T * 3 // 4)
    I_sh = rng.choice([0, 0, I, 2 * I])
    return {"op": "experts", "T": T, "H": H, "I": I, "E": E, "k": k, "group": group, "I_sh": I_sh,
            "gated": I_sh > 0 and rng.random() < 0.5, "local": E // 2 if E >= 8 and rng.random() < 0.25 else -1}


# ------------------------------------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _codes(shape, g):
    """Packed 4-bit codes, each nibble the rounded mean of two uniform ones: bell-shaped about 0, all of -8..7."""
    a = torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8)
    b = torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8)
    lo = ((a & 15) + (b & 15) + 1) >> 1
    hi = ((a >> 4) + (b >> 4) + 1) >> 1
    return lo | (hi << 4)


def _w4(rows, K, group, g):
    """A packed matrix (or a stack of them) with group scales that give weights of about 0.02."""
    s = torch.rand(rows + (K // group,), generator=g, device="cuda") * 0.004 + 0.004
    return _codes(rows + (K // 2,), g), s.to(torch.bfloat16)


def _rows(T, H, g):
    return torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    s = {"op": c["op"]}
    if c["op"] == "norm":
        T, H = c["T"], c["H"]
        r = torch.randn(T, H, generator=g, device="cuda") * 4.0  # a residual stream is wider than what one layer adds
        r[:, H // 3] *= 30.0                                       # and has a channel that is far larger than the rest
        s["x"] = _rows(T, H, g)
        s["residual"] = r if c["f32"] else r.to(torch.bfloat16)
        s["w"] = (1.0 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(torch.bfloat16)
        s["residual_out"] = torch.empty_like(s["residual"])
        s["y"] = torch.empty_like(s["x"])
        s["q"] = torch.empty(T, H, dtype=torch.uint8, device="cuda") if c["q8"] else None
        s["scale"] = torch.empty(T, dtype=torch.float32, device="cuda") if c["q8"] else None
        return s
    if c["op"] == "matvec":
        s["x"] = _rows(c["M"], c["K"], g)
        s["wq"], s["ws"] = _w4((c["N"],), c["K"], c["group"], g)
        s["y"] = torch.empty(c["M"], c["N"], dtype=torch.bfloat16, device="cuda")
        return s
    T, H, I, E, k, grp, I_sh = c["T"], c["H"], c["I"], c["E"], c["k"], c["group"], c["I_sh"]
    S = c["local"] if c["local"] >= 0 else E
    s["x"] = _rows(T, H, g)
    s["w1q"], s["w1s"] = _w4((S, 2 * I), H, grp, g)
    s["w2q"], s["w2s"] = _w4((S, H), I, grp, g)
    for n in ("sh1q", "sh1s", "sh2q", "sh2s", "gate"):
        s[n] = None
    if I_sh:
        s["sh1q"], s["sh1s"] = _w4((2 * I_sh,), H, grp, g)
        s["sh2q"], s["sh2s"] = _w4((H,), I_sh, grp, g)
        if c["gated"]:
            s["gate"] = (torch.randn(H, generator=g, device="cuda") * 0.02).to(torch.bfloat16)
    # the routing of a step, as moe_route and moe_permute leave it: k experts a token, pairs grouped by slot, and
    # pairs of slots that this rank does not hold dropped (row -1)
    score, ids = torch.randn(T, E, generator=g, device="cuda").topk(k, dim=1)
    s["topk_w"] = torch.softmax(score, dim=1).contiguous()
    slot = ids.reshape(-1)
    key = torch.where(slot < S, slot, S)
    order = torch.argsort(key, stable=True)
    counts = torch.bincount(key, minlength=S + 1)[:S]
    s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    row = torch.empty_like(order)
    row[order] = torch.arange(T * k, device="cuda")
    s["pair_row"] = torch.where(key < S, row, -1).reshape(T, k).to(torch.int32).contiguous()
    s["perm_src"] = order.to(torch.int32)
    s["out"] = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    # zero-filled, as moe_workspace_init leaves a workspace's header
    s["work"] = torch.zeros(4096 + T * k * (2 * I + 4 * H) + T * (2 * I_sh + 4 * H), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------------------------------------ plain forms

def _plain_weights(q, s):
    """The 32-bit weights [..., K] of packed codes [..., K / 2] and scales [..., K / group]."""
    b = q.reshape(q.shape[:-1] + (-1, 4, 1))
    n = torch.cat([b & 15, b >> 4], dim=-1).flatten(-2)                   # [..., K / 8, 8]: nibble order
    w = torch.stack([n[..., :4], n[..., 4:]], dim=-1).flatten(-3).float() - 8.0
    return (w.reshape(s.shape + (-1,)) * s.float().unsqueeze(-1)).flatten(-2)


def _plain_norm(s):
    r = s["residual"].float() + s["x"].float()
    y = r * torch.rsqrt(r.square().mean(dim=1, keepdim=True) + EPS) * s["w"].float()
    out = {"residual": r.to(s["residual"].dtype), "y": y.to(torch.bfloat16)}
    if s["q"] is not None:
        m, e = torch.frexp(y.abs().amax(dim=1))                            # amax = m 2^e, 1/2 <= m < 1; 448 = 0.875 2^9
        e = torch.clamp(e - 9 + (m > 0.875).to(e.dtype), min=-126)
        scale = torch.ldexp(torch.ones_like(m), e)
        out["q"] = (y / scale[:, None]).to(torch.float8_e4m3fn)
        out["scale"] = scale
    return out


def _plain_mlp(x, w1, w2):
    """The gated MLP of each of x's rows [P, H] with its own (or one common) weights w1 [., 2I, H], w2 [., H, I]."""
    gu = torch.matmul(w1, x.unsqueeze(-1)).squeeze(-1) if w1.dim() == 3 else x @ w1.t()
    gate, up = gu.chunk(2, dim=-1)
    h = gate / (1.0 + torch.exp(-gate)) * up
    return torch.matmul(w2, h.unsqueeze(-1)).squeeze(-1) if w2.dim() == 3 else h @ w2.t()


def _plain_experts(s):
    T, k = s["pair_row"].shape
    x = s["x"].float()
    S = s["w1q"].shape[0]
    rows = torch.arange(T * k, device=x.device, dtype=torch.int32)
    slot = torch.searchsorted(s["offsets"], rows, right=True).sub(1).clamp(max=S - 1)
    xr = x[(s["perm_src"] // k).long()]
    y = _plain_mlp(xr, _plain_weights(s["w1q"][slot], s["w1s"][slot]), _plain_weights(s["w2q"][slot], s["w2s"][slot]))
    pr = s["pair_row"].long()
    w = torch.where(pr >= 0, s["topk_w"], torch.zeros_like(s["topk_w"]))
    out = (y[pr.clamp(min=0)] * w.unsqueeze(-1)).sum(dim=1)
    if s["sh1q"] is not None:
        sh = _plain_mlp(x, _plain_weights(s["sh1q"], s["sh1s"]), _plain_weights(s["sh2q"], s["sh2s"]))
        if s["gate"] is not None:
            sh = sh / (1.0 + torch.exp(-(x @ s["gate"].float()))).unsqueeze(-1)
        out = out + sh
    return {"out": out.to(torch.bfloat16)}


def run(state):
    s = state
    if not own:
        if s["op"] == "norm":
            return _plain_norm(s)
        if s["op"] == "matvec":
            return {"y": (s["x"].float() @ _plain_weights(s["wq"], s["ws"]).t()).to(torch.bfloat16)}
        return _plain_experts(s)
    import serving_router_gate_gb300 as moe
    if s["op"] == "norm":
        moe.moe_add_rmsnorm(s["x"], s["residual"], s["w"], EPS, s["residual_out"], s["y"], s["q"], s["scale"])
        out = {"residual": s["residual_out"], "y": s["y"]}
        if s["q"] is not None:
            out["q"] = s["q"].view(torch.float8_e4m3fn)
            out["scale"] = s["scale"]
        return out
    if s["op"] == "matvec":
        moe.moe_matvec_w4(s["x"], s["wq"], s["ws"], s["y"])
        return {"y": s["y"]}
    moe.moe_forward_w4(s["x"], s["offsets"], s["perm_src"], s["w1q"], s["w1s"], s["w2q"], s["w2s"], s["pair_row"],
                       s["topk_w"], s["sh1q"], s["sh1s"], s["sh2q"], s["sh2s"], s["gate"], s["out"], s["work"])
    return {"out": s["out"]}


# ------------------------------------------------------------------------------------------------ work and 64-bit values

def work(case):
    c = case
    if c["op"] == "norm":
        n = c["T"] * c["H"]
        return {"bytes": n * (2 + 2 * (4 if c["f32"] else 2) + 2 + (1 if c["q8"] else 0)) + 2 * c["H"]
                + (4 * c["T"] if c["q8"] else 0), "flops": 6 * n}
    per = 0.5 + 2.0 / c["group"]  # bytes of a weight
    if c["op"] == "matvec":
        return {"bytes": c["N"] * c["K"] * per + 2 * c["M"] * (c["N"] + c["K"]), "flops": 2 * c["M"] * c["N"] * c["K"]}
    T, H, I, E, k, I_sh = c["T"], c["H"], c["I"], c["E"], c["k"], c["I_sh"]
    S = c["local"] if c["local"] >= 0 else E
    used = S * (1.0 - (1.0 - k / E) ** T)  # slots that a step of T tokens touches, on average
    mats = used * 3 * H * I + 3 * H * I_sh
    return {"bytes": mats * per + 4 * T * H + T * k * 12, "flops": 6 * T * H * (k * S / E * I + I_sh)}


def _exact_weights(q, s):
    K = 2 * q.shape[-1]
    i = torch.arange(K, device=q.device)
    nib = (i % 8) // 2 + 4 * (i % 2)                      # nibble of element i in its word of eight
    byte = 4 * (i // 8) + nib // 2
    c = (q.index_select(-1, byte).to(torch.int16) >> (4 * (nib % 2)).to(torch.int16)) & 15
    return (c - 8).double() * s.double().repeat_interleave(K // s.shape[-1], dim=-1)


def _exact_e4m3(v):
    """v rounded to the nearest E4M3 value, ties to even (|v| <= 448)."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), torch.clamp(e - 1, min=-6) - 3)
    return torch.round(v / step) * step


def _exact_mlp(x, w1, w2):
    gu = w1 @ x
    n = gu.shape[0] // 2
    h = gu[:n] * torch.sigmoid(gu[:n]) * gu[n:]
    return w2 @ h


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "norm":
        r = s["residual"].double() + s["x"].double()
        y = s["w"].double() * r / torch.sqrt(torch.mean(r * r, dim=1, keepdim=True) + EPS)
        out = {"residual": r, "y": y}
        if s["q"] is not None:
            amax = y.abs().max(dim=1).values
            e = torch.ceil(torch.log2(amax / 448.0)).clamp(min=-126)
            e = torch.where(amax <= 448.0 * torch.exp2(e - 1), e - 1, torch.where(amax > 448.0 * torch.exp2(e), e + 1, e))
            e = e.clamp(min=-126)
            out["q"] = _exact_e4m3(y * torch.exp2(-e)[:, None])
            out["scale"] = torch.exp2(e)
        return out
    if s["op"] == "matvec":
        step = 8192
        parts = [_exact_weights(s["wq"][n:n + step], s["ws"][n:n + step]) @ s["x"].double().t()
                 for n in range(0, s["wq"].shape[0], step)]
        return {"y": torch.cat(parts).t().contiguous()}
    T, k = s["pair_row"].shape
    x = s["x"].double()
    out = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    off, src = s["offsets"].tolist(), s["perm_src"].tolist()
    w = s["topk_w"].double().reshape(-1)
    for e in range(len(off) - 1):
        if off[e] == off[e + 1]:
            continue
        pairs = torch.tensor(src[off[e]:off[e + 1]], device=x.device)
        t = pairs // k
        y = _exact_mlp(x[t].t(), _exact_weights(s["w1q"][e], s["w1s"][e]), _exact_weights(s["w2q"][e], s["w2s"][e]))
        out.index_add_(0, t, y.t() * w[pairs][:, None])
    if s["sh1q"] is not None:
        sh = _exact_mlp(x.t(), _exact_weights(s["sh1q"], s["sh1s"]), _exact_weights(s["sh2q"], s["sh2s"])).t()
        if s["gate"] is not None:
            sh = sh * torch.sigmoid(x @ s["gate"].double())[:, None]
        out = out + sh
    return {"out": out}
