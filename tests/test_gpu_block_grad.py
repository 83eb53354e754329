"""The gradient calls together, as a training step of one MoE block uses them: the norm, the router, the permutation, the
experts (their products and gradients in torch), the combine with its gated shared expert, and the way back; and
MoELayer.block with a layer norm.

The reference differentiates the 64-bit block with the step's expert choice.  A bf16 rounding moves a tensor by at most
2^-8 of its norm.  At most four lie on a gradient's way back (dy, the experts' dx_perm, dx, dr or its copy) and four on the
values it is made of (the norm's rows, x_perm, y, y_shared); each is carried on by sums and products with random
matrices, which keep relative norms within a factor of 2: 8 * 2 * 2^-8 = 2^-4.  A term left out or counted twice moves
a gradient by more: the smallest part of any of them, the router's, is checked to be at least 2^-3 of the whole."""
import pytest
import torch

import serving_router_gate_gb300 as moe
from serving_router_gate_gb300.layer import MoELayer

import bwd_ref as ref

pytestmark = pytest.mark.gpu

T, H, I, I_SH, E, K, EPS = 96, 256, 128, 192, 8, 3, 1e-5
TOL = 2.0 ** -4


def _params(seed=0):
    p = dict(x=ref.rnd(T, H, seed=seed), r=ref.rnd(T, H, seed=seed + 1, std=2.0),
             nw=(1.0 + 0.2 * ref.rnd(H, seed=seed + 2, dtype=torch.float32)).to(torch.bfloat16),
             nb=ref.rnd(H, seed=seed + 3, std=0.2), Wg=ref.rnd(E, H, seed=seed + 4, std=0.15, dtype=torch.float32),
             bias=ref.rnd(E, seed=seed + 5, dtype=torch.float32), W1=ref.rnd(E, 2 * I, H, seed=seed + 6, std=H ** -0.5),
             W2=ref.rnd(E, H, I, seed=seed + 7, std=I ** -0.5), S1=ref.rnd(2 * I_SH, H, seed=seed + 8, std=H ** -0.5),
             S2=ref.rnd(H, I_SH, seed=seed + 9, std=I_SH ** -0.5), gw=ref.rnd(H, seed=seed + 10, std=0.1),
             dout=ref.rnd(T, H, seed=seed + 11), dstream=ref.rnd(T, H, seed=seed + 12))
    return p


def _mlp(x, w1, w2):
    g, u = (x @ w1.t()).chunk(2, dim=-1)
    return (torch.nn.functional.silu(g) * u) @ w2.t()


def _grouped(xp, off, w1, w2):
    """Rows of xp per expert through its gated MLP; rows behind the last stay 0."""
    out = [_mlp(xp[off[e]:off[e + 1]], w1[e], w2[e]) for e in range(len(off) - 1)]
    return torch.cat(out + [torch.zeros(xp.shape[0] - off[-1], w2.shape[1], dtype=xp.dtype, device=xp.device)])


def _step(p, ln, renorm, on_input, local):
    """One step with the library; returns the gradients by name, and the choice of experts."""
    bf = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    f32 = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    i32 = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    start, count = local
    S = E if count < 0 else count
    ws = torch.empty(max(moe.moe_workspace_size(T, H, I, E, E, K, I_SH), moe.moe_workspace_size_bwd(H)), dtype=torch.uint8,
                     device="cuda")
    moe.moe_workspace_init(ws)
    stream, xn = bf(T, H), bf(T, H)
    if ln:
        moe.moe_add_layernorm(p["x"], p["r"], p["nw"], p["nb"], EPS, stream, xn)
    else:
        moe.moe_add_rmsnorm(p["x"], p["r"], p["nw"], EPS, stream, xn)
    ids, w = i32(T, K), f32(T, K)
    moe.moe_route(xn, p["Wg"], p["bias"], K, renorm, ids, w, ws)
    w_all = w.clone()                                   # moe_permute zeroes the weights of other ranks' experts
    slot, cnt, off, src, pr, xp = i32(T, K), i32(S), i32(S + 1), i32(T * K), i32(T, K), torch.zeros(T * K, H, device="cuda",
                                                                                                    dtype=torch.bfloat16)
    moe.moe_permute(ids, w, E, None, None, E, start, count, moe.MOE_NONLOCAL_SKIP, xn, slot, cnt, off, src, pr, xp, ws,
                    on_input=on_input)
    o = off.tolist()
    W1, W2 = p["W1"][start:start + S].double(), p["W2"][start:start + S].double()
    xpd = xp.double().requires_grad_()
    yd = _grouped(xpd, o, W1, W2)
    y = yd.detach().to(torch.bfloat16)
    xnd = xn.double().requires_grad_()
    ysd = _mlp(xnd, p["S1"].double(), p["S2"].double())
    ysh = ysd.detach().to(torch.bfloat16)
    out = bf(T, H)
    moe.moe_finalize(y, pr, None if on_input else w, ysh, xn, p["gw"], out, ws)
    # and back
    g = dict(dgw=f32(H), dWg=None, dnw=f32(H), dnb=f32(H) if ln else None)
    dy, dw, dysh, dz = torch.zeros_like(y), f32(T, K), bf(T, H), f32(T)
    moe.moe_finalize_bwd(p["dout"], None if on_input else y, pr, None if on_input else w, ysh, xn, p["gw"], dy,
                         None if on_input else dw, dysh, dz, g["dgw"], ws)
    yd.backward(dy.double())
    ysd.backward(dysh.double())
    dxp = xpd.grad.to(torch.bfloat16)
    dxn = bf(T, H)
    if on_input:                                        # the weights' gradients come with the rows'
        moe.moe_permute_bwd(dxp, pr, w, xn, None, None, None, dxn, dw, ws)
    logits = (xn.double() @ p["Wg"].double().t() + p["bias"].double()).float()
    dl = f32(T, E)
    moe.moe_route_bwd(ids, w_all, dw, None if renorm else logits, renorm, dl, ws)
    g["dWg"], g["dbias"] = dl.t() @ xn.float(), dl.sum(0)
    router = dl @ p["Wg"]
    moe.moe_permute_bwd(dxp, pr, w if on_input else None, None, xnd.grad.float() + router, dz, p["gw"], dxn, None, ws)
    g["dr"] = bf(T, H)
    if ln:
        moe.moe_add_layernorm_bwd(dxn, stream, p["nw"], EPS, p["dstream"], g["dr"], None, g["dnw"], g["dnb"], ws)
    else:
        moe.moe_add_rmsnorm_bwd(dxn, stream, p["nw"], EPS, p["dstream"], g["dr"], None, g["dnw"], ws)
    assert moe.moe_get_device_status(ws) == 0
    return g, ids, out, (router, dxn)


def _reference(p, ids, ln, renorm, on_input, local):
    start, count = local
    v = {n: p[n].double().requires_grad_() for n in ("nw", "nb", "Wg", "bias", "gw")}
    r = (p["r"].double() + p["x"].double()).requires_grad_()
    xn = ref.norm(r, v["nw"], v["nb"] if ln else None, EPS, ln)[0]
    w = ref.weights(xn @ v["Wg"].t() + v["bias"], ids, renorm)
    if count >= 0:
        w = w * ((ids >= start) & (ids < start + count))
    out = torch.sigmoid(xn @ v["gw"]).unsqueeze(-1) * _mlp(xn, p["S1"].double(), p["S2"].double())
    for e in range(start, start + (E if count < 0 else count)):
        for j in range(K):
            hit = (ids[:, j] == e).nonzero().flatten()
            xe = xn[hit] * w[hit, j, None] if on_input else xn[hit]
            ye = _mlp(xe, p["W1"][e].double(), p["W2"][e].double())
            out = out.index_add(0, hit, ye if on_input else ye * w[hit, j, None])
    ((out * p["dout"].double()).sum() + (r * p["dstream"].double()).sum()).backward()
    return dict(dr=r.grad, dnw=v["nw"].grad, dnb=v["nb"].grad if ln else None, dWg=v["Wg"].grad, dbias=v["bias"].grad,
                dgw=v["gw"].grad), out.detach()


@pytest.mark.parametrize("ln", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("on_input", [False, True])
@pytest.mark.parametrize("local", [(0, -1), (2, 4)])
def test_a_training_step_of_one_block(ln, renorm, on_input, local):
    p = _params()
    got, ids, out, (router, dxn) = _step(p, ln, renorm, on_input, local)
    want, o = _reference(p, ids, ln, renorm, on_input, local)
    assert float((out.double() - o).norm() / o.norm()) <= TOL
    for n, g in got.items():
        if g is not None:
            assert float((g.double() - want[n]).norm() / want[n].norm()) <= TOL, n
    if local == (0, -1) and not renorm:
        assert float(router.norm() / dxn.float().norm()) >= 2.0 ** -3


@pytest.mark.parametrize("fmt", ["bf16", "w8a8", "w4"])
def test_block_with_a_layer_norm(fmt):
    p = _params(seed=20)
    W1, W2, S1, S2 = p["W1"], p["W2"], p["S1"], p["S2"]
    kw = dict(W1s=S1, W2s=S2, shared_gate_w=p["gw"], **{"w8a8": dict(fp8=True, act8=True), "w4": dict(w4=64)}.get(fmt, {}))
    block = MoELayer(p["Wg"], W1, W2, K, True, T, norm_w=p["nw"], norm_eps=EPS, layer_norm=True, norm_b=p["nb"], **kw)
    plain = MoELayer(p["Wg"], W1, W2, K, True, T, **kw)
    r = p["r"].clone()
    out = block.block(p["x"], r).clone()
    ro, xn = torch.empty_like(r), torch.empty_like(r)
    moe.moe_add_layernorm(p["x"], p["r"], p["nw"], p["nb"], EPS, ro, xn)
    want = plain.forward(xn)
    assert torch.equal(r, ro)
    if fmt == "w8a8":  # the experts' rows are rounded once instead of twice: E4M3 codes differ at some boundaries
        assert float((out.double() - want.double()).norm() / want.double().norm()) < 2.0 ** -4
    else:
        assert torch.equal(out, want)
    assert moe.moe_get_device_status(block.ws) == 0


def test_layer_norm_options_are_checked():
    p = _params(seed=30)
    for bad in (dict(layer_norm=True), dict(norm_b=p["nb"]), dict(norm_w=p["nw"], norm_b=p["nb"])):
        with pytest.raises(ValueError):
            MoELayer(p["Wg"], p["W1"], p["W2"], K, True, T, **bad)
