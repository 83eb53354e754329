"""The layer norm and the token path's gradients at the kernels and options that other tests do not reach: every variant of
the permutation's gradient, layer norms of every width's kernel with either stream, kept pairs of weight 0
(MOE_NONLOCAL_MOD), a layer norm in front of expert-parallel ranks; and what lies before and behind each output.

Tolerances: those of the files the helpers are from."""
import pytest
import torch

import serving_router_gate_gb300 as moe
from serving_router_gate_gb300.expert_parallel import EPMoELayer
from serving_router_gate_gb300.layer import MoELayer

import bwd_ref as ref
from test_gpu_norm_bwd import _bwd, _check, _check_ln, _inputs, _ln, _run
from test_gpu_token_bwd import _fin, _fin_check, _fin_inputs, _perm, _perm_check, _perm_inputs, _route, _route_inputs, _status
from test_gpu_token_bwd import _ws as _token_ws

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H,E,k,S", [(6500, 320, 16, 8, None), (8191, 2048, 32, 7, 20), (6100, 7168, 16, 5, 9),
                                       (2000, 192, 16, 2, None), (700, 320, 8, 1, None), (3000, 4096, 8, 2, 3),
                                       (620, 1024, 16, 3, None), (2600, 2112, 60, 4, 31), (1300, 512, 64, 32, 40)])
@pytest.mark.parametrize("on_input", [False, True])
@pytest.mark.parametrize("add,gated", [(None, True), (torch.float32, False)])
def test_permute_bwd_variants(T, H, E, k, S, on_input, add, gated):
    d = _perm_inputs(T, H, E, k, S, on_input, add, gated, seed=21, pad=1)
    ws = _token_ws()
    _perm_check(d, _perm(d, ws))
    assert _status(ws) == 0


@pytest.mark.parametrize("T,H,E,k,S", [(3000, 128, 16, 8, 9), (2100, 320, 8, 3, None), (1700, 4160, 16, 5, 7),
                                       (900, 8192, 8, 2, None), (700, 8256, 8, 2, 5)])
def test_finalize_bwd_variants(T, H, E, k, S):
    d = _fin_inputs(T, H, E, k, S, True, seed=22, pad=1)
    ws = _token_ws(H)
    _fin_check(d, _fin(d, ws))
    assert _status(ws) == 0


@pytest.mark.parametrize("H", [1000, 2560, 4104, 5120, 5640, 6144, 7176, 8192, 12288])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("bias", [False, True])
def test_layernorm_kernels(H, f32, bias):
    r, w, b, _ = _inputs(19, H, f32, seed=23)
    x = ref.rnd(19, H, seed=24)
    b = b if bias else None
    _check_ln(x, r, w, b, _ln(x, r, w, b, True))


@pytest.mark.parametrize("H", [264, 2048, 7168])
@pytest.mark.parametrize("ln", [False, True])
def test_a_bf16_streams_gradient_is_taken_at_the_rounded_stream(H, ln):
    """Far from zero a bf16 step is a good part of the deviations: the statistics are those of the r that the call is given."""
    _, w, _, dy = _inputs(9, H, False, seed=25)
    r = (3e4 + 300.0 * ref.rnd(9, H, seed=26, dtype=torch.float32)).to(torch.bfloat16)
    _check(ln, dy, r, w, None, _run(ln, dy, r, w, None))


# ------------------------------------------------------------------------------------------- pairs of weight 0

@pytest.mark.parametrize("renorm", [False, True])
def test_kept_pairs_of_weight_zero(renorm):
    """MOE_NONLOCAL_MOD gives another rank's pairs a row and the weight 0: their rows get no gradient and add none, their
    weights have one, which the mask takes out of the router's."""
    T, H, E, k, lo, n = 90, 320, 12, 4, 3, 5
    logits, ids, w, _ = _route_inputs(T, E, k, renorm, seed=31)
    ws = torch.empty(moe.moe_workspace_size(T, H, 64, E, E, k), dtype=torch.uint8, device="cuda")
    moe.moe_workspace_init(ws)
    i32 = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    slot, cnt, off, src, pr = i32(T, k), i32(n), i32(n + 1), i32(T * k), i32(T, k)
    wm, x = w.clone(), ref.rnd(T, H, seed=32)
    xp = torch.zeros(T * k, H, dtype=torch.bfloat16, device="cuda")
    moe.moe_permute(ids, wm, E, None, None, E, lo, n, moe.MOE_NONLOCAL_MOD, x, slot, cnt, off, src, pr, xp, ws)
    mask = (ids >= lo) & (ids < lo + n)
    assert (pr >= 0).all() and torch.equal(wm, w * mask) and not mask.all() and mask.any()
    d = dict(dout=ref.rnd(T, H, seed=33, std=0.1), y=ref.rnd(T * k, H, seed=34), pr=pr, w=wm, ysh=None, x=None, gw=None)
    o = _fin(d, ws)
    _fin_check(d, o)
    assert not o["dy"][pr[~mask].long()].any() and (o["dw"][~mask] != 0).any()
    p = dict(dxp=ref.rnd(T * k, H, seed=35, std=0.1), pr=pr, w=wm, x=x, add=None, dz=None, gw=None)
    dx, dw = _perm(p, ws)
    _perm_check(p, (dx, dw))
    assert (dw[~mask] != 0).any()
    # to the logits: the derivative of the masked weights
    lg = logits.double().requires_grad_()
    (ref.weights(lg, ids, renorm) * mask).backward(o["dw"].double())
    got = _route(logits, ids, w, (o["dw"] * mask).contiguous(), renorm, ws)
    c = (w * o["dw"]).double().abs().sum(1, keepdim=True)
    ref.inside(got, lg.grad, 2.0 ** -17 * c + 1e-37, "dlogits")   # each term of it at most c, twice the file's 2^-18
    assert _status(ws) == 0


# ------------------------------------------------------------------------------------------- expert-parallel ranks

@pytest.mark.parametrize("bias", [False, True])
def test_layer_norm_in_front_of_expert_parallel_ranks(bias):
    """The ranks one after the other.  bf16 partials and the one-GPU output are rounded once each: 2^-8 of their 2-norms,
    and as much again for sums of another order."""
    T, H, I, E, k = 33, 256, 128, 8, 3
    p = dict(Wg=ref.rnd(E, H, seed=41, std=0.15, dtype=torch.float32), W1=ref.rnd(E, 2 * I, H, seed=42, std=H ** -0.5),
             W2=ref.rnd(E, H, I, seed=43, std=I ** -0.5))
    opt = dict(norm_w=(1.0 + 0.2 * ref.rnd(H, seed=44, dtype=torch.float32)).to(torch.bfloat16), norm_eps=1e-5,
               layer_norm=True, norm_b=ref.rnd(H, seed=45, std=0.2) if bias else None)
    x, residual = ref.rnd(T, H, seed=46), ref.rnd(T, H, seed=47, std=3.0, dtype=torch.float32) + 2.0
    r0 = residual.clone()
    full = MoELayer(p["Wg"], p["W1"], p["W2"], k, True, T, **opt).block(x, r0).double()
    y = torch.empty_like(x)
    moe.moe_add_layernorm(x, residual, opt["norm_w"], opt["norm_b"], 1e-5, None, y)
    assert torch.equal(MoELayer(p["Wg"], p["W1"], p["W2"], k, True, T).forward(y).double(), full)
    acc, size = torch.zeros_like(full), full.norm()
    for r in range(2):
        rank = EPMoELayer(p["Wg"], p["W1"], p["W2"], k, True, T, 2, r, **opt)
        mine = residual.clone()
        part = rank.block(x, mine).double()
        assert torch.equal(mine, r0) and moe.moe_get_device_status(rank.layer.ws) == 0
        acc, size = acc + part, size + part.norm()
    assert (acc - full).norm() <= 2.0 ** -7 * size


# ------------------------------------------------------------------------------------------- around the outputs

GUARD = 64      # bytes before and behind an output


class Guarded:
    """Tensors that lie between guard bytes; the next one starts 16 bytes further on a 32-byte line than the last."""

    def __init__(self):
        self.bufs = []

    def __call__(self, *shape, dtype=torch.bfloat16):
        n = torch.Size(shape).numel() * torch.empty((), dtype=dtype).element_size()
        at = GUARD + 16 * (len(self.bufs) % 2)
        buf = torch.full((at + n + GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
        assert buf.data_ptr() % 32 == 0
        self.bufs.append((buf, at, n))
        return buf[at:at + n].view(dtype).view(shape)

    def check(self):
        torch.cuda.synchronize()
        for buf, at, n in self.bufs:
            assert (buf[:at] == 0xA5).all() and (buf[at + n:] == 0xA5).all()


@pytest.mark.parametrize("T", [1, 3, 5, 161])
@pytest.mark.parametrize("H", [8, 72, 520, 1032, 2568, 4104, 5640, 7176, 8200, 12296, 16384])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("ln", [False, True])
def test_norms_write_nothing_but_their_outputs(T, H, f32, ln):
    r, w, b, dy = _inputs(T, H, f32, seed=51)
    x, ds = ref.rnd(T, H, seed=52), ref.rnd(T, H, seed=53, std=0.01, dtype=r.dtype)
    G = Guarded()
    if ln:
        moe.moe_add_layernorm(x, r, w, b, 1e-5, G(T, H, dtype=r.dtype), G(T, H), G(T, H, dtype=torch.uint8),
                              G(T, dtype=torch.float32))
    ws = G(moe.moe_workspace_size_bwd(H), dtype=torch.uint8)
    moe.moe_workspace_init(ws)
    for stream in (None, ds):
        _bwd(ln, dy, r, w, stream, G(T, H, dtype=r.dtype), G(T, H), G(H, dtype=torch.float32),
             G(H, dtype=torch.float32) if ln else None, ws)
    G.check()
    assert _status(ws) == 0


@pytest.mark.parametrize("T,H,E,k", [(1, 64, 4, 1), (3, 192, 8, 2), (7, 320, 8, 5), (161, 576, 12, 8), (33, 2112, 12, 9),
                                     (5, 8256, 8, 3), (700, 512, 8, 2)])
def test_token_gradients_write_nothing_but_their_outputs(T, H, E, k):
    d = _fin_inputs(T, H, E, k, E - 1, True, seed=54)
    p = _perm_inputs(T, H, E, k, E - 1, True, torch.float32, True, seed=55)
    G = Guarded()
    f32 = dict(dtype=torch.float32)
    ws = G(moe.moe_workspace_size_bwd(H), dtype=torch.uint8)
    moe.moe_workspace_init(ws)
    moe.moe_finalize_bwd(d["dout"], d["y"], d["pr"], d["w"], d["ysh"], d["x"], d["gw"], G(T * k, H), G(T, k, **f32), G(T, H),
                         G(T, **f32), G(H, **f32), ws)
    small = G(moe.MOE_WS_HEADER_BYTES, dtype=torch.uint8)
    moe.moe_workspace_init(small)
    moe.moe_permute_bwd(p["dxp"], p["pr"], p["w"], p["x"], p["add"], p["dz"], p["gw"], G(T, H), G(T, k, **f32), small)
    for renorm in (False, True):
        for n in (E, E + 1, 4 * E + 3):
            logits, ids, w, dw = _route_inputs(T, n, min(k, n), renorm, seed=56)
            moe.moe_route_bwd(ids, w, dw, None if renorm else logits, renorm, G(T, n, **f32), small)
    G.check()
    assert _status(ws) == 0 and _status(small) == 0
