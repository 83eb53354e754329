"""4-bit weights with group scales against the 64-bit formulas of tests/block_ops_ref.py.

Tolerances (derived before the first run):
  * quantiser: bitwise against the same binary32 formulas in torch;
  * matvec: one bf16 rounding (2^-8 relative) of a binary32 sum; the sum's error is at most 2^-19.7 of
    143 sum_k s |x_k| (each group's codes enter as 128 + c + 8 <= 143, summed in about ten steps of relative error
    2^-23 each, before 136 sum x is taken off): 2^-19 of it here;
  * experts: the same per product; h's bf16 rounding moves out by at most 2^-8 sum |w| |W2| |h| (half a spacing each,
    added up in the worst case), out's rounding by 2^-8; and over all outputs, whose roundings are independent, the
    2-norm error is below 2^-7.
"""
import pytest
import torch

import moe_inputs as mi
import serving_router_gate_gb300 as moe
from serving_router_gate_gb300.layer import MoELayer

from block_ops_ref import pack_w4, unpack_w4, w4_experts

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _weights(lead, K, group, seed):
    g = _gen(seed)
    codes = torch.randint(-8, 8, lead + (K,), generator=g, device="cuda", dtype=torch.int8)
    s = ((torch.rand(lead + (K // group,), generator=g, device="cuda") + 0.5) * 0.01).to(torch.bfloat16)
    s = torch.where(torch.rand(s.shape, generator=g, device="cuda") < 0.1, -s, s)
    return pack_w4(codes), s


def test_packing_helpers_agree():
    codes = torch.randint(-8, 8, (5, 64), generator=_gen(1), device="cuda", dtype=torch.int8)
    got, _ = unpack_w4(pack_w4(codes), torch.ones(5, 2, dtype=torch.bfloat16, device="cuda"))
    assert torch.equal(got, codes.double())


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows,K", [(1, 128), (7, 384), (300, 1408), (33, 2048)])
def test_quantise_w4_rows(group, rows, K):
    g = _gen(rows + K + group)
    w = (torch.randn(rows, K, generator=g, device="cuda") * 0.05).to(torch.bfloat16)
    w[0, :group] = 0.0
    w[-1, group // 2] = 100.0
    q = torch.empty(rows, K // 2, dtype=torch.uint8, device="cuda")
    s = torch.empty(rows, K // group, dtype=torch.bfloat16, device="cuda")
    moe.moe_quantize_w4_rows(w, q, s)
    wf = w.float().reshape(rows, -1, group)
    seven = torch.full((), 7.0, device="cuda")
    ref_s = (wf.abs().amax(-1) / seven).to(torch.bfloat16)
    d = torch.where(ref_s == 0, torch.ones_like(ref_s), ref_s).float().unsqueeze(-1)
    codes = torch.where(ref_s.unsqueeze(-1) == 0, torch.zeros_like(wf), torch.round(wf / d).clamp(-8, 7))
    assert torch.equal(s, ref_s)
    assert torch.equal(q, pack_w4(codes.reshape(rows, K)))
    got, gs = unpack_w4(q, s)
    err = (got * gs - w.double()).abs().reshape(rows, -1, group)
    assert (err <= 0.51 * s.double().abs().unsqueeze(-1)).all()


@pytest.mark.parametrize("group", [32, 128])
def test_quantise_every_quotient(group):
    # every pair of eight-bit significands, f / s from 1/8 to 8, ties among them; scales from subnormal to the largest
    m = torch.arange(128, 256, device="cuda", dtype=torch.float64)
    for e in (-133, -130, -126, -100, -64, -63, -1, 0, 60, 117):
        amax = m * 2.0 ** e                                          # a group's largest element, 128 of them
        f = (m.repeat_interleave(2) * torch.tensor([1.0, -1.0], device="cuda").repeat(128)).repeat(128, 1)
        f = f[:, None, :] * 2.0 ** (e - torch.arange(0, 6, device="cuda", dtype=torch.float64))[:, None]
        f = torch.where(f.abs() <= amax[:, None, None], f, f / 2).reshape(128, -1, group)
        f[:, :, 0] = amax[:, None]
        w = f.to(torch.bfloat16).reshape(128, -1)
        q = torch.empty(128, w.shape[1] // 2, dtype=torch.uint8, device="cuda")
        s = torch.empty(128, w.shape[1] // group, dtype=torch.bfloat16, device="cuda")
        moe.moe_quantize_w4_rows(w, q, s)
        wf = w.float().reshape(128, -1, group)
        ref_s = (wf.abs().amax(-1) / torch.full((), 7.0, device="cuda")).to(torch.bfloat16)
        assert torch.equal(s, ref_s)
        ratio = wf.double() / ref_s.double().unsqueeze(-1)           # (a tie is exact in 64 bits, the rest far from one)
        codes = torch.where(ref_s.unsqueeze(-1) == 0, torch.zeros_like(ratio), torch.round(ratio).clamp(-8, 7))
        assert torch.equal(q, pack_w4(codes.reshape(128, -1)))


def _check_matvec(x, q, s, y):
    c, sc = unpack_w4(q, s)
    ref = x.double() @ (c * sc).t()
    mag = 143.0 * (x.double().abs() @ sc.abs().t())
    err = (y.double() - ref).abs()
    bad = err > 2.0 ** -8 * ref.abs() + 2.0 ** -19 * mag
    assert not bad.any(), (int(bad.sum()), float((err / (2.0 ** -8 * ref.abs() + 2.0 ** -19 * mag)).max()))


def _matvec(M, N, K, group, seed=0, scale_x=1.0):
    x = (torch.randn(M, K, generator=_gen(seed + M), device="cuda") * scale_x).to(torch.bfloat16)
    q, s = _weights((N,), K, group, seed + N + K)
    y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    moe.moe_matvec_w4(x, q, s, y)
    torch.cuda.synchronize()
    return x, q, s, y


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 33])
def test_matvec_row_counts(M, group):
    _check_matvec(*_matvec(M, 96, 512, group))


@pytest.mark.parametrize("N", [1, 2, 15, 16, 17, 31, 32, 33, 1000, 4097])
def test_matvec_output_counts(N):
    _check_matvec(*_matvec(3, N, 384, 128))


@pytest.mark.parametrize("K,group", [(32, 32), (64, 32), (96, 32), (64, 64), (192, 64), (128, 128), (1376, 32),
                                     (1408, 128), (1216, 64), (7168, 128), (8192, 64), (16384, 128), (20480, 32)])
def test_matvec_depths(K, group):
    _check_matvec(*_matvec(5, 77, K, group))
    _check_matvec(*_matvec(1, 77, K, group, seed=3))


def test_matvec_many_outputs():
    _check_matvec(*_matvec(1, 40001, 256, 64))
    _check_matvec(*_matvec(11, 20011, 128, 128))


def test_matvec_values_with_a_common_sign_and_wide_range():
    x, q, s, y = _matvec(4, 128, 2048, 128, seed=5)
    x = x.abs()
    x[1] *= 1e20
    x[2] *= 1e-20
    x[3, 5] = 3e4                               # one value far above the rest
    moe.moe_matvec_w4(x, q, s, y)
    _check_matvec(x, q, s, y)
    zero = torch.zeros_like(x)
    moe.moe_matvec_w4(zero, q, s, y)
    assert not y.float().abs().any()


def test_matvec_nonfinite_values_stay_in_their_row():
    x, q, s, _ = _matvec(3, 64, 256, 64, seed=6)
    want = torch.empty(3, 64, dtype=torch.bfloat16, device="cuda")
    moe.moe_matvec_w4(x, q, s, want)
    x[1, 9] = float("nan")
    y = torch.empty_like(want)
    moe.moe_matvec_w4(x, q, s, y)
    assert torch.isnan(y[1].float()).all()
    assert torch.equal(y[0], want[0]) and torch.equal(y[2], want[2])


@pytest.mark.parametrize("N,K,group", [(64, 2048, 128), (4096, 512, 64), (513, 1408, 32)])
def test_matvec_rows_do_not_depend_on_the_batch(N, K, group):
    x, q, s, y = _matvec(16, N, K, group, seed=7)
    for m in (0, 7, 8, 15):
        one = torch.empty(1, N, dtype=torch.bfloat16, device="cuda")
        moe.moe_matvec_w4(x[m:m + 1], q, s, one)
        assert torch.equal(one[0], y[m])


def test_matvec_writes_only_its_outputs():
    x, q, s, _ = _matvec(3, 50, 128, 32, seed=8)
    buf = torch.full((5, 50), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_matvec_w4(x, q, s, buf[1:4])
    assert (buf[0] == 7.0).all() and (buf[4] == 7.0).all()
    _check_matvec(x, q, s, buf[1:4])


def _at_the_end(t):
    """A copy of t whose last byte is the last of its allocation (whole pages of 2 MiB, a segment of its own)."""
    n = t.numel() * t.element_size()
    buf = torch.empty(-(-n // (2 << 20)) * (2 << 20) + (32 << 20), dtype=torch.uint8, device="cuda")
    out = buf[buf.numel() - n:].view(t.dtype).view(t.shape)
    out.copy_(t)
    return out


@pytest.mark.parametrize("M,N,K,group", [(1, 64, 512, 128), (8, 64, 1024, 128), (16, 96, 512, 128), (5, 32, 256, 64),
                                         (9, 32, 96, 32)])
def test_matvec_operands_that_end_with_their_allocations(M, N, K, group):
    # no read goes past the last row's end, whatever the fetches ahead ask for
    x, q, s, want = _matvec(M, N, K, group, seed=9)
    y = _at_the_end(torch.zeros_like(want))
    moe.moe_matvec_w4(_at_the_end(x), _at_the_end(q), _at_the_end(s), y)
    assert torch.equal(y, want)


@pytest.mark.parametrize("M", [3, 13])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_matvec_rows_on_16_bytes(M, group):
    # rows that start on 16 but not on 32 bytes take two loads where the others take one: the same results
    x, q, s, want = _matvec(M, 96, 384, group, seed=17)
    buf = torch.empty(M * 384 + 8, dtype=torch.bfloat16, device="cuda")
    odd = buf[8:].view(M, 384)
    odd.copy_(x)
    assert odd.data_ptr() % 32 == 16
    y = torch.empty_like(want)
    moe.moe_matvec_w4(odd, q, s, y)
    assert torch.equal(y, want)


def test_matvec_empty_batch():
    q, s = _weights((8,), 64, 64, 1)
    n = moe.moe_get_launch_count()
    moe.moe_matvec_w4(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), q, s,
                      torch.empty(0, 8, dtype=torch.bfloat16, device="cuda"))
    assert moe.moe_get_launch_count() == n


def test_matvec_codes_past_4_gib():
    # 530001 rows of 8 KiB: the last ones lie past 2^32 bytes and 2^33 codes
    N, K = 530001, 16384
    q, s = torch.empty(N, K // 2, dtype=torch.uint8, device="cuda"), torch.empty(N, K // 128, device="cuda")
    q.random_(0, 256, generator=_gen(11))
    s = s.uniform_(-0.01, 0.01, generator=_gen(12)).to(torch.bfloat16)
    x = torch.randn(2, K, generator=_gen(13), device="cuda").to(torch.bfloat16)
    y = torch.full((2, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    moe.moe_matvec_w4(x, q, s, y)
    rows = torch.tensor([0, 1, 31, 32, 262143, 262144, 262145, 524287, 524288, 524289, N - 33, N - 2, N - 1], device="cuda")
    _check_matvec(x, q[rows], s[rows], y[:, rows])
    assert torch.isfinite(y.float()).all()


def test_matvec_on_another_stream_and_in_a_graph():
    x, q, s, want = _matvec(3, 200, 512, 64, seed=14)
    y, stream = torch.empty_like(want), torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    moe.moe_matvec_w4(x, q, s, y, stream=stream)
    stream.synchronize()
    assert torch.equal(y, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_matvec_w4(x, q, s, y)
        moe.moe_matvec_w4(x, q, s, y)
    y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_matvec_of_weights_written_just_before():
    # the product's kernel may start while the quantiser finishes; it reads nothing of the weights before that
    g = _gen(15)
    x = torch.randn(4, 4096, generator=g, device="cuda").to(torch.bfloat16)
    q, s = torch.zeros(4096, 2048, dtype=torch.uint8, device="cuda"), torch.zeros(4096, 32, device="cuda").to(torch.bfloat16)
    y = torch.empty(4, 4096, dtype=torch.bfloat16, device="cuda")
    for i in range(5):
        w = torch.randn(4096, 4096, generator=g, device="cuda").to(torch.bfloat16)
        torch.cuda.synchronize()
        moe.moe_quantize_w4_rows(w, q, s)
        moe.moe_matvec_w4(x, q, s, y)
        _check_matvec(x, q, s, y)


def test_binding_refuses_what_it_would_misread():
    x, q, s, y = _matvec(4, 64, 256, 64, seed=16)
    for bad in (dict(x=x.t().contiguous().t()), dict(x=x.float()), dict(q=q[:, ::2]), dict(q=q.view(torch.int8)),
                dict(s=s[:-1]), dict(s=s.float()), dict(y=y.t().contiguous().t()), dict(y=y[:3]), dict(y=y.float())):
        a = {**dict(x=x, q=q, s=s, y=y), **bad}
        with pytest.raises(ValueError):
            moe.moe_matvec_w4(a["x"], a["q"], a["s"], a["y"])
    with pytest.raises(ValueError):
        moe.moe_quantize_w4_rows(torch.empty(8, 128, device="cuda"), q, s)
    with pytest.raises(moe.MoEError):
        moe.moe_matvec_w4(x.reshape(-1)[1:1 + 2 * 256].view(2, 256), q, s, y[:2])  # not 16-byte aligned
    with pytest.raises(moe.MoEError):
        moe.moe_quantize_w4_rows(torch.empty(8, 0, dtype=torch.bfloat16, device="cuda"),
                                 torch.empty(8, 0, dtype=torch.uint8, device="cuda"),
                                 torch.empty(8, 0, dtype=torch.bfloat16, device="cuda"))


# ---------------------------------------------------------------------------------------------- experts

def _tables(T, E, k, S, seed, hot=None):
    """Routing tables as moe_permute writes them, for slots 0 .. S-1 of E experts (other pairs dropped)."""
    g = _gen(seed)
    score = torch.randn(T, E, generator=g, device="cuda")
    if hot is not None:
        score[:, hot] += 100.0
    v, ids = score.topk(k, dim=1)
    w = torch.softmax(v, dim=1).contiguous()
    key = torch.where(ids < S, ids, torch.full_like(ids, S)).reshape(-1)
    order = torch.argsort(key, stable=True)
    counts = torch.bincount(key, minlength=S + 1)[:S]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    row = torch.empty_like(order)
    row[order] = torch.arange(T * k, device="cuda")
    pair_row = torch.where(key < S, row, torch.full_like(row, -1)).reshape(T, k).to(torch.int32).contiguous()
    return w, offsets, order.to(torch.int32), pair_row


def _experts(T, H, I, E, k, group, I_sh=0, gated=False, S=None, seed=0, hot=None, unit=False, poison=True):
    S = E if S is None else S
    x = torch.randn(T, H, generator=_gen(seed + 11), device="cuda").to(torch.bfloat16)
    w, offsets, perm_src, pair_row = _tables(T, E, k, S, seed + 12, hot)
    w1, w2 = _weights((S, 2 * I), H, group, seed + 13), _weights((S, H), I, group, seed + 14)
    sh1 = _weights((2 * I_sh,), H, group, seed + 15) if I_sh else (None, None)
    sh2 = _weights((H,), I_sh, group, seed + 16) if I_sh else (None, None)
    gate = (torch.randn(H, generator=_gen(seed + 17), device="cuda") * 0.02).to(torch.bfloat16) if gated else None
    ws = torch.empty(moe.moe_workspace_size_w4(T, H, I, k, I_sh), dtype=torch.uint8, device="cuda")
    ws.fill_(0xFF if poison else 0)
    moe.moe_workspace_init(ws)
    rows = int(offsets[-1])
    perm_src[rows:] = -5                        # entries past the rows are unspecified
    out = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    tw = None if unit else w
    args = (x, offsets, perm_src, *w1, *w2, pair_row, tw, *sh1, *sh2, gate, out, ws)
    moe.moe_forward_w4(*args)
    torch.cuda.synchronize()
    assert moe.moe_get_device_status(ws) == 0

    def deq(p):
        c, s = unpack_w4(*p)
        return c * s
    ref, mag = w4_experts(x, tw, pair_row, offsets, perm_src, deq(w1), deq(w2),
                          (deq(sh1), deq(sh2)) if I_sh else None, gate)
    err = (out.double() - ref).abs()
    assert (err <= 2.0 ** -8 * ref.abs() + 2.0 ** -8 * mag + 1e-30).all()
    assert (out.double() - ref).norm() <= 2.0 ** -7 * ref.norm()
    return args


@pytest.mark.parametrize("T", [1, 2, 5, 16, 40])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_experts_batches(T, group):
    _experts(T, 256, 128, 16, 4, group, I_sh=256, gated=True)


@pytest.mark.parametrize("H,I", [(64, 64), (128, 64), (192, 320), (2048, 1408), (7168, 256), (256, 2048)])
def test_experts_sizes(H, I):
    _experts(6, H, I, 8, 2, 64 if H % 128 or I % 128 else 128)


@pytest.mark.parametrize("I_sh", [128, 1024])
@pytest.mark.parametrize("gated", [False, True])
def test_experts_shared(I_sh, gated):
    _experts(3, 512, 128, 8, 3, 128, I_sh=I_sh, gated=gated, seed=3)


def test_experts_one_hot_slot():
    # every token's first pair goes to one slot: many rows in one slot, few in the others
    _experts(77, 256, 128, 32, 3, 64, seed=4, hot=9)


def test_experts_local_range_and_unit_weights():
    _experts(9, 256, 128, 32, 4, 32, S=10, seed=5)
    _experts(9, 256, 128, 32, 4, 32, S=10, seed=6, unit=True)


def test_experts_no_local_pair():
    # no pair lands on this rank: the shared expert alone, or zeros
    T, H, I, k = 4, 256, 128, 2
    args = list(_experts(T, H, I, 8, k, 64, I_sh=128, seed=7))
    args[1] = torch.zeros_like(args[1])
    args[7] = torch.full_like(args[7], -1)
    moe.moe_forward_w4(*args)
    ref, mag = w4_experts(args[0], args[8], args[7], args[1], args[2], None, None,
                          tuple(c * s for c, s in (unpack_w4(args[9], args[10]), unpack_w4(args[11], args[12]))))
    assert ((args[14].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -8 * mag).all()
    args[9:13] = [None] * 4
    moe.moe_forward_w4(*args)
    assert not args[14].float().abs().any()


def test_experts_many_slots():
    _experts(20, 128, 64, 500, 8, 64, seed=8)


def test_experts_one_token_of_a_batch_alone():
    args = _experts(12, 512, 256, 16, 3, 128, I_sh=256, gated=True, seed=9)
    x, offsets, perm_src, q1, s1, q2, s2, pair_row, w, a, b, c, d, gate, out, ws = args
    t = 5
    ids = torch.searchsorted(offsets, pair_row[t], right=True) - 1       # the token's slots
    counts = torch.bincount(ids, minlength=16)
    off1 = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    order = torch.argsort(ids, stable=True)
    row = torch.empty_like(order)
    row[order] = torch.arange(3, device="cuda")
    one = torch.empty(1, 512, dtype=torch.bfloat16, device="cuda")
    moe.moe_forward_w4(x[t:t + 1], off1, order.to(torch.int32), q1, s1, q2, s2, row.reshape(1, 3).to(torch.int32),
                       w[t:t + 1], a, b, c, d, gate, one, ws)
    # the two may add their partial sums in another order: h and out may each round to a neighbour
    assert (one[0].double() - out[t].double()).norm() <= 2.0 ** -7 * out[t].double().norm()


def test_experts_bad_indices_are_dropped_and_flagged():
    args = list(_experts(4, 256, 128, 8, 2, 64, seed=10))
    good = args[14].clone()
    pr = args[7].clone()
    pr[0, 0] = 10 ** 6
    args[7] = pr
    moe.moe_forward_w4(*args)
    assert moe.moe_get_device_status(args[15]) == moe.MOE_ERR_DEVICE_BOUNDS
    assert torch.equal(args[14][1:], good[1:])


def test_layer_with_4bit_experts_and_its_graph():
    cfg = mi.MoEConfig("w4", T=11, H=512, I=256, E=16, k=3, renorm=True, n_shared=1, I_shared=256, shared_gate=True)
    inp = mi.make_inputs(cfg)
    d = {n: (v.cuda() if isinstance(v, torch.Tensor) else v) for n, v in inp.items()}
    W1s, W2s = mi.shared_concat(d["W1s"], d["W2s"])
    w = (1.0 + 0.1 * torch.randn(512, generator=_gen(1), device="cuda")).to(torch.bfloat16)
    layer = MoELayer(d["Wg"], d["W1"], d["W2"], cfg.k, cfg.renorm, 16, W1s=W1s, W2s=W2s, shared_gate_w=d["w_s"],
                     w4=64, norm_w=w)
    res = torch.randn(11, 512, generator=_gen(2), device="cuda")
    out = layer.block(d["x"], res)
    torch.cuda.synchronize()
    v = layer.views(11)

    def deq(p):
        c, s = unpack_w4(*p)
        return c * s
    ref, mag = w4_experts(layer.x_norm[:11], v["topk_w"], v["pair_row"], v["offsets"], v["perm_src"], deq(layer.W1w4),
                          deq(layer.W2w4), (deq(layer.W1sw4), deq(layer.W2sw4)), layer.gate)
    assert ((out.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -8 * mag).all()
    # the quantised layer stays near the bf16 one
    full = MoELayer(d["Wg"], d["W1"], d["W2"], cfg.k, cfg.renorm, 16, W1s=W1s, W2s=W2s, shared_gate_w=d["w_s"])
    a, b = layer.forward(d["x"]).double(), full.forward(d["x"]).double()
    assert (a - b).norm() < 0.25 * b.norm()
    g = layer.capture(d["x"])
    want = layer.forward(d["x"]).clone()
    layer.out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(layer.out[:11], want)
    with pytest.raises(ValueError):
        MoELayer(d["Wg"], d["W1"], d["W2"], cfg.k, cfg.renorm, 16, w4=64, fp8=True)
    with pytest.raises(ValueError):
        MoELayer(d["Wg"], d["W1"], d["W2"], cfg.k, cfg.renorm, 16, w4=64, on_input=True)


def test_layer_with_4bit_experts_on_another_stream():
    cfg = mi.MoEConfig("w4", T=5, H=256, I=128, E=8, k=2, renorm=True, n_shared=1, I_shared=128, shared_gate=True)
    inp = mi.make_inputs(cfg)
    d = {n: (v.cuda() if isinstance(v, torch.Tensor) else v) for n, v in inp.items()}
    W1s, W2s = mi.shared_concat(d["W1s"], d["W2s"])
    layer = MoELayer(d["Wg"], d["W1"], d["W2"], cfg.k, cfg.renorm, 8, W1s=W1s, W2s=W2s, shared_gate_w=d["w_s"], w4=32)
    want = layer.forward(d["x"]).clone()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    for _ in range(20):  # calls in a row share the workspace
        layer.forward(d["x"], stream=stream)
    stream.synchronize()
    assert torch.equal(layer.out[:5], want)
