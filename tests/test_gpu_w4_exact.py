"""The 4-bit products where single elements count: one activation at a time, bounds that follow the kernel's own sums,
and the experts token by token.

Derived before the first run:
  * one activation x at k and zeros elsewhere: the codes enter as c / 64, exactly, and x c / 64 times the scale has at most
    8 + 4 + 8 significant bits, so y = bf16(scale c x), bit for bit;
  * a product in general, with mag = 8 sum_k s |x_k| (|c| <= 8): a group's sum takes group / 16 matrix instructions, each
    within 2^-22 of the magnitudes that it adds; the groups are added by K / group fused multiply-adds and at most eight
    parts, each within 2^-24 of what they have so far; then one bf16 rounding, 2^-8;
  * experts, per token against the formulas without any rounding of h: h's and out's bf16 roundings are at most 2^-8 of each
    value and independent, so their 2-norms add in squares: sqrt(2) 2^-8.
"""
import pytest
import torch

import serving_router_gate_gb300 as moe

import test_gpu_w4 as t4
from block_ops_ref import unpack_w4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K,group,N,M", [(32, 32, 5, 1), (96, 32, 33, 1), (1376, 32, 37, 16), (64, 64, 33, 8),
                                         (1216, 64, 37, 1), (1216, 64, 70, 16), (128, 128, 17, 1), (1408, 128, 37, 1),
                                         (1408, 128, 200, 8), (7168, 128, 37, 16), (2048, 32, 37, 1216)])
def test_one_activation_at_a_time(K, group, N, M):
    q, s = t4._weights((N,), K, group, 100 + K + N)
    c, sc = unpack_w4(q, s)
    v = (torch.rand(K, generator=t4._gen(K), device="cuda") + 0.5).to(torch.bfloat16)
    v[1::2] *= -3.0
    want = (c * sc * v.double()).to(torch.bfloat16).t().contiguous()   # [K, N]: what each element gives
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    got = torch.empty(K, N, dtype=torch.bfloat16, device="cuda")
    for k0 in range(0, K, M):
        m = min(M, K - k0)
        i = torch.arange(m, device="cuda")
        x.zero_()
        x[i, k0 + i] = v[k0:k0 + m]
        moe.moe_matvec_w4(x[:m], q, s, got[k0:k0 + m])
    assert torch.equal(got, want)


def _check(x, q, s, y):
    c, sc = unpack_w4(q, s)
    K = x.shape[1]
    group = K // s.shape[1]
    ref = x.double() @ (c * sc).t()
    mag = 8.0 * (x.double().abs() @ sc.abs().t())
    tol = 2.0 ** -8 * ref.abs() + ((group // 16) * 2.0 ** -22 + (K // group + 8) * 2.0 ** -24) * mag
    err = (y.double() - ref).abs()
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("M", [1, 8, 13, 16, 24, 33, 200])
@pytest.mark.parametrize("K,group", [(512, 32), (512, 128), (1408, 128), (1216, 64), (7168, 128), (16384, 128),
                                     (20480, 32)])
def test_products_within_their_own_bound(K, group, M):
    _check(*t4._matvec(M, 77, K, group, seed=30))


def _per_token(args):
    """args of moe_forward_w4 after a run: every token against the 64-bit formulas, h unrounded."""
    x, offsets, perm_src, q1, s1, q2, s2, pair_row, w, a, b, c, d, gate, out, ws = args
    T, k = pair_row.shape

    def deq(q, s):
        codes, sc = unpack_w4(q, s)
        return codes * sc

    def mlp(xr, w1, w2):
        gu = xr @ w1.t()
        n = w1.shape[0] // 2
        return (gu[:, :n] * torch.sigmoid(gu[:, :n]) * gu[:, n:]) @ w2.t()
    xd, off = x.double(), offsets.tolist()
    y = torch.zeros(max(off[-1], 1), x.shape[1], dtype=torch.float64, device="cuda")
    for s in range(len(off) - 1):
        r0, r1 = off[s], off[s + 1]
        if r1 > r0:
            y[r0:r1] = mlp(xd[(perm_src[r0:r1] // k).long()], deq(q1[s], s1[s]), deq(q2[s], s2[s]))
    wk = (torch.ones(T, k, device="cuda") if w is None else w).double() * (pair_row >= 0)
    ref = (y[pair_row.clamp(min=0).long()] * wk.unsqueeze(-1)).sum(1)
    if a is not None:
        sh = mlp(xd, deq(a, b), deq(c, d))
        ref = ref + (sh if gate is None else torch.sigmoid(xd @ gate.double()).unsqueeze(-1) * sh)
    err, size = (out.double() - ref).norm(dim=1), ref.norm(dim=1)
    assert (err <= 2.0 ** 0.5 * 2.0 ** -8 * size).all(), float((err / size.clamp(min=1e-300)).max())


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T", [1, 7, 33])
def test_experts_token_by_token(T, group):
    _per_token(t4._experts(T, 512, 384, 16, 4, group, I_sh=768, gated=True, seed=31))


def test_experts_listed_layer_token_by_token():
    _per_token(t4._experts(32, 2048, 1408, 64, 6, 128, I_sh=5632, seed=32))


@pytest.mark.parametrize("T,E,k", [(300, 8, 4), (1000, 64, 6), (500, 3, 2)])
def test_experts_large_batches(T, E, k):
    _per_token(t4._experts(T, 256, 128, E, k, 64, I_sh=128, gated=True, seed=33))


def test_experts_large_batch_with_one_hot_slot():
    _per_token(t4._experts(700, 256, 192, 32, 2, 64, seed=34, hot=31))


@pytest.mark.parametrize("E,k", [(32, 32), (40, 17), (1024, 32)])
def test_experts_many_per_token(E, k):
    _per_token(t4._experts(5, 256, 128, E, k, 64, I_sh=64, seed=35))


@pytest.mark.parametrize("S", [1023, 1024])
def test_experts_full_slot_table(S):
    # rows in the first and in the last slots of the table
    args = t4._experts(60, 128, 64, S, 8, 64, seed=36, hot=S - 1)
    assert int(args[1][-1]) - int(args[1][-2]) == 60
    _per_token(args)


@pytest.mark.parametrize("S", [1, 2, 8])
def test_experts_rank_with_few_slots(S):
    # an expert-parallel rank: most pairs are other ranks'
    args = t4._experts(64, 256, 128, 64, 8, 64, S=S, I_sh=64, seed=37)
    assert (args[7] < 0).any()
    _per_token(args)
