"""64-bit references of the norm and of the 4-bit products, in plain torch, for the tests of both."""
import torch


def e4m3_round(v: torch.Tensor) -> torch.Tensor:
    """float64 values rounded to the nearest E4M3 value, ties to even, saturating at 448."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), torch.clamp(e - 1, min=-6) - 3)
    return torch.clamp(torch.round(v / step) * step, -448.0, 448.0)


def rmsnorm(x, residual, w, eps):
    """(r, y) in float64 of the residual's addition (rounded to binary32, as the definition says) and its norm."""
    r = x.float() if residual is None else residual.float() + x.float()
    r = r.double()
    y = r / torch.sqrt((r * r).mean(dim=1, keepdim=True) + eps) * w.double()
    return r, y


def act_exponent(amax: torch.Tensor) -> torch.Tensor:
    """Smallest e >= -126 with amax <= 448 * 2^e."""
    m, e = torch.frexp(amax)
    return torch.clamp(e - 9 + (m > 0.875).to(e.dtype), min=-126)


def unpack_w4(q: torch.Tensor, scale: torch.Tensor):
    """(codes, scales) of packed 4-bit weights, both [..., K] float64."""
    K = 2 * q.shape[-1]
    codes = torch.empty(q.shape[:-1] + (K // 8, 8), dtype=torch.float64, device=q.device)
    b = q.reshape(q.shape[:-1] + (K // 8, 4)).to(torch.int32)
    for i in range(8):
        nib = i // 2 + 4 * (i % 2)
        codes[..., i] = ((b[..., nib // 2] >> (4 * (nib % 2))) & 15).double() - 8.0
    return codes.flatten(-2), scale.double().repeat_interleave(K // scale.shape[-1], dim=-1)


def pack_w4(codes: torch.Tensor) -> torch.Tensor:
    """Integer codes [..., K] in -8..7 packed to [..., K/2] uint8."""
    c = (codes.to(torch.int32) + 8).reshape(codes.shape[:-1] + (-1, 8))
    nib = torch.stack([c[..., 2 * (n % 4) + n // 4] for n in range(8)], dim=-1)
    return (nib[..., 0::2] | (nib[..., 1::2] << 4)).to(torch.uint8).flatten(-2)


def w4_experts(x, topk_w, pair_row, offsets, perm_src, W1, W2, shared=None, gate_w=None):
    """float64 output of the experts from float64 weights W1 [S, 2I, H], W2 [S, H, I] and the routing tables, h rounded
    to bf16, and the sum of the absolute values that h's rounding can move (a bound of its effect is 2^-8 of it)."""
    T, k = pair_row.shape
    xd = x.double()

    def mlp(xr, w1, w2):
        gu = xr @ w1.t()
        n = w1.shape[0] // 2
        h = gu[:, :n] * torch.sigmoid(gu[:, :n]) * gu[:, n:]
        h = h.float().to(torch.bfloat16).double()
        return h @ w2.t(), h.abs() @ w2.abs().t()

    rows = int(offsets[-1])
    y = torch.zeros(max(rows, 1), x.shape[1], dtype=torch.float64, device=x.device)
    ya = torch.zeros_like(y)
    off = offsets.tolist()
    for s in range(len(off) - 1):
        a, b = off[s], off[s + 1]
        if b > a:
            y[a:b], ya[a:b] = mlp(xd[(perm_src[a:b] // k).long()], W1[s], W2[s])
    keep = (pair_row >= 0).double()
    w = (torch.ones_like(keep) if topk_w is None else topk_w.double()) * keep
    pr = pair_row.clamp(min=0).long()
    out = (y[pr] * w.unsqueeze(-1)).sum(1)
    mag = (ya[pr] * w.abs().unsqueeze(-1)).sum(1)
    if shared is not None:
        sh, sha = mlp(xd, *shared)
        g = torch.ones(T, 1, dtype=torch.float64, device=x.device)
        if gate_w is not None:
            g = torch.sigmoid(xd @ gate_w.double()).unsqueeze(-1)
        out, mag = out + g * sh, mag + g * sha
    return out, mag
