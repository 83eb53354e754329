"""64-bit references of the layer norm and of the token path's gradients, in plain torch, each with the sum of absolute
values that its binary32 evaluation rounds against."""
import torch

U = 2.0 ** -24          # a binary32 rounding, relative
BF = 2.0 ** -8          # a bf16 rounding, relative
SUM = 2.0 ** -18        # a row's sum: no chain of more than 64 additions, relative to the sum of absolute values


def norm(r, w, b, eps, ln):
    """y of the rows r (float64) and the magnitude its error is relative to: the mean's own error, relative to the
    values' absolute mean, reaches every deviation from it and the root of their squares."""
    d = r - r.mean(1, keepdim=True) if ln else r
    rstd = 1.0 / torch.sqrt((d * d).mean(1, keepdim=True) + eps)
    y = d * rstd * w
    K = 1.0 + (rstd * r.abs().mean(1, keepdim=True) if ln else 0.0)
    mag = K * ((d * rstd).abs() + (1.0 if ln else 0.0)) * w.abs()
    return (y if b is None else y + b), mag + (0.0 if b is None else b.abs())


def norm_bwd(dy, r, w, eps, dstream, ln):
    """(dr, its magnitude, dweight, its magnitude, dbias, its magnitude), all float64.

    Of dr = dstream + rstd (g - mean(g) - d rstd^2 mean(g d)): every term is off by at most a sum's error (SUM), 3 / 2
    of one for rstd's powers and a few roundings, so 2^-16 of the terms' absolute values; with a mean, by K times that.
    """
    dy, r, w = dy.double(), r.double(), w.double()
    d = r - r.mean(1, keepdim=True) if ln else r
    rstd = 1.0 / torch.sqrt((d * d).mean(1, keepdim=True) + eps)
    K = 1.0 + (rstd * r.abs().mean(1, keepdim=True) if ln else 0.0)
    g = dy * w
    mgd = rstd * rstd * (g * d).mean(1, keepdim=True)
    dr = rstd * (g - (g.mean(1, keepdim=True) if ln else 0.0) - d * mgd)
    amag = (g * d).abs().mean(1, keepdim=True)
    if ln:  # an error of the mean moves g d by g's absolute mean, and d itself
        amag = amag + g.abs().mean(1, keepdim=True) / rstd
    mag = rstd * K * (g.abs() + (g.abs().mean(1, keepdim=True) if ln else 0.0)
                      + (d.abs() + (1.0 / rstd if ln else 0.0)) * rstd * rstd * amag)
    if dstream is not None:
        dr, mag = dr + dstream.double(), mag + dstream.double().abs()
    xh = d * rstd
    wmag = (dy.abs() * K * (xh.abs() + (1.0 if ln else 0.0))).sum(0)
    return dr, mag, (dy * xh).sum(0), wmag, dy.sum(0), dy.abs().sum(0)


def finalize(y, pair_row, w, y_sh, x, gate_w):
    """out [T, H] of float64 y [rows, H], w [T, k] (or None) and a gated shared expert (or None)."""
    keep = (pair_row >= 0).to(y.dtype)
    wk = keep if w is None else w * keep
    out = (y[pair_row.clamp(min=0).long()] * wk.unsqueeze(-1)).sum(1)
    return out if gate_w is None else out + torch.sigmoid(x @ gate_w).unsqueeze(-1) * y_sh


def permuted(x, pair_row, w, rows):
    """x_perm [rows, H] of float64 x and weights (or None)."""
    T, k = pair_row.shape
    live = (pair_row >= 0).nonzero()
    src = x[live[:, 0]]
    if w is not None:
        src = src * w[live[:, 0], live[:, 1]].unsqueeze(-1)
    out = torch.zeros(rows, x.shape[1], dtype=x.dtype, device=x.device)
    return out.index_put((pair_row[live[:, 0], live[:, 1]].long(),), src)


def weights(logits, ids, renorm):
    """The routing weights of the chosen experts, float64."""
    chosen = logits.gather(1, ids.long())
    return torch.softmax(chosen, 1) if renorm else torch.softmax(logits, 1).gather(1, ids.long())


def routing(T, E, k, S=None, seed=0, pad=0):
    """(pair_row [T, k] int32, topk_w [T, k] fp32, rows) as moe_route and moe_permute leave them: experts at or above S
    are another rank's (row -1, weight 0)."""
    g = torch.Generator().manual_seed(seed * 1009 + T * 31 + E)
    score, ids = torch.randn(T, E, generator=g).topk(k, dim=1)
    S = E if S is None else S
    key = torch.where(ids < S, ids, S).reshape(-1)
    order = torch.argsort(key, stable=True)
    row = torch.empty_like(order)
    row[order] = torch.arange(T * k)
    keep = (key < S).reshape(T, k)
    pr = torch.where(keep, row.reshape(T, k), -1).to(torch.int32)
    w = torch.where(keep, torch.softmax(score, 1), torch.zeros(()))
    return pr.contiguous().cuda(), w.contiguous().cuda(), T * k + pad


def rnd(*shape, seed=0, std=1.0, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed * 7919 + sum(shape))
    return (torch.randn(*shape, generator=g) * std).to(dtype).cuda()


def inside(got, ref, tol, what):
    """Every element of got within tol (a tensor, or 0) of ref, and one bf16 rounding where got is bf16."""
    got = got.double()
    err = (got - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err / (tol + 1e-300)).max()):.3g} x"
