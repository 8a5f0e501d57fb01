"""Layer norm and its gradient in 64 bits, with the error that fp32 arithmetic may add.

Bounds: U = 2^-24 is one fp32 rounding.  A sum of terms t_i formed with at
most k additions on any path is off by at most k U sum |t_i| (first order).
A row's sums run through at most ROW_ADDS(cols) additions per value: a thread
of a workgroup of at least 16 threads adds its own cols / 16 values at most,
then 10 joins.  A column's sums run through at most COL_ADDS(rows): strips
of rows / 256 + 8 at most, joined from at most 2048 of them.
"""
import numpy as np
import torch

U = 2.0 ** -24


def row_adds(cols):
    return -(-cols // 16) + 10


def col_adds(rows):
    return rows if rows <= 2048 else rows // 256 + 8 + 2048


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def norm_ref(x, gamma, beta, eps, out_dtype):
    """(y, bound of y, mu, bound of mu, r, bound of r) in float64 from float64 inputs."""
    n = x.shape[1]
    k = row_adds(n)
    mu = x.mean(1)
    e_mu = (k + 1) * U * x.abs().mean(1)
    d = x - mu[:, None]
    var = d.square().mean(1)
    # d carries e_mu and one rounding; its square two more, the sum k, the division and eps one each
    e_d = e_mu[:, None] + U * d.abs()
    e_var = (2 * d.abs() * e_d + e_d.square()).mean(1) + (k + 4) * U * (var + eps)
    r = 1 / (var + eps).sqrt()
    lo = (var + eps - e_var).clamp(min=0)
    e_r = torch.where(lo > 0, 0.5 * e_var / lo.clamp(min=1e-300) * r, torch.inf) + 3 * U * r
    nrm = d * r[:, None]
    e_n = e_d * r[:, None] + d.abs() * e_r[:, None] + 2 * U * nrm.abs()
    y = nrm * gamma + beta
    e_y = e_n * gamma.abs() + 2 * U * (nrm * gamma).abs() + 2 * U * y.abs()
    return y, e_y + half_step(out_dtype) * (y.abs() + e_y), mu, e_mu, r, e_r


def norm_grad_ref(dy, x, gamma, mean, rstd, out_dtype):
    """(dx, bound, dgamma, bound, dbeta, bound) in float64; mean / rstd are inputs, as the call has them."""
    rows, n = x.shape
    k = row_adds(n)
    r = rstd[:, None]
    nrm = (x - mean[:, None]) * r
    u = dy * gamma
    mu_u, mu_un = u.mean(1, keepdim=True), (u * nrm).mean(1, keepdim=True)
    dx = r * (u - mu_u - nrm * mu_un)
    e_n = 3 * U * nrm.abs() + U * (x - mean[:, None]).abs() * r
    e_u = U * u.abs()
    e_mu = (k + 2) * U * u.abs().mean(1, keepdim=True)
    e_un = ((u * nrm).abs() * ((k + 4) * U) + u.abs() * e_n).mean(1, keepdim=True)
    e = e_u + e_mu + e_n * mu_un.abs() + nrm.abs() * e_un + 3 * U * (u.abs() + mu_u.abs() + (nrm * mu_un).abs())
    e_dx = r.abs() * e + 2 * U * dx.abs()
    kc = col_adds(rows)
    t = dy * nrm
    e_dg = (dy.abs() * e_n + (kc + 1) * U * t.abs()).sum(0)
    e_db = kc * U * dy.abs().sum(0)
    return dx, e_dx + half_step(out_dtype) * (dx.abs() + e_dx), t.sum(0), e_dg, dy.sum(0), e_db


def assert_within(got, want, bound, what):
    got = got.double().cpu()
    off = (got - want).abs()
    bad = ~(off <= bound)
    if bad.any():
        i = tuple(int(v) for v in np.argwhere(bad.numpy())[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound; first {i}: got "
                             f"{got[i].item()!r} want {want[i].item()!r} bound {bound[i].item()!r}")
