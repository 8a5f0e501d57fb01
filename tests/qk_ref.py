"""Norm and rotation of queries and keys and their gradient in 64 bits, with the error that fp32 arithmetic may add.

Bounds: U = 2^-24 is one fp32 rounding.  A row's sums run through at most ROW_ADDS
additions per value: a lane adds up to 16 of its own, then 6 joins.  cos and sin
carry E_CS: the reduced angle, at most half a turn, is rounded once (pi U), the
function adds at most 2 units in the last place (4 U), and three roundings in 64
bits ahead of the reduction count relative to the whole angle, twice over since the
reference rounds too.
"""
import math

import torch

U = 2.0 ** -24
ROW_ADDS = 24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def turn(x, cos, sin, interleaved):
    rot = 2 * cos.shape[-1]
    if rot == 0:
        return x
    h, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        p, q = h[..., 0::2], h[..., 1::2]
        return torch.cat((torch.stack((p * cos - q * sin, q * cos + p * sin), -1).flatten(-2), rest), -1)
    p, q = h.chunk(2, -1)
    return torch.cat((p * cos - q * sin, q * cos + p * sin, rest), -1)


def turn_bound(x, e_x, cos, sin, e_cs, interleaved):
    """Bound of turn(x) for x off by e_x and cos, sin off by e_cs."""
    rot = 2 * cos.shape[-1]
    if rot == 0:
        return e_x

    def part(p, q, ep, eq):
        lead = p.abs() * e_cs + q.abs() * e_cs + ep * (cos.abs() + e_cs) + eq * (sin.abs() + e_cs)
        return lead + 3 * U * ((p.abs() + ep) * (cos.abs() + e_cs) + (q.abs() + eq) * (sin.abs() + e_cs))

    h, e, rest = x[..., :rot], e_x[..., :rot], e_x[..., rot:]
    if interleaved:
        p, q, ep, eq = h[..., 0::2], h[..., 1::2], e[..., 0::2], e[..., 1::2]
        return torch.cat((torch.stack((part(p, q, ep, eq), part(q, p, eq, ep)), -1).flatten(-2), rest), -1)
    (p, q), (ep, eq) = h.chunk(2, -1), e.chunk(2, -1)
    return torch.cat((part(p, q, ep, eq), part(q, p, eq, ep), rest), -1)


def angles(positions, freqs, shape, device):
    """cos, sin and their bound, [batch, seq, 1, rot / 2]."""
    B, S = shape[:2]
    pos = torch.arange(S, device=device) if positions is None else positions.to(device)
    if freqs is None:
        z = torch.zeros(B, S, 1, 0, dtype=torch.float64, device=device)
        return z, z, z
    a = pos.double().expand(B, S)[:, :, None, None] * freqs.to(device)
    return a.cos(), a.sin(), math.pi * U + 4 * U + 6 * 2.0 ** -53 * a.abs()


def normed(x, eps, norm):
    """n = x r, r, and the relative error of r and of n."""
    if not norm:
        one = torch.ones_like(x[..., :1])
        return x, one, 0 * one
    ms = x.square().mean(-1, keepdim=True)
    r = 1 / (ms + eps).sqrt()
    rel = 0.5 * (ROW_ADDS + 4) * U + 3 * U
    return x * r, r, rel + 0 * r


def forward_ref(x, w, positions, freqs, interleaved, eps, norm, out_dtype):
    """(y, bound) in float64 from a float64 x [B, S, H, D]."""
    cos, sin, e_cs = angles(positions, freqs, x.shape, x.device)
    n, _, rel = normed(x, eps, norm)
    u = n if w is None else n * w
    e_u = (rel + 2 * U) * u.abs()
    y = turn(u, cos, sin, interleaved)
    e = turn_bound(u, e_u, cos, sin, e_cs, interleaved)
    return y, e + half_step(out_dtype) * (y.abs() + e) + 1e-40


def grad_ref(dy, x, w, positions, freqs, interleaved, eps, norm, out_dtype, strips):
    """(dx, bound, dw, bound); strips: workgroups that share the rows' sums."""
    B, S, H, D = x.shape
    cos, sin, e_cs = angles(positions, freqs, x.shape, x.device)
    n, r, rel = normed(x, eps, norm)
    g = turn(dy, cos, -sin, interleaved)
    e_g = turn_bound(dy, 0 * dy, cos, sin, e_cs, interleaved)
    ww = torch.ones(D, dtype=torch.float64, device=x.device) if w is None else w
    v, e_v = g * ww, (e_g + U * g.abs()) * ww.abs()
    dx, e = r * v, r * (e_v + (rel + 2 * U) * v.abs())
    if norm:
        mean = (v * n).mean(-1, keepdim=True)
        e_mean = (e_v * n.abs() + (rel + (ROW_ADDS + 5) * U) * (v * n).abs()).mean(-1, keepdim=True)
        dx = r * (v - n * mean)
        e = r * (e_v + n.abs() * e_mean + (2 * rel + 4 * U) * (v.abs() + (n * mean).abs()))
    t = g * n
    chain = -(-(B * S) // (4 * strips)) * H + 6 + 4 + 768 // 64 + 64
    e_dw = (e_g * n.abs() + (rel + 2 * U) * t.abs() + chain * U * t.abs()).sum((0, 1, 2))
    return dx, e + half_step(out_dtype) * (dx.abs() + e) + 1e-40, t.sum((0, 1, 2)), e_dw + 1e-40


def strips_of(tokens, heads, all_heads):
    """At most as many workgroups as share the sums of a tensor of `heads` among `all_heads` heads: a part's share
    of 768 goes by its rounds of heads and a constant, so it is no less than half of its share of the heads."""
    return max(1, min(-(-tokens // 4), 384 * heads // all_heads - 1))
