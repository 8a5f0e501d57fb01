"""The linear head's losses and gradients in 64 bits, with the error that the
calls' arithmetic may add (first order, worst case).

U = 2^-24: one fp32 rounding.  The matrix instruction's sums run through at
most ``hidden`` (``vocab``, tokens) fp32 additions.  Half a step of bf16 is
2^-8 of the value; up to PAIR_TOKENS tokens dz is a sum of two bf16 terms,
2^-16 of the value.  TINY = 2^-126, the smallest normal number of fp32 and of
bf16: the exponential instruction and the matrix instruction may take anything
below it for 0, so a q or a dz smaller than that is off by up to TINY (a logit
100 below the maximum gives q = 4e-44; times x = 1000 summed into dw, the
formula's 1e-36 and the call's 0 differ by no more than TINY * 1000 a term).
"""
import torch

U = 2.0 ** -24
TINY = 2.0 ** -126
PAIR_TOKENS = 128
BF16 = torch.finfo(torch.bfloat16).eps / 2


def slots_of(targets=None, top_ids=None, top_logits=None, tau=1.0):
    """(ids [T, k], p [T, k], live [T], sum p log p [T]) in float64; unused slots have id -1 and p 0."""
    if targets is not None:
        live = targets >= 0
        return targets[:, None], live.double()[:, None], live, torch.zeros(len(targets), dtype=torch.float64)
    t = top_logits.double().masked_fill(top_ids < 0, -torch.inf)
    live = ~(t == -torch.inf).all(1)
    high = torch.where(live, t.amax(1), 0.0)[:, None]
    e = (t - high) / tau
    p = torch.where(live[:, None], e.exp(), 0.0)
    total = torch.where(live, p.sum(1), 1.0)[:, None]
    p = p / total
    ent = torch.where(p > 0, p * (e - total.log()), 0.0).sum(1)
    return torch.where(p > 0, top_ids, -1), p, live, ent


def head_ref(x, w, slots, tau=1.0, dloss=None, kept=(None, None)):
    """x [T, H], w [V, H] float64 (rows of x that take no part may hold anything).

    Returns a dict of (value, bound) for loss, lse and, with dloss, dx (bf16
    store) and dw (before its own store's rounding).  kept: masks [T, V] of the
    values of dz that reach dx, and dw, with what their rounding left out.
    """
    ids, p, live, ent = slots
    T, H = x.shape
    V = w.shape[0]
    x = torch.where(live[:, None], x, 0.0)
    z = x @ w.t() / tau
    # H additions, the multiplication by 1/tau and the rounding of 1/tau
    e_z = (H + 3) * U * (x.abs() @ w.abs().t()) / tau
    lse = torch.logsumexp(z, 1)
    q = (z - lse[:, None]).exp()
    # an exponential: its argument's rounding (z - max, times log2 e), weighted by itself, and the function
    # (2 U); at most V / 8 + 200 additions on a path; the logarithm and the last addition
    reach = z.amax(1) - lse
    e_lse = (q * e_z).sum(1) + (V / 8 + 220 + 4 * (q * (z.amax(1, keepdim=True) - z)).sum(1)) * U + 4 * U * (
        lse.abs() + reach.abs())
    k = p.shape[1]
    at = ids.clamp(min=0)
    zs, e_zs = z.gather(1, at), e_z.gather(1, at)
    t = zs - lse[:, None]
    e_p = (k + 12 + 4 * (-p.clamp(min=1e-300).log())) * U * p
    loss = torch.where(live, ent - (p * t).sum(1), 0.0)
    e_loss = ((p * (e_zs + e_lse[:, None]) + e_p * (t.abs() + p.clamp(min=1e-300).log().abs() + 1)).sum(1) +
              (k + 4) * U * ((p * t.abs()).sum(1) + ent.abs()))
    out = dict(loss=(loss, torch.where(live, e_loss, 0.0)),
               lse=(torch.where(live, lse, 0.0), torch.where(live, e_lse, 0.0)))
    if dloss is None:
        return out
    c = torch.where(live, dloss, 0.0)[:, None] / tau
    hit = torch.zeros_like(z).scatter_add_(1, at, p)
    e_hit = torch.zeros_like(z).scatter_add_(1, at, e_p)
    dz = c * (q - hit)
    # q carries the logit's and lse's errors, the argument's roundings and the function's
    e_q = q * (e_z + 2 * e_lse[:, None] + (4 * (z - lse[:, None]).abs() + 6) * U)
    e_dz = c.abs() * (e_q + e_hit + 4 * U * (q + (k + 1) * hit))
    e_32 = e_dz

    def rounded(mask):
        step = BF16 ** 2 if T <= PAIR_TOKENS else BF16 if mask is None else torch.where(mask, BF16 ** 2, BF16)
        return e_32 + step * (dz.abs() + e_32) + TINY * (1 + c.abs())

    dx = dz @ w
    e_dx = rounded(kept[0]) @ w.abs() + (V + 40) * U * (dz.abs() @ w.abs())
    out["dx"] = (dx, e_dx + BF16 * (dx.abs() + e_dx) + TINY)
    dw = dz.t() @ x
    out["dw"] = (dw, rounded(kept[1]).t() @ x.abs() + (T + 40) * U * (dz.abs().t() @ x.abs()) + TINY)
    return out


def stored(value_bound, dtype):
    v, e = value_bound
    return v, e + torch.finfo(dtype).eps / 2 * (v.abs() + e)
