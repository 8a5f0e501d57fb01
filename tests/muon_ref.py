"""Newton-Schulz orthogonalisation and Muon's update in 64 bits, and the error that the kernels' number formats may add.

Formats: X is held as a pair of fp16 (22 bits), A and P as fp16 with P's diagonal
in fp32, all times one power of two S; products take fp16 operands (of X the high
one) and add in fp32; y is bf16.

One step has a bound for every element (one_step_bound), from these half steps
alone.  Over several steps a bound of that kind grows by the largest slope of the
steps' polynomial each time and says little, so several steps are held to what the
same roundings do to the same matrix: `emulated` takes them in 64-bit arithmetic,
and the kernel's error may be three times the emulation's (whose roundings fall
otherwise, since the order of the fp32 sums differs), row by row and column by
column, beside the result's own rounding.
"""
import torch

STEP = (3.4445, -4.7750, 2.0315)
U32, U16 = 2.0 ** -24, 2.0 ** -11
SCALE = 2.0 ** 14


def orthogonal(x, steps, eps=1e-7):
    x = x.double()
    n = x.norm()
    x = x / (n + eps) if n + eps > 0 else x
    tall = x.shape[0] > x.shape[1]
    x = x.t() if tall else x
    for a, b, c in steps:
        g = x @ x.t()
        x = a * x + (b * g + c * (g @ g)) @ x
    return x.t() if tall else x


def f16(x, scale=SCALE):
    return (x * scale).to(torch.float16).double() / scale


def emulated(x, steps, eps=1e-7, scale=SCALE):
    """`orthogonal` with the kernels' roundings (not the final one)."""
    x = x.double()
    x = x / (x.norm() + eps)
    tall = x.shape[0] > x.shape[1]
    x = x.t() if tall else x
    for a, b, c in steps:
        hi = f16(x, scale)
        lo = f16((x - hi) * 2048, scale) / 2048
        g = f16(hi @ hi.t(), scale)
        p = b * g + c * (g @ g)
        d = p.diagonal().clone()
        off = f16(p - torch.diag(d), scale)
        x = (a + d)[:, None] * (hi + lo) + off @ hi
    return x.t() if tall else x


def one_step_bound(x, step, eps=1e-7, scale=SCALE):
    """(X' in 64 bits, its bound ahead of the final rounding) for one step from x."""
    a, b, c = (abs(v) for v in step)
    want = orthogonal(x, (step,), eps)
    x = x.double()
    x = x / (x.norm() + eps)
    tall = x.shape[0] > x.shape[1]
    x = x.t() if tall else x
    m, n = x.shape
    least = 2.0 ** -25 / scale                       # half a step of fp16's smallest values
    h, dh = x.abs(), U16 * x.abs() + least + 4 * U32 * x.abs()
    g = x @ x.t()
    e_g = 2 * dh @ h.t() + dh @ dh.t() + (n + 64) * U32 * (h @ h.t())
    e_g = e_g + U16 * (g.abs() + e_g) + least
    p = step[1] * g + step[2] * (g @ g)
    ga = g.abs()
    e_p = b * e_g + c * (e_g @ ga + ga @ e_g + e_g @ e_g + (m + 64) * U32 * (ga @ ga)) + 4 * U32 * (b * ga + c * (ga @ ga))
    e_p = e_p + U16 * (p.abs() + e_p) + least
    pa = p.abs()
    e = a * (2.0 ** -21 + 6 * U32) * h + 2 * least + e_p @ (h + dh) + pa @ dh + (m + 64) * U32 * (pa @ h) + 4 * U32 * want.t().abs() \
        if tall else a * (2.0 ** -21 + 6 * U32) * h + 2 * least + e_p @ (h + dh) + pa @ dh + (m + 64) * U32 * (pa @ h) + \
        4 * U32 * want.abs()
    return want, e.t() if tall else e


def assert_near(got, x, steps, eps=1e-7, scale=SCALE, what="", slack=None):
    """Rows and columns of `got` against `orthogonal` within the emulation's error and, of each element, `slack` (None:
    bf16's rounding)."""
    want = orthogonal(x, steps, eps)
    rough = emulated(x, steps, eps, scale)
    off, own = got.double() - want, torch.finfo(torch.bfloat16).eps / 2
    slack = own * want.abs() if slack is None else slack
    for dim in (0, 1):
        line = want.norm(dim=dim)
        most = slack.norm(dim=dim) + 3 * (rough - want).norm(dim=dim).max() * (1 + own) + 1e-30
        bad = ~(off.norm(dim=dim) <= most)
        assert not bad.any(), (f"{what}: {int(bad.sum())} {'columns' if dim == 0 else 'rows'} off, first {int(bad.nonzero()[0])}: "
                               f"{off.norm(dim=dim)[bad][0].item():.3g} of {line[bad][0].item():.3g}, bound {most[bad][0].item():.3g}")


def emulated_pairs(x, steps, eps=1e-7, scale=SCALE):
    """The same with X, A and P as pairs of fp16, three products of their parts and fp32 sums: matrices of 33 to 64 by up to 256."""
    def pair(v):
        hi = f16(v, scale)
        return hi.float(), f16((v - hi) * 2048, scale).float()

    def product(u, v):
        return (u[0] @ v[0] + (u[0] @ v[1] + u[1] @ v[0]) / 2048).double()

    x = x.double()
    x = x / (x.norm() + eps)
    tall = x.shape[0] > x.shape[1]
    x = x.t() if tall else x
    for a, b, c in steps:
        xs = pair(x)
        g = pair(product(xs, [t.t() for t in xs]))
        p = pair(b * (g[0].double() + g[1].double() / 2048) + c * product(g, g))
        x = a * (xs[0].double() + xs[1].double() / 2048) + product(p, xs)
    return x.t() if tall else x


def emulated_gram(x, steps, eps=1e-7):
    """Shorter sides up to 64, growth up to 2048: polynomials of the Gram matrix in 64 bits, their product Q and Q U in fp32."""
    x = x.double()
    tall = x.shape[0] > x.shape[1]
    x = x.t() if tall else x
    inv = 1 / (x.norm() + eps)
    r, one = (x @ x.t()) * inv * inv, torch.eye(len(x), dtype=torch.float64)
    q = one
    for a, b, c in steps:
        p = a * one + b * r + c * (r @ r)
        q, r = p @ q, p @ r @ p
    x = (q.float() @ (x * inv).float()).double()
    return x.t() if tall else x
