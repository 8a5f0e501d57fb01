"""Layer norm where every workgroup walks over several rows, for each of the kernels' shapes (threads a row, chunks a
thread) in each type: the next row's loads, the sums' places in turn, a last round that not all workgroups have."""
import pytest
import torch

from precision_block_scaled_amd import pipeline as PL
from tests.norm_ref import norm_grad_ref, norm_ref

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
TYPES = [(BF, BF, BF), (F32, BF, F32), (F32, F32, F32), (BF, F32, BF)]
# (rows, cols): more than twice the workgroups' rows (16 rows of 16 threads, 4 of 64, one of more; at most 1024, 768 and
# 768 workgroups, 512 and 256 for the widest, 2048 beyond 16384 columns), widths of whole chunks and others
SHAPES = [(33001, 24), (33001, 127), (33001, 200), (33001, 253), (33001, 320), (33001, 381), (6203, 512), (6203, 509),
          (6203, 1000), (6203, 1001), (6203, 1048), (6203, 1027), (6203, 1400), (6203, 1401), (1603, 2000), (1603, 2043),
          (1603, 2080), (1603, 2081), (1603, 2600), (1603, 2601), (1603, 4096), (1603, 4091), (1603, 5008), (1603, 5003),
          (1101, 8192), (1101, 8187), (601, 10008), (601, 10007), (1101, 16384), (1101, 16381), (4201, 16392)]


def make(rows, cols, tx, ty, tw, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    x = (normal(rows, cols) * (1 + normal(rows, 1).abs()) + normal(rows, 1)).to(tx)      # no two rows alike
    return x, (1 + 0.3 * normal(cols)).to(tw), (0.2 * normal(cols)).to(tw), (0.1 * normal(rows, cols)).to(ty)


def within(got, want, bound, what):
    off = (got.double() - want).abs()
    bad = ~(off <= bound)
    if bad.any():
        at = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound; first {at}: got "
                             f"{got[at].item()!r} want {want[at].item()!r} bound {bound[at].item()!r}")


def check(x, gamma, beta, dy, ty, in_place):
    amax = torch.empty(1, device="cuda")
    y, mean, rstd = PL.layernorm(x, gamma, beta, 1e-5, out_dtype=ty, amax=amax)
    want = norm_ref(x.double(), gamma.double(), beta.double(), 1e-5, ty)
    for got, k, name in ((y, 0, "y"), (mean, 2, "mean"), (rstd, 4, "rstd")):
        within(got, want[k], want[k + 1], name)
    assert amax.item() == y.float().abs().max().item()
    del want
    grads = PL.layernorm_grad(dy, x, gamma, mean, rstd)
    want = norm_grad_ref(dy.double(), x.double(), gamma.double(), mean.double(), rstd.double(), x.dtype)
    for got, k, name in zip(grads, (0, 2, 4), ("dx", "dgamma", "dbeta")):
        within(got, want[k], want[k + 1], name)
    del want
    if not in_place:
        return
    for on_dy in (False, True):                       # dx in the place of x, and of dy
        if on_dy and dy.dtype != x.dtype:
            continue
        a, b = x.clone(), dy.clone()
        got = PL.layernorm_grad(b, a, gamma, mean, rstd, dx=b if on_dy else a)
        assert all(torch.equal(u, v) for u, v in zip(got, grads))
    if ty == x.dtype:
        again = PL.layernorm(x, gamma, beta, 1e-5, y=x)
        assert torch.equal(x, y) and torch.equal(again[1], mean) and torch.equal(again[2], rstd)


@pytest.mark.parametrize("types", TYPES, ids=lambda t: "-".join(str(d)[6:] for d in t))
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_several_rows_a_workgroup(rows, cols, types):
    """The results within the formulas' bounds; in place, the same bytes (rows of odd width end in a window that holds
    columns of another thread, in wide rows of another wave)."""
    tx, ty, tw = types
    check(*make(rows, cols, tx, ty, tw, seed=rows + cols), ty, in_place=True)


@pytest.mark.parametrize("rows,cols", [(270001, 250), (66001, 1100), (33001, 2048), (33001, 2057), (26001, 2600),
                                       (16501, 4096)])
def test_fp32_past_the_last_level_cache(rows, cols):
    """Inputs of more than 256 MiB from fp32 to fp32, which fewer workgroups walk over."""
    check(*make(rows, cols, F32, F32, F32, seed=cols), F32, in_place=False)
