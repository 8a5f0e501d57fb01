"""Layer norm and its gradient on the GPU against the formulas in 64 bits."""
import pytest
import torch

import precision_block_scaled_amd as P
from precision_block_scaled_amd import pipeline as PL
from tests.norm_ref import assert_within, norm_grad_ref, norm_ref

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
# widths around every split of a row over threads: one to 16 values a thread group, 128, 256, 384, 512, 1024, 1536, 2048,
# 2816, 4096, 5632, 8192, 12288, 16384 and beyond
SHAPES = [(1, 1), (1, 7), (3, 8), (5, 9), (70, 64), (2, 127), (17, 128), (65, 129), (33, 512), (9, 513), (7, 1000),
          (5, 2048), (3, 2049), (515, 4096), (2, 4097), (3, 5003), (2, 5632), (2, 5640),
          (3, 8192), (2, 8200), (3, 10007), (2, 12288), (2, 12290), (2, 16384), (2, 16391), (1, 40000),
          (5000, 24), (2500, 770), (70, 136), (5000, 256), (33, 257), (4100, 384), (9, 385), (66, 1032), (2100, 1536),
          (5, 1537), (3, 2056), (600, 2816), (4, 2817)]
TYPES = [(BF, BF, BF), (F32, BF, F32), (F32, F32, F32), (BF, F32, BF)]


def make(rows, cols, tx, ty, tw, seed=0, offset=0.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, cols, generator=g) * (1 + 10 * (torch.rand(cols, generator=g) < 0.02)) + offset).to(tx)
    gamma = (1 + 0.3 * torch.randn(cols, generator=g)).to(tw)
    beta = (0.2 * torch.randn(cols, generator=g)).to(tw)
    dy = (torch.randn(rows, cols, generator=g) * 0.1).to(ty)
    return x, gamma, beta, dy


def check_forward(x, gamma, beta, y, mean, rstd, eps, what):
    want, e, mu, e_mu, r, e_r = norm_ref(x.double(), gamma.double(), beta.double(), eps, y.dtype)
    assert_within(mean, mu, e_mu, what + " mean")
    assert_within(rstd, r, e_r, what + " rstd")
    assert_within(y, want, e, what + " y")


def check_grad(dy, x, gamma, mean, rstd, dx, dgamma, dbeta, what):
    w = norm_grad_ref(dy.double(), x.double(), gamma.double(), mean.double().cpu(), rstd.double().cpu(), x.dtype)
    assert_within(dx, w[0], w[1], what + " dx")
    assert_within(dgamma, w[2], w[3], what + " dgamma")
    assert_within(dbeta, w[4], w[5], what + " dbeta")


@pytest.mark.parametrize("types", TYPES, ids=lambda t: "-".join(str(d)[6:] for d in t))
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward_and_gradient(rows, cols, types):
    tx, ty, tw = types
    x, gamma, beta, dy = make(rows, cols, tx, ty, tw, seed=rows + cols)
    amax = torch.full((1,), 99.0, device="cuda")
    xg, gg, bg, dyg = (t.cuda() for t in (x, gamma, beta, dy))
    y, mean, rstd = PL.layernorm(xg, gg, bg, 1e-5, out_dtype=ty, amax=amax)
    assert y.dtype == ty
    if cols > 1:
        check_forward(x, gamma, beta, y, mean, rstd, 1e-5, f"{rows}x{cols}")
    else:
        assert torch.equal(y.cpu(), beta.to(ty).expand(rows, 1))   # x - mean(x) = 0
    assert amax.item() == y.float().abs().max().item()
    dx, dgamma, dbeta = PL.layernorm_grad(dyg, xg, gg, mean, rstd)
    assert dx.dtype == tx and dgamma.dtype == F32
    check_grad(dy, x, gamma, mean, rstd, dx, dgamma, dbeta, f"{rows}x{cols}")
    again = PL.layernorm_grad(dyg, xg, gg, mean, rstd)
    for a, b in zip(again, (dx, dgamma, dbeta)):
        assert torch.equal(a, b)


def test_many_rows():
    """Many rows a strip, and a last row that is not the last strip's."""
    x, gamma, beta, dy = make(33001, 1601, BF, BF, BF, seed=5)
    y, mean, rstd = PL.layernorm(x.cuda(), gamma.cuda(), beta.cuda(), 1e-5)
    check_forward(x, gamma, beta, y, mean, rstd, 1e-5, "rows")
    got = PL.layernorm_grad(dy.cuda(), x.cuda(), gamma.cuda(), mean, rstd)
    check_grad(dy, x, gamma, mean, rstd, *got, "rows")


def test_no_weights_and_single_outputs():
    x, _, _, dy = make(37, 200, BF, BF, BF)
    one, zero = torch.ones(200), torch.zeros(200)
    y, mean, rstd = PL.layernorm(x.cuda())
    check_forward(x, one, zero, y, mean, rstd, 1e-5, "plain")
    full = PL.layernorm_grad(dy.cuda(), x.cuda(), None, mean, rstd)
    check_grad(dy, x, one, mean, rstd, *full, "plain")
    # any of the three outputs alone, through the C names
    n = P.pbs_layernorm_grad_bytes(37, 200)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    for i, want in enumerate(full):
        out = torch.full_like(want, 7.0)
        outs = [out if j == i else None for j in range(3)]
        P.pbs_layernorm_grad(dy.cuda(), P.PBS_FMT_BF16, 200, x.cuda(), P.PBS_FMT_BF16, 200, 37, 200, None,
                             P.PBS_FMT_F32, mean, rstd, outs[0], 200, outs[1], outs[2], ws if i else None,
                             n if i else 0)
        assert torch.equal(out, want)


@pytest.mark.parametrize("tx,cols,ld,skip", [(BF, 96, 111, 1), (BF, 4096, 4099, 3), (F32, 1000, 1003, 1),
                                             (F32, 9000, 9001, 3), (BF, 17000, 17001, 1), (BF, 13, 13, 1)])
def test_strided_rows_and_odd_addresses(tx, cols, ld, skip):
    """Rows ld apart that start at any element; what lies between them stays as it was."""
    rows = 5
    x, gamma, beta, dy = make(rows, cols, tx, tx, BF, seed=cols)

    def placed(t):
        flat = torch.full((rows * ld + 16,), 123.0, dtype=tx, device="cuda")
        view = flat[skip:skip + rows * ld].view(rows, ld)[:, :cols]
        if t is not None:
            view.copy_(t)
        return flat, view

    _, xv = placed(x)
    _, dyv = placed(dy)
    yf, yv = placed(None)
    dxf, dxv = placed(None)
    gp = torch.empty(cols + 1, dtype=BF, device="cuda")[1:]
    gp.copy_(gamma)
    _, mean, rstd = PL.layernorm(xv, gp, beta.cuda(), y=yv)
    check_forward(x, gamma, beta, yv, mean, rstd, 1e-5, "strided")
    _, dgamma, dbeta = PL.layernorm_grad(dyv, xv, gp, mean, rstd, dx=dxv)
    check_grad(dy, x, gamma, mean, rstd, dxv, dgamma, dbeta, "strided")
    for f, v in ((yf, yv), (dxf, dxv)):
        v.fill_(123.0)
        assert (f == 123.0).all()


@pytest.mark.parametrize("cols", [64, 300, 4096, 20000])
def test_in_place(cols):
    x, gamma, beta, dy = make(11, cols, BF, BF, F32, seed=cols)
    xg, gg, bg, dyg = (t.cuda() for t in (x, gamma, beta, dy))
    y, mean, rstd = PL.layernorm(xg, gg, bg)
    dx, dgamma, dbeta = PL.layernorm_grad(dyg, xg, gg, mean, rstd)
    for target in (0, 1):
        a, b = xg.clone(), dyg.clone()
        got = PL.layernorm_grad(b, a, gg, mean, rstd, dx=(a, b)[target])
        assert got[0].data_ptr() == (a, b)[target].data_ptr()
        for u, v in zip(got, (dx, dgamma, dbeta)):
            assert torch.equal(u, v)
    PL.layernorm(xg, gg, bg, y=xg)
    assert torch.equal(xg, y)


@pytest.mark.parametrize("cols", [100, 4096, 16384, 20000])
def test_common_offset_and_constant_rows(cols):
    """A large common offset costs no digits beyond the input's own; a constant row has no spread."""
    x, gamma, beta, dy = make(6, cols, F32, F32, F32, seed=3, offset=1000.0)
    x[2] = 5.0
    y, mean, rstd = PL.layernorm(x.cuda(), gamma.cuda(), beta.cuda(), 1e-5)
    check_forward(x, gamma, beta, y, mean, rstd, 1e-5, "offset")
    got = PL.layernorm_grad(dy.cuda(), x.cuda(), gamma.cuda(), mean, rstd)
    check_grad(dy, x, gamma, mean, rstd, *got, "offset")


@pytest.mark.parametrize("cols", [5, 64, 256, 768, 2304, 8256, 17000])
def test_mean_times_rstd_past_the_range(cols):
    """Constant rows of 2^83 with eps = 1e-30: n is 0 although mean * rstd overflows, and dx = rstd (u - mean(u))."""
    x = torch.full((3, cols), 2.0 ** 83)
    _, gamma, beta, dy = make(3, cols, F32, F32, F32, seed=cols)
    mean, rstd = torch.full((3,), 2.0 ** 83), torch.full((3,), 1e15)
    got = PL.layernorm_grad(dy.cuda(), x.cuda(), gamma.cuda(), mean.cuda(), rstd.cuda())
    check_grad(dy, x, gamma, mean, rstd, *got, "overflow")


@pytest.mark.parametrize("cols", [48, 4096, 17000])
def test_nan_and_infinite_rows_stay_alone(cols):
    x, gamma, beta, _ = make(9, cols, BF, BF, BF, seed=1)
    want, mean0, rstd0 = PL.layernorm(x.cuda(), gamma.cuda(), beta.cuda())
    x[3, 1], x[5, 2], x[7, 0] = float("nan"), float("inf"), float("-inf")
    y, mean, rstd = PL.layernorm(x.cuda(), gamma.cuda(), beta.cuda())
    for r in range(9):
        if r in (3, 5, 7):
            assert y[r].isnan().all()
        else:
            assert torch.equal(y[r], want[r]) and mean[r] == mean0[r] and rstd[r] == rstd0[r]


def test_no_rows():
    x = torch.empty(0, 40, dtype=BF, device="cuda")
    amax = torch.full((1,), 5.0, device="cuda")
    y, mean, rstd = PL.layernorm(x, amax=amax)
    assert y.shape == (0, 40) and mean.shape == (0,) and amax.item() == 0
    dx, dgamma, dbeta = PL.layernorm_grad(x, x, None, mean, rstd)
    assert dx.shape == (0, 40) and not dgamma.any() and not dbeta.any() and dgamma.shape == (40,)


def test_rows_beyond_four_gib():
    """Row offsets past 2^32 bytes: a strided view of a buffer of 4.5 GiB, whose rows lie 512 MiB apart."""
    ld = (1 << 29) // 2 + 1
    flat = torch.zeros(9 * ld, dtype=BF, device="cuda")
    xv = flat.view(9, ld)[:, :300]
    x, gamma, beta, dy = make(9, 300, BF, BF, BF, seed=2)
    xv.copy_(x)
    y, mean, rstd = PL.layernorm(xv, gamma.cuda(), beta.cuda())
    check_forward(x, gamma, beta, y, mean, rstd, 1e-5, "far rows")
    dx, dgamma, dbeta = PL.layernorm_grad(dy.cuda(), xv, gamma.cuda(), mean, rstd, dx=xv)
    check_grad(dy, x, gamma, mean, rstd, dx, dgamma, dbeta, "far rows")


def test_other_stream_and_graph():
    x, gamma, beta, dy = (t.cuda() for t in make(130, 1000, BF, BF, BF, seed=9))
    amax0, amax1 = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")
    y, mean, rstd = PL.layernorm(x, gamma, beta, amax=amax0)
    want = PL.layernorm_grad(dy, x, gamma, mean, rstd)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for s in (side, side.cuda_stream):
        got = PL.layernorm(x, gamma, beta, amax=amax1, stream=s)
        grads = PL.layernorm_grad(dy, x, gamma, mean, rstd, stream=s)
        side.synchronize()
        assert torch.equal(got[0], y) and torch.equal(amax0, amax1)
        for a, b in zip(grads, want):
            assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gy, gm, gr = PL.layernorm(x, gamma, beta, amax=amax1)
        gg = PL.layernorm_grad(dy, x, gamma, gm, gr)
    for k in range(3):
        x.copy_(x.flip(0))
        dy.copy_(dy * 0.5)
        y, mean, rstd = PL.layernorm(x, gamma, beta, amax=amax0)
        want = PL.layernorm_grad(dy, x, gamma, mean, rstd)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(gy, y) and torch.equal(amax0, amax1), k
        for a, b in zip(gg, want):
            assert torch.equal(a, b), k


def test_norm_feeds_the_quantizer():
    """The norm's own maximum in place of the quantizer's pass: the same codes and scale, for both copies' recipes."""
    x, gamma, beta, _ = (t.cuda() for t in make(256, 512, BF, BF, BF, seed=4))
    amax = torch.empty(1, device="cuda")
    y, _, _ = PL.layernorm(x, gamma, beta, amax=amax)
    for recipe in ("fp8_current", "nvfp4"):
        a = PL.quantize(recipe, y, "x", "row", "fprop")
        b = PL.quantize(recipe, y, "x", "row", "fprop", known_amax=amax)
        assert torch.equal(a.codes, b.codes) and torch.equal(a.tensor_scale_inv, b.tensor_scale_inv)
