"""Orthogonalisation over many steps and of matrices without full rank, on the GPU against the formulas in 64 bits."""
import pytest
import torch

import precision_block_scaled_amd as P
from precision_block_scaled_amd import pipeline as PL
from tests.muon_ref import emulated, emulated_gram, emulated_pairs, orthogonal
from tests.test_gpu_muon import matrix
from tests.test_muon_coefficients import RISING, within

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
# (coefficients are fp32: the references take them as the calls do)
MUON, CUBIC, QUINTIC = ((tuple(torch.tensor(s).tolist()),) for s in (PL.MUON_STEPS[0], (1.5, -0.5, 0.0), (1.875, -1.25, 0.375)))


def fp32_x(x, steps, eps=1e-7):
    """The last X in fp32: a weight of zeros moved by -1 times it."""
    x = x.cuda()
    w, m = torch.zeros(x.shape, device="cuda"), torch.zeros(x.shape, device="cuda")
    PL.muon(w, m, x, 1.0, beta=0.0, scale=-1.0, coefficients=steps, eps=eps)
    return w


def by_values(x, steps, rank, eps=1e-7):
    """X from the `rank` singular values of x that are not 0, which the steps' polynomials take each by itself."""
    u, s, v = torch.linalg.svd(x.double().cpu(), full_matrices=False)
    assert rank == len(s) or s[rank] < 1e-12 * s[0] < 1e-6 * s[rank - 1]
    u, s, v = u[:, :rank], s[:rank] / (x.double().norm().cpu() + eps), v[:rank]
    for a, b, c in steps:
        s = s * (a + b * s ** 2 + c * s ** 4)
    return (u * s) @ v


def low_rank(r, c, kind, seed=0):
    """Matrices whose entries are small whole numbers, so that their rank is exact in every type; (matrix, rank)."""
    g = torch.Generator().manual_seed(seed + r + 3 * c)
    if kind == "ones":
        return torch.ones(r, c), 1
    k = {"one": 1, "four": min(4, r, c)}[kind]
    u, v = torch.randint(1, 4, (r, k), generator=g).float(), torch.randint(-3, 4, (k, c), generator=g).float()
    u[:, 1:] *= torch.randint(0, 2, (r, k - 1), generator=g) * 2 - 1
    x = u @ v
    return x, int(torch.linalg.matrix_rank(x.double()))


def largest_gain(x, steps, rank, eps=1e-7):
    """The most that an error of a step grows by until the last one, among x's values that are not 0."""
    s = torch.linalg.svdvals(x.double())[:rank] / (x.double().norm() + eps)
    gain, most = torch.ones_like(s), 1.0
    for a, b, c in steps:
        gain = (gain * (a + 3 * b * s ** 2 + 5 * c * s ** 4).abs()).clamp(min=1.0)
        s = s * (a + b * s ** 2 + c * s ** 4)
        most = max(most, gain.max().item())
    return most


def growth(steps):
    """What a direction that x does not have grows by."""
    g = 1.0
    for a, _, _ in steps:
        g *= a
    return g


# every number of 16-row blocks, either side the longer
SHORT = [(16, 300), (5, 3), (1, 700), (24, 5000), (300, 32), (33, 300), (600, 50), (64, 1000)]


@pytest.mark.parametrize("kind", ["ones", "one", "four"])
@pytest.mark.parametrize("steps", [MUON * 5, MUON * 7, MUON * 9, MUON * 10, MUON * 16, CUBIC * 48, QUINTIC * 32, MUON * 4 + CUBIC * 3 + QUINTIC * 8],
                         ids=["muon5", "muon7", "muon9", "muon10", "muon16", "cubic48", "quintic32", "mixed"])
@pytest.mark.parametrize("r,c", SHORT)
def test_ranks_of_short_sides(r, c, steps, kind):
    """A long run of steps on a matrix without full rank is the one that 64 bits make of it."""
    x, rank = low_rank(r, c, kind)
    want, got = by_values(x, steps, rank), fp32_x(x, steps).cpu().double()
    # Directions that x lacks start from what each step's roundings leave there and grow by a a step.  Up to the growth
    # of 2048, the product's Q and its sums are fp32: a few roundings of them, 2^-24 each, growing by all the steps'; the
    # sums of one sign of `ones` add up to as many as the shorter side.  Beyond, all is in 64 bits, sums of m + n
    # values; the store rounds to fp32.
    m = min(r, c)
    noise = growth(steps) * (m * 2.0 ** -24 if growth(steps) <= 2048 else (r + c) * 2.0 ** -53)
    assert noise < 0.002
    off = (got - want).norm() / want.norm()
    assert off <= 2.0 ** -23 + noise, (off.item(), noise)


@pytest.mark.parametrize("steps", [MUON * 64, CUBIC * 64, QUINTIC * 64], ids=["muon", "cubic", "quintic"])
@pytest.mark.parametrize("r,c", [(16, 300), (24, 5000), (600, 50), (64, 1000)])
def test_equal_rows_stay_equal(r, c, steps):
    x = torch.randn(r, c, generator=torch.Generator().manual_seed(r))
    short = x if r <= c else x.t()
    short[1] = short[0]
    short[-2] = 0
    got = fp32_x(x, steps).cpu().double()
    want = by_values(x, steps, min(r, c) - 2)
    rows = got if r <= c else got.t()
    assert torch.equal(rows[0], rows[1]) and (rows[-2] == 0).all()
    # fp32's rounding, and those of sums of r + c values in 64 bits in each step, which grow by its slopes
    each = (r + c) * 2.0 ** -53 * largest_gain(x, steps, min(r, c) - 2)
    assert each < 1e-7
    assert (got - want).norm() <= (2.0 ** -24 + len(steps) * each) * want.norm()


@pytest.mark.parametrize("kind", ["ones", "one", "four"])
@pytest.mark.parametrize("r,c", [(16, 300), (64, 1000), (64, 64), (60, 200), (130, 300), (300, 300), (520, 900), (1100, 1500)])
def test_many_steps_stay_bounded(r, c, kind):
    """Whatever the roundings add, no singular value leaves what the polynomials allow."""
    x, _ = low_rank(r, c, kind)
    for steps, top in ((MUON * 64, 1.2025), (CUBIC * 64, 1.0), (QUINTIC * 64, 1.0)):
        for got in (PL.orthogonalize(x.cuda(), coefficients=steps), fp32_x(x, steps)):
            assert got.isfinite().all()
            # the largest value of the steps' polynomials on what they make of [0, 1]; 1% for the formats
            y = got.double().cpu() if r <= c else got.double().cpu().t()
            assert torch.linalg.eigvalsh(y @ y.t())[-1].sqrt() <= 1.01 * top, (len(steps), top)


def whole(shape, low, high, g):
    return torch.randint(low, high + 1, shape, generator=g).float()


@pytest.mark.parametrize("types", [(BF, F32, BF), (F32, F32, F32), (F32, BF, BF), (BF, BF, F32)],
                         ids=lambda t: "-".join(str(d)[6:] for d in t))
@pytest.mark.parametrize("turned", [False, True])
@pytest.mark.parametrize("nesterov", [False, True])
@pytest.mark.parametrize("steps", [MUON * 5, MUON * 8, QUINTIC * 20], ids=["muon5", "muon8", "quintic20"])
@pytest.mark.parametrize("r,c", [(16, 300), (300, 20), (40, 600), (900, 64), (3, 5)])
def test_update_of_short_sides(r, c, steps, nesterov, turned, types):
    """Momentum, gradient and their mean are whole multiples of 1/4 and no rounding touches them: the weight's own rounding
    is all that its formula leaves, beside X's error."""
    tg, tm, tw = types
    rnd = torch.Generator().manual_seed(r + c)
    m, g, w = (whole((2, r, c), -8, 8, rnd) for _ in range(3))
    cw, cm, cg = (0.25 * w).to(tw).cuda(), m.to(tm).cuda(), g.to(tg).cuda()
    if turned:
        cg = cg.transpose(1, 2).contiguous().transpose(1, 2)
    lr = torch.full((1,), 0.5, device="cuda")
    PL.muon(cw, cm, cg, lr, beta=0.5, nesterov=nesterov, weight_decay=0.5, scale=0.5, coefficients=steps)
    m1 = 0.5 * m + 0.5 * g
    assert torch.equal(cm.cpu().float(), m1.to(tm).float())
    for i in range(2):
        u = 0.5 * m1[i] + 0.5 * g[i] if nesterov else m1[i]
        x = orthogonal(u, steps)
        want = 0.75 * 0.25 * w[i].double() - 0.25 * x
        # X: fp32 roundings of Q U, at most 485 of them beside X's norm; the weight: three fp32 roundings and its store's
        half = torch.finfo(tw).eps / 2
        off = (cw[i].cpu().double() - want).norm()
        assert off <= (half + 3 * 2.0 ** -24) * (want.norm() + 0.25 * x.norm()) + 0.25 * 485 * 2.0 ** -24 * x.norm()


@pytest.mark.parametrize("steps", [MUON * 5, MUON * 8, MUON * 10], ids=["muon5", "muon8", "muon10"])
@pytest.mark.parametrize("r,c,skip,pad", [(16, 300, 0, 0), (30, 261, 3, 5), (300, 41, 1, 2), (64, 270, 2, 3), (7, 20, 1, 1)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_short_sides_where_they_lie(r, c, skip, pad, dtype, steps):
    """Rows and matrices at any element and stride, in place, in a captured graph with a learning rate from the device."""
    rnd = torch.Generator().manual_seed(r * c)
    w, m, g = ((s * torch.randn(3, r, c, generator=rnd)).to(dtype) for s in (0.02, 1.0, 1.0))
    want_w, want_m = w.cuda(), m.cuda()
    PL.muon(want_w, want_m, g.cuda(), 0.02, coefficients=steps)

    def between(t):
        flat = torch.full((skip + 3 * r * (c + pad) + 8,), 77.0, dtype=dtype, device="cuda")
        v = flat[skip:skip + 3 * r * (c + pad)].view(r, 3, c + pad)[:, :, :c].transpose(0, 1)
        v.copy_(t)
        return flat, v

    (fw, vw), (fm, vm), (_, vg) = between(w), between(m), between(g)
    PL.muon(vw, vm, vg, 0.02, coefficients=steps)
    assert torch.equal(vw, want_w) and torch.equal(vm, want_m)
    for flat in (fw, fm):
        assert (flat[:skip] == 77).all() and (flat[-8:] == 77).all()
        assert not pad or (flat[skip:-8].view(-1, c + pad)[:, c:] == 77).all()
    x = g.to(BF).cuda()
    y = PL.orthogonalize(x, coefficients=steps)
    a = x.clone()
    PL.orthogonalize(a, y=a, coefficients=steps)
    assert torch.equal(a, y)
    for i in range(3):
        assert torch.equal(PL.orthogonalize(x[i], coefficients=steps), y[i])
    bad = x.clone()
    bad[1, r - 1, c // 2] = float("nan")
    bad[2] = 0
    got = PL.orthogonalize(bad, coefficients=steps, eps=0.0)
    assert torch.equal(got[0], PL.orthogonalize(x[0], coefficients=steps, eps=0.0)) and got[1].isnan().all() and (got[2] == 0).all()
    lr = torch.full((1,), 0.02, device="cuda")
    a, b = w.cuda(), m.cuda()
    cg = g.cuda()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        PL.muon(a, b, cg, lr, coefficients=steps)
    want_w, want_m = w.cuda(), m.cuda()
    for f in (0.02, 0.0, 0.05):
        lr.fill_(f)
        PL.muon(want_w, want_m, cg, f, coefficients=steps)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, want_w) and torch.equal(b, want_m), f
        _ = PL.orthogonalize(x, coefficients=steps)


@pytest.mark.parametrize("steps", [MUON * 5, MUON * 8, MUON * 10], ids=["muon5", "muon8", "muon10"])
@pytest.mark.parametrize("power", [-38, -20, 20, 37])
@pytest.mark.parametrize("r,c", [(16, 300), (300, 64)])
def test_magnitudes_of_short_sides(r, c, power, steps):
    """Values whose squares fp32 does not hold."""
    x = torch.randn(r, c, generator=torch.Generator().manual_seed(7)) * 10.0 ** power
    got, want = fp32_x(x, steps, eps=0.0).cpu().double(), orthogonal(x.double() * 10.0 ** -power, steps, eps=0.0)
    assert (got - want).norm() <= 485 * 2.0 ** -24 * want.norm()


def coherent(r, c, kind, dtype):
    """A direction that stands far out of the noise of the rest: a constant, or a random one."""
    g = torch.Generator(device="cuda").manual_seed(r + c)
    z = torch.randn(r, c, device="cuda", generator=g)
    if kind == "direction":
        x = z + 3000 * torch.randn(r, 1, device="cuda", generator=g) @ torch.randn(1, c, device="cuda", generator=g)
    else:
        x = 1 + float(kind) * z
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", ["1e-1", "1e-2", "1e-3", "1e-4", "direction"])
@pytest.mark.parametrize("r,c", [(1024, 2048), (4500, 1100), (1024, 4096), (520, 1300), (1024, 1024), (130, 1900), (64, 200), (64, 300)])
def test_one_direction_far_out(r, c, kind, dtype):
    """Documented: 0.2% of the result where the largest direction is up to a few hundred times the others, 1% beyond."""
    x = coherent(r, c, kind, dtype)
    got, want = fp32_x(x, MUON * 5).double(), orthogonal(x, MUON * 5)
    off = ((got - want).norm() / want.norm()).item()
    assert off <= (0.002 if kind in ("1e-1", "1e-2") else 0.01), off


def mixed(*names):
    """Steps of which no two in a row are alike; d's growth keeps it, and the steps beside it, by themselves."""
    steps = dict(a=(3.4445, -4.7750, 2.0315), b=(1.875, -1.25, 0.375), c=(1.5, -0.5, 0.0), d=(4.3, -7.0, 3.7), e=(3.0, -3.6, 1.6),
                 f=(2.5, -2.5, 1.0))
    return tuple(tuple(torch.tensor(steps[n]).tolist()) for n in names)


@pytest.mark.parametrize("names", ["ae", "eaf", "aebf", "feacb", "bcaefb", "aebfcd", "bdcacd", "fcabeba", "facbacb"])
@pytest.mark.parametrize("shape", [(1024, 4096), (768, 2304), (3000, 700), (2, 640, 1500), (130, 400), (700, 700), (64, 256), (40, 90),
                                   (16, 300), (33, 300), (600, 50), (2, 24, 700)], ids=str)
def test_schedules(shape, names):
    """Steps that differ, by every path: in pairs, one by one, of the small kernel and of the Gram matrix."""
    steps = mixed(*names)
    r, c = shape[-2:]
    g = torch.Generator(device="cuda").manual_seed(r + c)
    x = torch.randn(shape, device="cuda", generator=g)
    x = 0.1 * x + torch.randn(*shape[:-1], 4, device="cuda", generator=g) @ torch.randn(*shape[:-2], 4, c, device="cuda", generator=g)
    got = fp32_x(x, steps).double()
    for y, z in zip(*(t.reshape(-1, r, c) for t in (got, x))):
        want = orthogonal(z, steps)
        off = ((y - want).norm() / want.norm()).item()
        # documented; and where X is held with 22 bits or more throughout, its roundings and those of short sums in fp32,
        # a few 2^-22 that grow with the steps
        assert off <= (0.002 if min(r, c) > 64 else 8 * growth(steps) * 2.0 ** -22), off


@pytest.mark.parametrize("kind", ["noise", "low"])
@pytest.mark.parametrize("r,c", [(130, 300), (300, 300), (1024, 2100), (4500, 1100), (64, 200), (16, 300), (1000, 64)])
def test_polynomials_of_a_shrinking_range(r, c, kind):
    """Steps that begin steeply, a = 8.2: all else as documented of Muon's."""
    steps = tuple(tuple(torch.tensor(s).tolist()) for s in within(RISING))
    x = matrix(r, c, kind).cuda()
    got, want = fp32_x(x, steps).double(), orthogonal(x, steps)
    assert ((got - want).norm() / want.norm()).item() <= 0.002


@pytest.mark.parametrize("steps", [MUON * 5, MUON * 8, MUON * 12], ids=["muon5", "muon8", "muon12"])
@pytest.mark.parametrize("shape", [(3, 5), (7, 3, 5), (5, 16, 300), (2, 40, 700), (3, 600, 64), (3, 64, 64), (2, 33, 256), (2, 65, 100),
                                   (1, 520, 700), (2, 1100, 640)], ids=str)
def test_workspace_ends_where_it_says(shape, steps):
    """No byte behind the workspace is written, and what it held before has no part in the result."""
    b, (r, c) = shape[0] if len(shape) == 3 else 1, shape[-2:]
    x = torch.randn(b, r, c, generator=torch.Generator().manual_seed(r)).cuda()
    n = P.pbs_orthogonalize_bytes(b, r, c)
    got = []
    for fill in (0, 255):
        ws = torch.full((n + (1 << 20),), fill, dtype=torch.uint8, device="cuda")
        y = torch.empty(b, r, c, dtype=BF, device="cuda")
        P.pbs_orthogonalize(x, P.PBS_FMT_F32, c, r * c, b, r, c, steps, 1e-7, y, c, r * c, ws, n)
        assert (ws[n:] == fill).all()
        got.append(y)
    assert torch.equal(*got) and got[0].isfinite().all()


@pytest.mark.parametrize("kind", ["noise", "low", "lower"])
@pytest.mark.parametrize("r,c", [(64, 256), (256, 64), (64, 64), (33, 65), (255, 40), (48, 100), (16, 300), (300, 16), (33, 300), (64, 257),
                                 (600, 50), (5, 3), (24, 5000)])
def test_short_sides_keep_their_bits(r, c, kind):
    """Shorter sides up to 64 are as exact as their formats' emulation, far from what fp16 operands alone would leave."""
    x, steps = matrix(r, c, kind), MUON * 5
    want, got = orthogonal(x, steps), fp32_x(x, steps).cpu().double()
    small = 32 < min(r, c) and max(r, c) <= 256
    rough = emulated_pairs(x, steps) if small else emulated_gram(x, steps)
    # the emulation's roundings fall otherwise than the kernel's; the last one is fp32's
    bound = 4 * (rough - want).norm() + 2.0 ** -24 * want.norm()
    assert (got - want).norm() <= bound, ((got - want).norm() / want.norm(), bound / want.norm())
    if min(r, c) > 16:
        assert (emulated(x, steps) - want).norm() > 10 * bound


@pytest.mark.parametrize("b,r,c,dtype", [(32, 128, 512, F32), (3, 1537, 1001, BF), (1, 4500, 1500, BF), (300, 64, 64, F32), (40, 16, 700, BF)],
                         ids=str)
def test_identical_bytes(b, r, c, dtype):
    """The same inputs again and again, alone, beside a call on another stream, and through a transposed view."""
    x = torch.randn(b, r, c, generator=torch.Generator().manual_seed(b)).to(dtype).cuda()
    other = torch.randn(700, 900, device="cuda")
    w0, m0 = (0.02 * torch.randn(b, r, c, device="cuda")).to(BF), torch.randn(b, r, c, device="cuda")
    turned, side = x.transpose(1, 2).contiguous().transpose(1, 2), torch.cuda.Stream()
    want, first = PL.orthogonalize(x), None
    for i in range(6):
        assert torch.equal(PL.orthogonalize(x), want), i
        side.wait_stream(torch.cuda.current_stream())
        PL.orthogonalize(other, stream=side)
        w, m = w0.clone(), m0.clone()
        PL.muon(w, m, turned if i % 2 else x, 0.02)
        first = first or (w, m)
        assert torch.equal(w, first[0]) and torch.equal(m, first[1]), i
        torch.cuda.synchronize()
