"""Newton-Schulz orthogonalisation and Muon's update on the GPU against the formulas in 64 bits."""
import pytest
import torch

import precision_block_scaled_amd as P
from precision_block_scaled_amd import pipeline as PL
from tests.muon_ref import STEP, assert_near, one_step_bound, orthogonal
from tests.norm_ref import assert_within, half_step

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
# single rows and values, sides around 16, 32, 64 and every tile, either side the longer, long and short contractions
SHAPES = [(1, 1), (1, 70), (5, 3), (16, 16), (17, 200), (33, 64), (64, 64), (64, 65), (65, 64), (100, 31), (128, 128),
          (129, 400), (400, 129), (192, 192), (193, 385), (256, 256), (257, 257), (300, 1000), (520, 320), (640, 640), (700, 520),
          (24, 5000), (3000, 60), (1100, 1030)]


def matrix(r, c, kind="low", seed=0, dtype=F32):
    """Noise alone, or a few directions that stand 10 or 300 times out of it."""
    g = torch.Generator().manual_seed(seed + 7 * r + c)
    x = torch.randn(r, c, generator=g)
    if kind != "noise":
        k = min(4, r, c)
        u, v = torch.randn(r, k, generator=g), torch.randn(k, c, generator=g)
        x = x * (0.1 if kind == "low" else 0.003) + (u * 0.5 ** torch.arange(k)) @ v
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("r,c", SHAPES)
def test_one_step(r, c, dtype):
    """Every element within the bound that the formats' half steps give."""
    x = matrix(r, c, dtype=dtype)
    got = PL.orthogonalize(x.cuda(), coefficients=(STEP,))
    assert got.dtype == BF and got.shape == x.shape
    want, e = one_step_bound(x.double(), STEP)
    assert_within(got, want, e + half_step(BF) * (want.abs() + e), f"{r}x{c}")


@pytest.mark.parametrize("kind", ["noise", "low", "lower"])
@pytest.mark.parametrize("r,c", SHAPES)
def test_five_steps(r, c, kind):
    x = matrix(r, c, kind)
    got = PL.orthogonalize(x.cuda())
    assert_near(got.cpu(), x, PL.MUON_STEPS, what=f"{r}x{c} {kind}")
    assert torch.equal(got, PL.orthogonalize(x.cuda()))


@pytest.mark.parametrize("steps", [((1.5, -0.5, 0.0),) * 12, ((3.4445, -4.7750, 2.0315),) * 2 + ((1.875, -1.25, 0.375),) * 3,
                                   ((2.0, 0.0, 0.0),), ((0.5, 0.25, -0.125),) * 3, ((8.0, -20.0, 13.0),) * 2])
@pytest.mark.parametrize("r,c", [(48, 100), (200, 130), (300, 300)])
def test_other_steps(steps, r, c):
    """Other polynomials and numbers of steps, one step after the other of different kinds, larger ranges of values."""
    x = matrix(r, c)
    got = PL.orthogonalize(x.cuda(), coefficients=steps)
    # the scale that the call documents: the largest power of two that holds X, A and P with a third to spare
    top, most = 1.0, 1.0
    for a, b, c_ in steps:
        s = torch.linspace(0, top, 100001, dtype=torch.float64)
        poly, nxt = (s ** 2 * (b + c_ * s ** 2)).abs().max().item(), (s * (a + b * s ** 2 + c_ * s ** 4)).abs().max().item()
        most, top = max(most, top ** 2, poly, nxt), nxt
    scale = 2.0 ** 14
    while scale * most * 1.02 > 49152:
        scale /= 2
    assert_near(got.cpu(), x, steps, scale=scale, what=str(steps))


@pytest.mark.parametrize("power", [-38, -20, 20, 37])
@pytest.mark.parametrize("r,c", [(40, 90), (300, 200)])
def test_magnitudes(power, r, c):
    """Values whose squares fp32 does not hold."""
    x = matrix(r, c) * 10.0 ** power
    got = PL.orthogonalize(x.cuda(), eps=0.0)
    assert_near(got.cpu(), x.double() * 10.0 ** -power, PL.MUON_STEPS, eps=0.0, what=str(power))


@pytest.mark.parametrize("r,c", [(20, 50), (64, 64), (130, 200), (300, 130)])
def test_matrices_of_a_batch_stay_apart(r, c):
    x = torch.stack([matrix(r, c, seed=s) for s in range(5)])
    want = PL.orthogonalize(x.cuda())
    for i in range(5):
        assert torch.equal(PL.orthogonalize(x[i].cuda()), want[i])
    for bad in (float("nan"), float("inf")):
        y = x.clone()
        y[1, r - 1, c // 2] = bad
        y[3] = 0
        got = PL.orthogonalize(y.cuda())
        for i in (0, 2, 4):
            assert torch.equal(got[i], want[i])
        assert got[1].isnan().all() and (got[3] == 0).all()
        assert (PL.orthogonalize(y[3].cuda(), eps=0.0) == 0).all()


def update_ref(w, m, g, lr, beta, nesterov, decay, scale, steps):
    m = beta * m.double() + (1 - beta) * g.double()
    u = beta * m + (1 - beta) * g.double() if nesterov else m
    return (1 - lr * decay) * w.double() - lr * scale * orthogonal(u, steps), m, u


@pytest.mark.parametrize("types", [(BF, F32, BF), (F32, F32, F32), (F32, BF, BF), (BF, BF, F32)],
                         ids=lambda t: "-".join(str(d)[6:] for d in t))
@pytest.mark.parametrize("turned", [False, True])
@pytest.mark.parametrize("r,c", [(40, 90), (64, 64), (90, 40), (300, 200), (200, 300), (257, 129), (1, 9)])
def test_muon(r, c, turned, types):
    tg, tm, tw = types
    g0 = torch.Generator().manual_seed(r + c)
    w = (0.02 * torch.randn(2, r, c, generator=g0)).to(tw)
    m = torch.stack([matrix(r, c, seed=1), matrix(r, c, "noise", seed=2)]).to(tm)
    g = torch.stack([matrix(r, c, seed=3), matrix(r, c, seed=4)]).to(tg)
    for nesterov, decay, scale in ((True, 0.1, None), (False, 0.0, 0.7)):
        cw, cm = w.cuda(), m.cuda()
        cg = g.cuda().transpose(1, 2).contiguous().transpose(1, 2) if turned else g.cuda()
        out = PL.muon(cw, cm, cg, 0.02, beta=0.9, nesterov=nesterov, weight_decay=decay, scale=scale)
        assert out is cw
        s = max(1.0, r / c) ** 0.5 if scale is None else scale
        for i in range(2):
            want, wm, u = update_ref(w[i], m[i], g[i], 0.02, 0.9, nesterov, decay, s, PL.MUON_STEPS)
            # beta and 1 - beta are fp32: 2^-24 of each term, and the products' and sums' roundings
            assert_within(cm[i], wm, half_step(tm) * wm.abs() + 4 * 2.0 ** -24 * (0.9 * m[i].double().abs() + 0.1 * g[i].double().abs()) *
                          (1 + half_step(tm)), "momentum")
            # X from the weight: beside X's own error the weight's rounding and arithmetic over lr scale, and U's fp32
            # roundings: 4 of them beside a norm of 1, which grow by at most the steps' largest slopes, 3.9 each, 902 in
            # all.  (Not held to another run of nearly the same U: whose A and P round otherwise, so that the two runs'
            # errors add.)
            ours = (w[i].double() * (1 - 0.02 * decay) - cw[i].cpu().double()) / (0.02 * s)
            slack = (half_step(tw) * want.abs() + 6 * 2.0 ** -24 * w[i].double().abs()) / (0.02 * s) + 902 * 4 * 2.0 ** -24
            assert_near(ours, u, PL.MUON_STEPS, slack=slack, what=f"{i} {nesterov}")


@pytest.mark.parametrize("r,c,skip,pad", [(40, 90, 0, 0), (40, 90, 3, 5), (90, 41, 1, 2), (260, 200, 2, 3), (130, 300, 1, 1), (64, 64, 4, 4)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_strides_and_places(r, c, skip, pad, dtype):
    """Rows and matrices at any element and any stride, matrices between each other's rows; what lies beside them stays."""
    w, m, g = ((s * torch.stack([matrix(r, c, seed=i + k) for i in range(3)])).to(dtype) for k, s in ((0, 0.02), (10, 1.0), (20, 1.0)))
    want = [t.cuda() for t in (w, m)]
    PL.muon(*want, g.cuda(), 0.02)

    def rows(t):
        flat = torch.full((skip + 3 * r * (c + pad) + 8,), 77.0, dtype=dtype, device="cuda")
        v = flat[skip:skip + 3 * r * (c + pad)].view(3, r, c + pad)[:, :, :c]
        v.copy_(t)
        return flat, v

    def between(t):
        flat = torch.full((skip + 3 * r * (c + pad) + 8,), 77.0, dtype=dtype, device="cuda")
        v = flat[skip:skip + 3 * r * (c + pad)].view(r, 3, c + pad)[:, :, :c].transpose(0, 1)
        v.copy_(t)
        return flat, v

    for lay_w, lay_m in ((rows, between), (between, rows)):
        (fw, vw), (fm, vm), (_, vg) = lay_w(w), lay_m(m), lay_w(g)
        PL.muon(vw, vm, vg, 0.02)
        assert torch.equal(vw, want[0]) and torch.equal(vm, want[1])
        for flat in (fw, fm):
            assert (flat[:skip] == 77).all() and (flat[-8:] == 77).all()
            if pad:
                assert (flat[skip:-8].view(-1, c + pad)[:, c:] == 77).all()
    # x in place, and another place
    x = (g * 1.0).to(BF)
    y = PL.orthogonalize(x.cuda())
    a = x.cuda()
    PL.orthogonalize(a, y=a)
    assert torch.equal(a, y)
    flat, v = (torch.full((3 * r * (c + pad) + skip,), 5.0, dtype=BF, device="cuda"), None)
    v = flat[skip:].view(r, 3, c + pad)[:, :, :c].transpose(0, 1)
    PL.orthogonalize(x.cuda(), y=v)
    assert torch.equal(v, y)


def test_empty_and_trivial():
    for shape in ((0, 5), (5, 0), (0, 4, 4), (2, 0, 3)):
        x = torch.empty(shape, device="cuda")
        assert PL.orthogonalize(x).shape == x.shape
        PL.muon(torch.empty_like(x), torch.empty_like(x), x, 0.1)
    # beta 1: the gradient has no part; lr 0: the weight stays to the bit
    w, m, g = (torch.randn(70, 80, device="cuda") for _ in range(3))
    w0, m0 = w.clone(), m.clone()
    PL.muon(w, m, g, 0.0, beta=1.0)
    assert torch.equal(w, w0) and torch.equal(m, m0)


@pytest.mark.parametrize("r,c", [(48, 200), (300, 200)])
def test_streams_graph_and_factor(r, c):
    w, m, g = (torch.stack([matrix(r, c, seed=i + k) for i in range(2)]).cuda() for k in (0, 10, 20))
    lr = torch.full((1,), 0.02, device="cuda")
    want_w, want_m = w.clone(), m.clone()
    history = []
    for f in (0.02, 0.01, 0.0, 0.05):
        PL.muon(want_w, want_m, g, f, weight_decay=0.1)
        history.append((want_w.clone(), want_m.clone()))
    side = torch.cuda.Stream()
    a, b = w.clone(), m.clone()
    side.wait_stream(torch.cuda.current_stream())
    PL.muon(a, b, g, lr, weight_decay=0.1, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(a, history[0][0]) and torch.equal(b, history[0][1])
    a, b = w.clone(), m.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        PL.muon(a, b, g, lr, weight_decay=0.1)
    for f, (x, y) in zip((0.02, 0.01, 0.0, 0.05), history):
        lr.fill_(f)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, x) and torch.equal(b, y), f
        _ = PL.orthogonalize(g)                          # eager work between the replays


def test_two_calls_at_once():
    xs = [matrix(700, 500, seed=s).cuda() for s in range(4)]
    want = [PL.orthogonalize(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [PL.orthogonalize(x, stream=s) for x, s in zip(xs, streams)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """Matrices whose places lie past 2^31 values."""
    stride = (1 << 30) + 8
    flat = torch.empty(2 * stride + 4096, dtype=BF, device="cuda")
    w = flat.as_strided((3, 40, 60), (stride, 60, 1))
    x = torch.stack([matrix(40, 60, seed=s) for s in range(3)]).to(BF)
    w.copy_(x)
    want = PL.orthogonalize(x.cuda())
    PL.orthogonalize(w, y=w)
    assert torch.equal(w, want)


def test_large_square():
    """A benchmark-sized matrix against 64 bits on the GPU: the result's own rounding and a third more."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x = 0.1 * torch.randn(2048, 4096, device="cuda", generator=g) + torch.randn(2048, 6, device="cuda", generator=g) @ torch.randn(
        6, 4096, device="cuda", generator=g)
    for t in (x, x.t().contiguous()):
        got, want = PL.orthogonalize(t), orthogonal(t, PL.MUON_STEPS)
        # bf16's rounding: at most 2^-8, and uniform within a step 2^-9 / sqrt(3) times 1.5 on average over a binade
        assert ((got.double() - want).norm() / want.norm()).item() < 2.0 ** -9


@pytest.mark.parametrize("kind", ["noise", "low", "lower"])
@pytest.mark.parametrize("r,c", [(130, 1900), (200, 12000), (2100, 300), (1024, 4096), (4500, 1100), (1030, 2100)])
def test_long_sides(r, c, kind):
    """Sides of which the longer is several times the shorter, where steps are taken together: 64 bits on the GPU, within
    the documented 0.2% and bf16's own rounding (0.17%)."""
    x = matrix(r, c, kind).cuda()
    for steps in (PL.MUON_STEPS, PL.MUON_STEPS[:2], PL.MUON_STEPS + PL.MUON_STEPS[:2]):
        got, want = PL.orthogonalize(x, coefficients=steps), orthogonal(x, steps)
        off = (got.double() - want).norm() / want.norm()
        assert off.item() < (0.002 ** 2 + 0.0018 ** 2) ** 0.5, (len(steps), off.item())
        assert torch.equal(got, PL.orthogonalize(x, coefficients=steps))
    b = torch.stack([x, 2 * x])
    got = PL.orthogonalize(b, coefficients=PL.MUON_STEPS[:2], eps=0.0)
    assert torch.equal(got[0], got[1])


def test_a_step_around_the_projection():
    """QKV product, norm and rotation, attention, their gradients with the maximum, the quantized products, the update."""
    torch.manual_seed(0)
    B, S, H, D, C = 2, 64, 4, 64, 256
    x = torch.randn(B * S, C, device="cuda").to(BF)
    w = (0.05 * torch.randn(3 * H * D, C, device="cuda")).to(BF)
    qw, kw = (1 + 0.1 * torch.randn(2, D, device="cuda")).unbind()
    f = PL.rope_frequencies(D)
    M, N, K = PL.pass_dims("fprop", B * S, C, 3 * H * D)
    A, Bq = PL.quantize_pass("fp8_current", "fprop", x, w, None)
    qkv = PL.gemm("fp8_current", "fprop", A, Bq, M, N, K).view(B, S, 3 * H, D)
    q, k, v = qkv.split(H, 2)
    yq, yk = PL.qk_norm_rope(q, k, qw, kw, None, f)
    leaves = [t.float().transpose(1, 2).contiguous().requires_grad_() for t in (yq, yk, v)]
    prob = (torch.matmul(leaves[0], leaves[1].transpose(2, 3).contiguous()) * D ** -0.5).softmax(-1)
    out = torch.matmul(prob, leaves[2])
    dq, dk, dv = (t.to(BF).contiguous().transpose(1, 2) for t in torch.autograd.grad(out.square().sum(), leaves))
    d = torch.empty_like(qkv)
    parts, amax = d.split(H, 2), torch.empty(1, device="cuda")
    _, _, dqw, dkw = PL.qk_norm_rope_grad(dq, dk, q, k, qw, kw, None, f, dv=dv, dq_out=parts[0], dk_out=parts[1],
                                          dv_out=parts[2], amax=amax)
    assert amax.item() == d.float().abs().max().item()
    dy = d.view(B * S, 3 * H * D)
    # the cast with the handed maximum is the cast that takes its own
    a = PL.quantize("fp8_current", dy, "dy", "col", "wgrad", known_amax=amax)
    b = PL.quantize("fp8_current", dy, "dy", "col", "wgrad")
    assert torch.equal(a.codes, b.codes) and torch.equal(a.tensor_scale_inv, b.tensor_scale_inv)
    xa = PL.quantize("fp8_current", x, "x", "col", "wgrad")
    M, N, K = PL.pass_dims("wgrad", B * S, C, 3 * H * D)
    dw = PL.gemm("fp8_current", "wgrad", xa, a, M, N, K, out_dtype=F32)              # [in, out]
    # the three projections each by themselves
    momentum = torch.zeros(3, H * D, C, device="cuda")
    before = w.clone()
    PL.muon(w.view(3, H * D, C), momentum, dw.t().unflatten(0, (3, H * D)), 0.02)
    assert torch.allclose(momentum.view(-1, C), 0.05 * dw.t(), rtol=1e-6)
    for i in range(3):
        moved = (before.view(3, -1, C)[i].double() - w.view(3, -1, C)[i].double()) / 0.02
        u = dw.t().reshape(3, -1, C)[i].cpu()
        want = orthogonal(u, PL.MUON_STEPS)
        # the weight's rounding, half a step of values up to 0.3, over lr; and the orthogonalisation's own error
        assert (moved.cpu() - want).abs().max() <= 2.0 ** -9 * w.float().abs().max().item() * 2 / 0.02 + 0.01
    assert dqw.isfinite().all() and dkw.isfinite().all()


@pytest.mark.parametrize("r,c,ld", [(300, 200, 1 << 21), (200, 300, (1 << 23) - 4), (130, 100, (1 << 25) + 4), (100, 130, (1 << 25) + 1)])
def test_rows_far_apart(r, c, ld):
    """Weight, momentum and gradient whose rows lie megabytes apart, up to 2^32 bytes and more from the first."""
    w, m, g = (matrix(r, c, seed=s).to(BF) for s in (1, 2, 3))
    want_w, want_m = w.cuda(), m.cuda()
    PL.muon(want_w, want_m, g.cuda(), 0.02)
    flat = torch.empty((r - 1) * ld + 3 * c + 8, dtype=BF, device="cuda")
    views = [flat[i * (c + 4):].as_strided((r, c), (ld, 1)) for i in range(3)]
    for v, t in zip(views, (w, m, g)):
        v.copy_(t)
    PL.muon(*views, 0.02)
    assert torch.equal(views[0], want_w) and torch.equal(views[1], want_m) and torch.equal(views[2].cpu(), g)


def test_largest_batch():
    """65535 matrices, each by itself."""
    g = torch.Generator().manual_seed(1)
    x = torch.randn(65535, 3, 5, generator=g)
    got = PL.orthogonalize(x.cuda())
    want = x.double() / (x.double().flatten(1).norm(dim=1)[:, None, None] + 1e-7)
    for a, b, c in PL.MUON_STEPS:
        r = want @ want.transpose(1, 2).contiguous()
        want = a * want + (b * r + c * r @ r) @ want
    # bf16's half step, and fp32 roundings of short sums
    assert ((got.cpu().double() - want).abs() <= half_step(BF) * want.abs() + 1e-5).all()
    for i in (0, 65534):
        assert torch.equal(PL.orthogonalize(x[i].cuda()), got[i])


# around the largest matrix whose steps run in one launch, and short sides of every block count beyond it
EDGES = [(64, 256), (256, 64), (64, 257), (257, 64), (40, 129), (191, 7), (192, 64), (2, 255), (16, 300), (17, 600), (33, 300),
         (64, 640), (600, 50), (2, 700), (300, 32)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("r,c", EDGES)
def test_one_step_of_small_matrices(r, c, dtype):
    test_one_step(r, c, dtype)


@pytest.mark.parametrize("kind", ["noise", "low", "lower"])
@pytest.mark.parametrize("r,c", EDGES)
def test_five_steps_of_small_matrices(r, c, kind):
    test_five_steps(r, c, kind)


@pytest.mark.parametrize("turned", [False, True])
@pytest.mark.parametrize("r,c", [(64, 256), (255, 33), (50, 300), (300, 64), (20, 20)])
def test_muon_of_small_matrices(r, c, turned):
    """fp32 throughout: the update to a few fp32 roundings of the steps' slopes, where bf16's store hides nothing."""
    g0 = torch.Generator().manual_seed(r * c)
    w, m, g = (torch.randn(3, r, c, generator=g0) for _ in range(3))
    cw, cm = w.cuda(), m.cuda()
    cg = g.cuda().transpose(1, 2).contiguous().transpose(1, 2) if turned else g.cuda()
    PL.muon(cw, cm, cg, 1.0, weight_decay=0.5, scale=1.0)
    for i in range(3):
        want, _, u = update_ref(w[i], m[i], g[i], 1.0, 0.95, True, 0.5, 1.0, PL.MUON_STEPS)
        x = orthogonal(u, PL.MUON_STEPS)
        # fp16 pairs, 2^-22 of a value, in U, A, P and X of five steps, which grow by the steps' largest slopes: at most
        # 3.9 each, 902 in all; beside them the weight's fp32 roundings
        off = (cw[i].cpu().double() - want).norm()
        assert off <= 20 * 902 * 2.0 ** -22 * x.norm() + 4 * 2.0 ** -24 * w[i].double().norm(), (off / x.norm()).item()
