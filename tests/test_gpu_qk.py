"""Norm and rotation of queries and keys, and the gradient, on the GPU against the formulas in 64 bits."""
import pytest
import torch

import precision_block_scaled_amd as P
from precision_block_scaled_amd import pipeline as PL
from tests.norm_ref import assert_within
from tests.qk_ref import forward_ref, grad_ref, strips_of

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
# batch, seq, heads, kv_heads, head_dim, rot: every chunk width and number of lanes a row, rotations of all, part and none
SHAPES = [(1, 1, 1, 1, 128, 128), (2, 3, 4, 2, 64, 64), (1, 17, 9, 3, 128, 64), (3, 5, 7, 7, 96, 96), (2, 9, 5, 1, 80, 40),
          (1, 6, 3, 2, 256, 256), (1, 5, 2, 1, 512, 512), (2, 2, 3, 3, 192, 128), (1, 7, 5, 5, 72, 24), (1, 4, 2, 2, 33, 30),
          (2, 3, 2, 1, 1, 0), (1, 3, 4, 2, 7, 2), (1, 3, 2, 2, 509, 300), (1, 5, 3, 1, 20, 8), (1, 5, 3, 1, 24, 24),
          (1, 3, 70, 1, 128, 128), (5, 67, 8, 2, 16, 16), (2, 5, 2, 2, 128, 0), (1, 5, 2, 2, 132, 132), (1, 2, 2, 1, 300, 8),
          (1, 1500, 4, 4, 128, 128), (7, 300, 3, 1, 65, 64)]
TYPES = [(BF, BF, BF), (F32, F32, F32), (F32, BF, BF), (BF, F32, F32)]


def make(shape, tx, ty, tw, seed=0, far=1000):
    B, S, H, K, D, rot = shape
    g = torch.Generator().manual_seed(seed)
    scale = 1 + 6 * (torch.rand(D, generator=g) < 0.05)

    def normal(n):
        return torch.randn(B, S, n, D, generator=g)

    q, k = (normal(H) * scale).to(tx), (normal(K) * scale).to(tx)
    qw, kw = ((1 + 0.3 * torch.randn(D, generator=g)).to(tw) for _ in range(2))
    dq, dk, dv = normal(H).to(ty), normal(K).to(ty), normal(K).to(ty)
    pos = torch.randint(-far, far + 1, (B, S), generator=g)
    freqs = PL.rope_frequencies(rot, device="cpu") if rot else None
    return q, k, qw, kw, dq, dk, dv, pos, freqs


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def dbl(t):
    return None if t is None else t.double()


def check(got, x, w, pos, freqs, inter, eps, norm, what):
    want, e = forward_ref(x.double(), dbl(w), pos, freqs, inter, eps, norm, got.dtype)
    assert_within(got, want, e, what)


def check_grad(got, gw, dy, x, w, pos, freqs, inter, eps, norm, strips, what):
    want = grad_ref(dy.double(), x.double(), dbl(w), pos, freqs, inter, eps, norm, got.dtype, strips)
    assert_within(got, want[0], want[1], what + " dx")
    if gw is not None:
        assert_within(gw, want[2], want[3], what + " dw")


@pytest.mark.parametrize("types", TYPES, ids=lambda t: "-".join(str(d)[6:] for d in t))
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward_and_gradient(shape, inter, types):
    tx, ty, tw = types
    B, S, H, K, D, rot = shape
    q, k, qw, kw, dq, dk, dv, pos, freqs = make(shape, tx, ty, tw, seed=sum(shape))
    cq, ck, cqw, ckw, cdq, cdk, cdv, cpos, cf = cuda(q, k, qw, kw, dq, dk, dv, pos, freqs)
    yq, yk = PL.qk_norm_rope(cq, ck, cqw, ckw, cpos, cf, inter, 1e-6, out_dtype=ty)
    assert yq.dtype == yk.dtype == ty
    check(yq, q, qw, pos, freqs, inter, 1e-6, True, "q")
    check(yk, k, kw, pos, freqs, inter, 1e-6, True, "k")
    packed = torch.full((B, S, H + 2 * K, D), 7.0, dtype=tx, device="cuda")
    parts = packed.split((H, K, K), 2)
    amax = torch.full((1,), 99.0, device="cuda")
    oq, ok, gqw, gkw = PL.qk_norm_rope_grad(cdq, cdk, cq, ck, cqw, ckw, cpos, cf, inter, 1e-6, dv=cdv, dq_out=parts[0],
                                            dk_out=parts[1], dv_out=parts[2], amax=amax)
    n = B * S
    check_grad(oq, gqw, dq, q, qw, pos, freqs, inter, 1e-6, True, strips_of(n, H, H + 2 * K), "q")
    check_grad(ok, gkw, dk, k, kw, pos, freqs, inter, 1e-6, True, strips_of(n, K, H + 2 * K), "k")
    assert torch.equal(parts[2].cpu(), dv.to(tx))
    assert amax.item() == packed.float().abs().max().item()
    again = PL.qk_norm_rope_grad(cdq, cdk, cq, ck, cqw, ckw, cpos, cf, inter, 1e-6)
    # without the values' part other workgroups share the sums: dx is the same, the sums within their bounds
    assert torch.equal(again[0], oq) and torch.equal(again[1], ok)
    more = PL.qk_norm_rope_grad(cdq, cdk, cq, ck, cqw, ckw, cpos, cf, inter, 1e-6)
    assert all(torch.equal(a, b) for a, b in zip(again, more))


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("weights", [True, False])
def test_without_weights_norm_or_keys(norm, weights):
    shape = (2, 11, 6, 2, 128, 64)
    q, k, qw, kw, dq, dk, _, pos, freqs = make(shape, BF, BF, F32, seed=3)
    if not weights:
        qw = kw = None
    cq, ck, cqw, ckw, cdq, cdk, cf = cuda(q, k, qw, kw, dq, dk, freqs)
    yq, yk = PL.qk_norm_rope(cq, ck, cqw, ckw, None, cf, norm=norm)
    check(yq, q, qw, None, freqs, False, 1e-6, norm, "q")
    check(yk, k, kw, None, freqs, False, 1e-6, norm, "k")
    g = PL.qk_norm_rope_grad(cdq, cdk, cq, ck, cqw, ckw, None, cf, norm=norm)
    check_grad(g[0], g[2], dq, q, qw, None, freqs, False, 1e-6, norm, strips_of(22, 6, 8), "q")
    check_grad(g[1], g[3], dk, k, kw, None, freqs, False, 1e-6, norm, strips_of(22, 2, 8), "k")
    alone, none = PL.qk_norm_rope(cq, None, cqw, None, None, cf, norm=norm)
    assert none is None and torch.equal(alone, yq)
    a = PL.qk_norm_rope_grad(cdq, None, cq, None, cqw, None, None, cf, norm=norm)
    assert torch.equal(a[0], g[0]) and a[1] is None and a[3] is None
    check_grad(a[0], a[2], dq, q, qw, None, freqs, False, 1e-6, norm, strips_of(22, 6, 6), "q alone")
    shared = PL.qk_norm_rope(cq, ck, cqw, ckw, torch.arange(11, device="cuda"), cf, norm=norm)
    assert torch.equal(shared[0], yq) and torch.equal(shared[1], yk)


def test_gradient_against_differences():
    """The formula that the gradient is held to, and through it the gradient, against central differences."""
    torch.manual_seed(1)
    B, S, H, D = 1, 2, 2, 12
    x, w, dy = torch.randn(B, S, H, D).double(), 1 + 0.3 * torch.randn(D).double(), torch.randn(B, S, H, D).double()
    pos, freqs = torch.tensor([[3, -50]]), PL.rope_frequencies(8, device="cpu")

    def loss(x, w):
        return (forward_ref(x, w, pos, freqs, False, 1e-6, True, torch.float64)[0] * dy).sum()

    dx, _, dw, _ = grad_ref(dy, x, w, pos, freqs, False, 1e-6, True, torch.float64, 1)
    for t, d in ((x, dx), (w, dw)):
        flat, est = t.view(-1), torch.empty(t.numel(), dtype=torch.float64)
        for i in range(t.numel()):
            old = flat[i].item()
            flat[i] = old + 1e-5
            up = loss(x, w)
            flat[i] = old - 1e-5
            est[i] = (up - loss(x, w)) / 2e-5
            flat[i] = old
        # a central difference of step h is off by h^2 / 6 times the third derivative, below 10^3 here, and its roundings
        assert (est.view_as(d) - d).abs().max() < 1e-7
    cx, cw, cdy, cp, cf = cuda(x.float(), w.float(), dy.float(), pos, freqs)
    got = PL.qk_norm_rope_grad(cdy, None, cx, None, cw, None, cp, cf)
    check_grad(got[0], got[2], dy.float(), x.float(), w.float(), pos, freqs, False, 1e-6, True, 1, "differences")


@pytest.mark.parametrize("tx", [BF, F32])
@pytest.mark.parametrize("dim,rot,skip", [(128, 128, 0), (128, 64, 1), (80, 40, 4), (96, 96, 2), (13, 12, 3)])
def test_strides_and_places(tx, dim, rot, skip):
    """Parts of a packed projection and heads ahead of positions, at any element; what lies beside them stays."""
    B, S, H, K = 2, 7, 3, 2
    q, k, qw, kw, dq, dk, dv, pos, freqs = make((B, S, H, K, dim, rot), tx, tx, BF, seed=dim)
    cqw, ckw, cpos, cf = cuda(qw, kw, pos, freqs)

    def packed(*ts):
        ld = (H + 2 * K) * dim + 5
        flat = torch.full((B * S * ld + 64,), 123.0, dtype=tx, device="cuda")
        rows = flat[skip:skip + B * S * ld].view(B, S, ld)[:, :, :(H + 2 * K) * dim].unflatten(2, (H + 2 * K, dim))
        parts = rows.split((H, K, K), 2)
        for part, t in zip(parts, ts):
            part.copy_(t)
        return flat, parts

    def first(n, t=None):
        flat = torch.full((B * n * S * dim + 64,), 55.0, dtype=tx, device="cuda")
        view = flat[skip:skip + B * n * S * dim].view(B, n, S, dim).transpose(1, 2)
        if t is not None:
            view.copy_(t)
        return flat, view

    want = PL.qk_norm_rope(q.cuda(), k.cuda(), cqw, ckw, cpos, cf)
    _, (pq, pk, pv) = packed(q, k, dv)
    fq, oq = first(H)
    fk, ok = first(K)
    got = PL.qk_norm_rope(pq, pk, cqw, ckw, cpos, cf, q_out=oq, k_out=ok)
    assert got[0].data_ptr() == oq.data_ptr()
    # other chunks may add a row's squares in another order: held to the formula, and to what lies around
    check(oq, q, qw, pos, freqs, False, 1e-6, True, "q")
    check(ok, k, kw, pos, freqs, False, 1e-6, True, "k")
    check(want[0], q, qw, pos, freqs, False, 1e-6, True, "q contiguous")
    for flat, n in ((fq, H), (fk, K)):
        assert (flat[:skip] == 55).all() and (flat[skip + B * n * S * dim:] == 55).all()
    _, gq = first(H, dq)
    _, gk = first(K, dk)
    _, gv = first(K, dv)
    flat, outs = packed()
    amax = torch.empty(1, device="cuda")
    res = PL.qk_norm_rope_grad(gq, gk, pq, pk, cqw, ckw, cpos, cf, dv=gv, dq_out=outs[0], dk_out=outs[1], dv_out=outs[2],
                               amax=amax)
    check_grad(outs[0], res[2], dq, q, qw, pos, freqs, False, 1e-6, True, strips_of(B * S, H, H + 2 * K), "q")
    check_grad(outs[1], res[3], dk, k, kw, pos, freqs, False, 1e-6, True, strips_of(B * S, K, H + 2 * K), "k")
    assert torch.equal(outs[2].cpu(), dv)
    ld = (H + 2 * K) * dim + 5
    assert (flat[:skip] == 123).all() and (flat[skip + B * S * ld:] == 123).all()
    assert (flat[skip:skip + B * S * ld].view(B * S, ld)[:, -5:] == 123).all()
    assert amax.item() == max(t.float().abs().max().item() for t in outs)


@pytest.mark.parametrize("dim,rot", [(128, 128), (80, 40), (37, 36)])
def test_in_place(dim, rot):
    shape = (2, 9, 4, 2, dim, rot)
    q, k, qw, kw, dq, dk, dv, pos, freqs = make(shape, BF, BF, BF, seed=9)
    cq, ck, cqw, ckw, cdq, cdk, cpos, cf = cuda(q, k, qw, kw, dq, dk, pos, freqs)
    want = PL.qk_norm_rope(cq, ck, cqw, ckw, cpos, cf)
    grads = PL.qk_norm_rope_grad(cdq, cdk, cq, ck, cqw, ckw, cpos, cf)
    a, b = cq.clone(), ck.clone()
    PL.qk_norm_rope(a, b, cqw, ckw, cpos, cf, q_out=a, k_out=b)
    assert torch.equal(a, want[0]) and torch.equal(b, want[1])
    a, b = cdq.clone(), ck.clone()                       # dq over dq, dk over k
    got = PL.qk_norm_rope_grad(a, cdk, cq, b, cqw, ckw, cpos, cf, dq_out=a, dk_out=b)
    assert all(torch.equal(x, y) for x, y in zip(got, grads))
    v = dv.cuda()
    PL.qk_norm_rope_grad(cdq, cdk, cq, ck, cqw, ckw, cpos, cf, dv=v, dv_out=v)
    assert torch.equal(v.cpu(), dv)


@pytest.mark.parametrize("pos0", [0, 1 << 20, (1 << 40) + 12345, -(1 << 33)])
def test_far_positions(pos0):
    """Angles of far positions, up to where 64 bits leave them 2^-13 of a turn."""
    q, k, qw, kw, *_, freqs = make((1, 5, 2, 1, 128, 128), F32, F32, F32, seed=4)
    pos = pos0 + torch.arange(5)
    yq, yk = PL.qk_norm_rope(q.cuda(), k.cuda(), qw.cuda(), kw.cuda(), pos.cuda(), freqs.cuda())
    check(yq, q, qw, pos, freqs, False, 1e-6, True, "q")
    check(yk, k, kw, pos, freqs, False, 1e-6, True, "k")


def test_values_that_are_not_numbers_stay_in_their_row():
    shape = (1, 6, 4, 2, 128, 128)
    q, k, qw, kw, dq, dk, _, pos, freqs = make(shape, BF, BF, BF, seed=5)
    cq, ck, cqw, ckw, cdq, cdk, cpos, cf = cuda(q, k, qw, kw, dq, dk, pos, freqs)
    want = PL.qk_norm_rope(cq, ck, cqw, ckw, cpos, cf)
    gwant = PL.qk_norm_rope_grad(cdq, cdk, cq, ck, cqw, ckw, cpos, cf)
    for bad in (float("nan"), float("inf")):
        x = cq.clone()
        x[0, 2, 1, 5] = bad
        x[0, 3, 2] = 0                                   # a row of zeros: r = 1 / sqrt(eps)
        got = PL.qk_norm_rope(x, ck, cqw, ckw, cpos, cf)
        same = torch.ones(1, 6, 4, dtype=torch.bool, device="cuda")
        same[0, 2, 1] = same[0, 3, 2] = False
        assert torch.equal(got[0][same], want[0][same]) and torch.equal(got[1], want[1])
        assert not got[0][0, 2, 1].isfinite().all() and (got[0][0, 3, 2] == 0).all()
        g = PL.qk_norm_rope_grad(cdq, cdk, x, ck, cqw, ckw, cpos, cf)
        assert torch.equal(g[0][same], gwant[0][same]) and torch.equal(g[1], gwant[1])
        assert g[0][0, 3, 2].isfinite().all()


def test_large_values_and_eps():
    """Squares up to 2^126, and rows whose squares are far below eps."""
    q, _, qw, *_ , freqs = make((1, 4, 2, 1, 64, 64), F32, F32, F32, seed=6)
    for scale, eps in ((2.0 ** 59, 1e-6), (1e-12, 1e-6), (1e-12, 0.0)):
        x = q * scale
        y, _ = PL.qk_norm_rope(x.cuda(), None, qw.cuda(), None, None, freqs.cuda(), eps=eps)
        check(y, x, qw, None, freqs, False, eps, True, f"scale {scale}")


def test_empty():
    f = PL.rope_frequencies(64)
    w = torch.ones(64, device="cuda")
    for shape in ((0, 5, 2, 64), (2, 0, 2, 64), (2, 5, 0, 64)):
        x = torch.empty(shape, device="cuda", dtype=BF)
        y, z = PL.qk_norm_rope(x, x, w, w, None, f)
        assert y.shape == z.shape == x.shape
        amax = torch.full((1,), 5.0, device="cuda")
        g = PL.qk_norm_rope_grad(x, x, x, x, w, w, None, f, dv=x, dv_out=torch.empty_like(x), amax=amax)
        assert g[0].shape == x.shape and (g[2] == 0).all() and (g[3] == 0).all() and amax.item() == 0
    # keys alone have rows: the queries' weight gets zeros
    q, k = torch.empty(1, 3, 0, 64, device="cuda"), torch.randn(1, 3, 2, 64, device="cuda")
    g = PL.qk_norm_rope_grad(q, k, q, k, w, w, None, f)
    assert (g[2] == 0).all() and g[3].abs().max() > 0


def test_offsets_past_32_bits():
    """A row stride that takes the last rows past 2^32 bytes and 2^31 values."""
    S, H, D = 3, 2, 128
    flat = torch.empty(2 * (1 << 31) // 2 + (1 << 22), dtype=BF, device="cuda")
    stride = (1 << 30) + 64
    q, _, qw, _, dq, _, _, pos, freqs = make((1, S, H, 1, D, D), BF, BF, BF, seed=8)
    view = flat.as_strided((1, S, H, D), (S * stride, stride, D, 1))
    view.copy_(q)
    cqw, cpos, cf, cdq = cuda(qw, pos, freqs, dq)
    y, _ = PL.qk_norm_rope(view, None, cqw, None, cpos, cf)
    check(y, q, qw, pos, freqs, False, 1e-6, True, "far rows")
    PL.qk_norm_rope_grad(cdq, None, view, None, cqw, None, cpos, cf, dq_out=view)
    check_grad(view.contiguous(), None, dq, q, qw, pos, freqs, False, 1e-6, True, 1, "far rows")


def test_streams_and_graph():
    shape = (4, 33, 8, 2, 128, 128)
    q, k, qw, kw, dq, dk, dv, pos, freqs = make(shape, BF, BF, BF, seed=12)
    cq, ck, cqw, ckw, cdq, cdk, cdv, cpos, cf = cuda(q, k, qw, kw, dq, dk, dv, pos, freqs)
    packed = torch.empty(4, 33, 12, 128, dtype=BF, device="cuda")
    parts, amax = packed.split((8, 2, 2), 2), torch.empty(1, device="cuda")

    def step():
        y = PL.qk_norm_rope(cq, ck, cqw, ckw, cpos, cf)
        g = PL.qk_norm_rope_grad(cdq, cdk, cq, ck, cqw, ckw, cpos, cf, dv=cdv, dq_out=parts[0], dk_out=parts[1],
                                 dv_out=parts[2], amax=amax)
        return [*y, packed, *g[2:], amax]

    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = PL.qk_norm_rope(cq, ck, cqw, ckw, cpos, cf, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y[0], want[0]) and torch.equal(y[1], want[1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i in range(3):
        for t in outs:
            t.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b), i
        _ = step()                                      # eager work of the same tensors between replays
        cpos.add_(0)


def test_c_names_single_outputs():
    """A weight's gradient alone or left out, through the C names."""
    B, S, H, K, D = 2, 9, 3, 2, 64
    q, k, qw, kw, dq, dk, _, pos, freqs = make((B, S, H, K, D, D), BF, BF, F32, seed=2)
    cq, ck, cqw, ckw, cdq, cdk, cpos, cf = cuda(q, k, qw, kw, dq, dk, pos, freqs)
    full = PL.qk_norm_rope_grad(cdq, cdk, cq, ck, cqw, ckw, cpos, cf)
    n = P.pbs_qk_norm_rope_grad_bytes(B, S, D)
    for want_q, want_k in ((1, 0), (0, 1), (0, 0)):
        ws = torch.empty(n, dtype=torch.uint8, device="cuda") if want_q or want_k else None
        oq, ok = torch.empty_like(cq), torch.empty_like(ck)
        gq, gk = torch.full((D,), 5.0, device="cuda"), torch.full((D,), 5.0, device="cuda")
        P.pbs_qk_norm_rope_grad(cdq, cdq.stride()[:3], cdk, cdk.stride()[:3], None, None, P.PBS_FMT_BF16, cq,
                                cq.stride()[:3], H, ck, ck.stride()[:3], K, P.PBS_FMT_BF16, B, S, D, cqw, ckw,
                                P.PBS_FMT_F32, 1, 1e-6, cpos, S, cf, D, 0, oq, oq.stride()[:3], ok, ok.stride()[:3], None,
                                None, gq if want_q else None, gk if want_k else None, None, ws, n if ws is not None else 0)
        assert torch.equal(oq, full[0]) and torch.equal(ok, full[1])
        assert torch.equal(gq, full[2]) if want_q else (gq == 5).all()
        assert torch.equal(gk, full[3]) if want_k else (gk == 5).all()


def test_benchmark_layer_whole():
    """The benchmark's layer, every row."""
    B, S, H, D = 31, 512, 32, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    qkv = torch.randn(B, S, 3 * H, D, device="cuda", generator=g).to(BF)
    q, k, _ = qkv.split(H, 2)
    qw = (1 + 0.2 * torch.randn(D, device="cuda", generator=g)).to(BF)
    dy = [(1e-3 * torch.randn(B, S, H, D, device="cuda", generator=g)).to(BF) for _ in range(3)]
    f = PL.rope_frequencies(D)
    yq, yk = PL.qk_norm_rope(q, k, qw, qw, None, f)
    out = torch.empty_like(qkv)
    oq, ok, ov = out.split(H, 2)
    amax = torch.empty(1, device="cuda")
    res = PL.qk_norm_rope_grad(dy[0], dy[1], q, k, qw, qw, None, f, dv=dy[2], dq_out=oq, dk_out=ok, dv_out=ov, amax=amax)
    assert amax.item() == out.float().abs().max().item() and torch.equal(ov, dy[2])
    for x, y, d, o, w in ((q, yq, dy[0], oq, res[2]), (k, yk, dy[1], ok, res[3])):
        want, e = forward_ref(x.double(), qw.double(), None, f, False, 1e-6, True, BF)
        assert ((y.double() - want).abs() <= e).all()
        del want, e
        want = grad_ref(d.double(), x.double(), qw.double(), None, f, False, 1e-6, True, BF, strips_of(B * S, H, 3 * H))
        assert ((o.double() - want[0]).abs() <= want[1]).all()
        assert ((w.double() - want[2]).abs() <= want[3]).all()
        del want


@pytest.mark.parametrize("types", [(BF, BF, BF), (F32, F32, F32)], ids=["bf16", "fp32"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("heads,dim,rot", [(1, 128, 128), (3, 64, 32), (5, 96, 96), (9, 256, 128), (1, 37, 36), (2, 512, 512)])
def test_gradient_with_eps_zero(heads, dim, rot, inter, types):
    """Rounds of heads that end behind the last head: what is not there adds nothing to the weights' gradients."""
    tx, ty, tw = types
    q, _, qw, _, dq, _, _, pos, freqs = make((2, 5, heads, 1, dim, rot), tx, ty, tw, seed=heads + dim)
    cq, cqw, cdq, cpos, cf = cuda(q, qw, dq, pos, freqs)
    g = PL.qk_norm_rope_grad(cdq, None, cq, None, cqw, None, cpos, cf, inter, 0.0)
    check_grad(g[0], g[2], dq, q, qw, pos, freqs, inter, 0.0, True, 1, "q")


def test_rotation_alone_and_values_that_are_not_numbers():
    """Without the norm the gradient of the inputs does not depend on them."""
    shape = (1, 6, 4, 2, 128, 64)
    q, k, qw, kw, dq, dk, _, pos, freqs = make(shape, BF, BF, BF, seed=15)
    cq, ck, cqw, ckw, cdq, cdk, cpos, cf = cuda(q, k, qw, kw, dq, dk, pos, freqs)
    want = PL.qk_norm_rope_grad(cdq, cdk, cq, ck, cqw, ckw, cpos, cf, norm=False)
    for bad in (float("nan"), float("inf"), -float("inf")):
        x = cq.clone()
        x[0, 2, 1, 5] = bad
        x[0, 4] = bad
        got = PL.qk_norm_rope_grad(cdq, cdk, x, ck, cqw, ckw, cpos, cf, norm=False)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(got[3], want[3])


def test_more_tokens_than_one_axis_of_a_launch():
    """2^26 rows of two values: 2^32 threads and more."""
    B, S = 2, (1 << 24) - 3
    g = torch.Generator(device="cuda").manual_seed(5)
    q, k = (torch.randn(B, S, 1, 2, device="cuda", generator=g).to(BF) for _ in range(2))
    q2, k2 = (torch.randn(B * 4, S, 1, 2, device="cuda", generator=g).to(BF) for _ in range(2))
    f = torch.tensor([0.01], dtype=torch.float64, device="cuda")
    for a, b in ((q, k), (q2, k2)):
        ya, yb = PL.qk_norm_rope(a, b, None, None, None, f)
        for x, y in ((a, ya), (b, yb)):
            for i in range(x.shape[0]):
                # the formula in fp32, angles in 64 bits: a few roundings of 2^-24 beside bf16's own half step, 2^-8
                t = torch.arange(S, device="cuda").double() * 0.01
                c, s = t.cos().float(), t.sin().float()
                v = x[i, :, 0].float()
                n = v * torch.rsqrt(v.square().mean(-1, keepdim=True) + 1e-6)
                want = torch.stack((n[:, 0] * c - n[:, 1] * s, n[:, 1] * c + n[:, 0] * s), -1)
                assert ((y[i, :, 0].float() - want).abs() <= 2.0 ** -8 * want.abs() + 2e-6).all(), i
