"""The linear head's losses and gradients on the GPU against the formulas in 64 bits."""
import pytest
import torch

import precision_block_scaled_amd as P
from precision_block_scaled_amd import pipeline as PL
from tests.head_ref import head_ref, slots_of, stored
from tests.norm_ref import assert_within

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
# one token, one id, tile edges on either side, products whose K loop is split (few tokens against a long
# vocabulary; a small vocabulary against many tokens), one to several stages of K; the last two take 256 x 256 tiles
# for the logits, the last for the gradients' products too, the others 128 x 128
SHAPES = [(1, 1, 64), (1, 257, 64), (2, 256, 128), (37, 300, 64), (63, 1000, 192), (64, 64, 64), (65, 129, 128),
          (128, 128, 256), (129, 500, 64), (255, 1000, 192), (256, 512, 64), (257, 513, 128),
          (300, 2003, 320), (513, 131, 64), (70, 9001, 512), (2100, 300, 64), (1500, 17, 128),
          (300, 33001, 192), (4100, 4100, 128), (2000, 8100, 64), (2000, 8100, 832)]


def make(T, V, H, seed=0, masked=0.0):
    g = torch.Generator().manual_seed(seed)
    w = (torch.randn(V, H, generator=g) * 0.05).to(BF)
    targets = torch.randint(0, V, (T,), generator=g)
    x = (torch.randn(T, H, generator=g) + torch.rand(T, 1, generator=g) * 60 / H ** 0.5 * w[targets].float()).to(BF)
    dloss = torch.rand(T, generator=g) - 0.3
    out = torch.rand(T, generator=g) < masked
    return x, w, torch.where(out, -100, targets), dloss


def teacher(T, V, k, targets, seed=0, dtype=F32):
    g = torch.Generator().manual_seed(seed + 1000)
    ids = torch.rand(T, max(V, k), generator=g).argsort(1)[:, :k] % V
    ids[:, 0] = targets.clamp(min=0)
    logits = (2 * torch.randn(T, k, generator=g)).to(dtype)
    ids = torch.where(torch.rand(T, k, generator=g) < 0.15, -1, ids)
    ids[targets < 0] = -7
    return ids, logits


def check(got, want, dw_dtype=BF):
    for name, value in got.items():
        if name == "dw":
            assert_within(value, *stored(want["dw"], dw_dtype), name)
        else:
            assert_within(value, *want[name], name)


def xent(x, w, targets, dloss, **kw):
    x, w, targets, dloss = (t.cuda() for t in (x, w, targets, dloss))
    loss, lse = PL.linear_xent(x, w, targets)
    dx, dw = PL.linear_xent_grad(dloss, x, w, targets, lse, **kw)
    return dict(loss=loss, lse=lse, dx=dx, dw=dw)


def distill(x, w, ids, logits, tau, dloss, **kw):
    x, w, ids, logits, dloss = (t.cuda() for t in (x, w, ids, logits, dloss))
    loss, lse = PL.linear_distill(x, w, ids, logits, tau)
    dx, dw = PL.linear_distill_grad(dloss, x, w, ids, logits, tau, lse, **kw)
    return dict(loss=loss, lse=lse, dx=dx, dw=dw)


def same(a, b):
    return all(torch.equal(a[k], b[k]) for k in a)


@pytest.mark.parametrize("masked", [0.0, 0.4], ids=["all", "masked"])
@pytest.mark.parametrize("T,V,H", SHAPES)
def test_cross_entropy(T, V, H, masked):
    x, w, targets, dloss = make(T, V, H, seed=T + V, masked=masked)
    want = head_ref(x.double(), w.double(), slots_of(targets), 1.0, dloss.double())
    got = xent(x, w, targets, dloss)
    assert got["dx"].dtype == BF and got["dw"].dtype == BF
    check(got, want)
    assert same(got, xent(x, w, targets, dloss))


@pytest.mark.parametrize("T,V,H", [(33000, 69, 1024), (8300, 1100, 2048)])
def test_small_vocabulary(T, V, H):
    """Many tokens against few ids: dx is stored by its product, zeros for the tokens left out."""
    x, w, targets, dloss = make(T, V, H, seed=14, masked=0.3)
    want = head_ref(x.double(), w.double(), slots_of(targets), 1.0, dloss.double())
    got = xent(x, w, targets, dloss)
    check(got, want)
    assert not got["dx"][(targets < 0).cuda()].any()
    assert same(got, xent(x, w, targets, dloss))
    alone, _ = PL.linear_xent_grad(dloss.cuda(), x.cuda(), w.cuda(), targets.cuda(), got["lse"], need_dw=False)
    assert torch.equal(alone, got["dx"])


@pytest.mark.parametrize("k,tau,dtype", [(1, 1.0, F32), (5, 2.0, BF), (32, 0.7, F32), (130, 3.0, F32)])
@pytest.mark.parametrize("T,V,H", SHAPES)
def test_distillation(T, V, H, k, tau, dtype):
    x, w, targets, dloss = make(T, V, H, seed=T + V, masked=0.1)
    ids, logits = teacher(T, V, k, targets, seed=k, dtype=dtype)
    want = head_ref(x.double(), w.double(), slots_of(None, ids, logits, tau), tau, dloss.double())
    got = distill(x, w, ids, logits, tau, dloss)
    check(got, want)
    assert same(got, distill(x, w, ids, logits, tau, dloss))


@pytest.mark.parametrize("T,V,H,piece", [(300, 2003, 320, 1), (300, 2003, 320, 256), (300, 2003, 320, 700),
                                         (300, 2003, 320, 1024), (300, 2003, 320, 100000), (4200, 9000, 64, 4096)])
def test_pieces_of_the_vocabulary(T, V, H, piece):
    x, w, targets, dloss = make(T, V, H, seed=8, masked=0.2)
    want = head_ref(x.double(), w.double(), slots_of(targets), 1.0, dloss.double())
    for dtype in (BF, F32):
        got = xent(x, w, targets, dloss, piece=piece, dw_dtype=dtype)
        assert got["dw"].dtype == dtype
        check(got, want, dtype)
    ids, logits = teacher(T, V, 9, targets)
    want = head_ref(x.double(), w.double(), slots_of(None, ids, logits, 2.0), 2.0, dloss.double())
    check(distill(x, w, ids, logits, 2.0, dloss, piece=piece), want)


def test_one_gradient_alone():
    x, w, targets, dloss = make(70, 1000, 128, seed=2)
    full = xent(x, w, targets, dloss, piece=512)
    a = xent(x, w, targets, dloss, piece=512, need_dw=False)
    b = xent(x, w, targets, dloss, piece=512, need_dx=False)
    assert a["dw"] is None and b["dx"] is None
    assert torch.equal(a["dx"], full["dx"]) and torch.equal(b["dw"], full["dw"])


@pytest.mark.parametrize("T,V,H", [(37, 300, 64), (300, 1000, 128), (600, 70, 64)])
def test_masked_rows_hold_anything(T, V, H):
    """Infinities and NaN in the rows of masked tokens, wherever these stand, reach nothing."""
    x, w, targets, dloss = make(T, V, H, seed=3, masked=0.5)
    for edge in (0, T - 1):
        targets[edge] = -1
    want = xent(x, w, targets, dloss)
    x[targets < 0] = float("nan")
    x[0] = float("inf")
    dloss[targets < 0] = float("nan")
    got = xent(x, w, targets, dloss)
    assert same(got, want)
    out = targets < 0
    assert not got["loss"].cpu()[out].any() and not got["lse"].cpu()[out].any() and not got["dx"].cpu()[out].any()
    assert got["dw"].isfinite().all()


def test_every_token_masked():
    x, w, targets, dloss = make(50, 300, 64)
    got = xent(x * float("nan"), w, torch.full_like(targets, -100), dloss)
    for v in got.values():
        assert not v.any()
    ids, logits = teacher(50, 300, 6, targets)
    for i, l in ((torch.full_like(ids, -1), logits * float("nan")), (ids, torch.full_like(logits, -torch.inf))):
        got = distill(x, w, i, l, 1.0, dloss)
        for v in got.values():
            assert not v.any()


def test_no_tokens():
    w = torch.randn(300, 64, device="cuda").to(BF)
    x, none = torch.empty(0, 64, dtype=BF, device="cuda"), torch.empty(0, device="cuda")
    targets = torch.empty(0, dtype=torch.int64, device="cuda")
    loss, lse = PL.linear_xent(x, w, targets)
    dx, dw = PL.linear_xent_grad(none, x, w, targets, lse)
    assert loss.shape == lse.shape == (0,) and dx.shape == (0, 64) and dw.shape == w.shape and not dw.any()
    ids, logits = torch.empty(0, 3, dtype=torch.int64, device="cuda"), torch.empty(0, 3, device="cuda")
    PL.linear_distill(x, w, ids, logits)
    dx, dw = PL.linear_distill_grad(none, x, w, ids, logits, 1.0, lse, dw_dtype=F32)
    assert not dw.any() and dw.dtype == F32


def test_slots_that_are_empty_repeated_lowest_or_infinite():
    x, w, targets, dloss = make(8, 500, 64, seed=6)
    ids, logits = teacher(8, 500, 6, targets)
    ids = ids.abs()
    low = torch.finfo(F32).min
    logits[0] = low                                    # a uniform distribution
    logits[1, 1:] = low                                # all on one
    logits[2, :3] = -torch.inf                         # probability 0
    ids[3] = 77                                        # the same id in every slot
    ids[4, 2:] = -1
    logits[4, 2:] = float("nan")                       # unused slots hold anything
    ids[5, :5], ids[5, 5] = -1, 499                    # one slot: a hard target
    ids[6, 0], ids[6, 4] = 255, 255                    # twice, among others
    for tau in (1.0, 0.25, 4.0):
        want = head_ref(x.double(), w.double(), slots_of(None, ids, logits, tau), tau, dloss.double())
        check(distill(x, w, ids, logits, tau, dloss), want)


@pytest.mark.parametrize("T,V,H", [(40, 300, 64), (2000, 8100, 64)])
def test_many_slots_of_one_id(T, V, H):
    """Seventy slots over four ids each: their probabilities add up, in the same order every time."""
    x, w, targets, dloss = make(T, V, H, seed=12, masked=0.1)
    ids, logits = teacher(T, V, 70, targets, seed=3)
    ids = torch.where(ids < 0, ids, ids % 4 * (V // 4) + 5)
    want = head_ref(x.double(), w.double(), slots_of(None, ids, logits, 1.5), 1.5, dloss.double())
    got = distill(x, w, ids, logits, 1.5, dloss)
    check(got, want)
    assert same(got, distill(x, w, ids, logits, 1.5, dloss))


def test_one_slot_is_cross_entropy():
    x, w, targets, dloss = make(90, 700, 128, seed=7, masked=0.2)
    a = xent(x, w, targets, dloss)
    b = distill(x, w, targets[:, None].contiguous(), torch.randn(90, 1), 1.0, dloss)
    assert same(a, b)


@pytest.mark.parametrize("bad", [300, 1 << 31, (1 << 32) + 5, 1 << 62])
def test_ids_past_the_vocabulary_give_nan(bad):
    x, w, targets, dloss = make(40, 300, 64, seed=4)
    fine = xent(x, w, targets, dloss)
    targets = targets.clone()
    targets[11] = bad
    got = xent(x, w, targets, dloss)
    others = torch.arange(40) != 11
    assert got["loss"][11].isnan() and got["dx"][11].isnan().all() and got["dw"].isnan().all()
    assert torch.equal(got["loss"].cpu()[others], fine["loss"].cpu()[others])
    assert torch.equal(got["dx"].cpu()[others], fine["dx"].cpu()[others])
    assert torch.equal(got["lse"], fine["lse"])
    ids, logits = teacher(40, 300, 3, targets.clamp(max=299))
    ids[11, 1] = bad
    got = distill(x, w, ids, logits, 1.0, dloss)
    assert got["loss"][11].isnan() and got["dx"][11].isnan().all() and got["dw"].isnan().all()
    assert got["loss"].cpu()[others].isfinite().all()


def test_nan_in_a_live_row():
    x, w, targets, dloss = make(40, 300, 64, seed=4)
    fine = xent(x, w, targets, dloss)
    x[39, 5] = float("nan")
    got = xent(x, w, targets, dloss)
    assert got["loss"][39].isnan() and got["dx"][39].isnan().all() and got["dw"].isnan().all()
    assert torch.equal(got["loss"][:39], fine["loss"][:39]) and torch.equal(got["dx"][:39], fine["dx"][:39])


@pytest.mark.parametrize("scale", [30.0, 1000.0])
def test_large_logits(scale):
    """Logits of hundreds to tens of thousands: no overflow, one id takes nearly all."""
    x, w, targets, dloss = make(70, 900, 64, seed=5)
    x = (x.float() * scale).to(BF)
    want = head_ref(x.double(), w.double(), slots_of(targets), 1.0, dloss.double())
    check(xent(x, w, targets, dloss), want)


def test_outputs_stay_within_their_rows():
    x, w, targets, dloss = make(37, 301, 64, seed=9)
    full = xent(x, w, targets, dloss)
    x, w, targets, dloss = (t.cuda() for t in (x, w, targets, dloss))
    loss, lse = (torch.full((37 + 64,), 5.0, device="cuda") for _ in range(2))
    dx = torch.full((37 + 4, 64), 5.0, dtype=BF, device="cuda")
    dw = torch.full((301 + 4, 64), 5.0, dtype=BF, device="cuda")
    a, b = P.pbs_linear_loss_bytes(37, 301, 64)
    ws = torch.full((max(a, b) + 256,), 0x5A, dtype=torch.uint8, device="cuda")
    P.pbs_linear_xent(x, w, 37, 301, 64, targets, loss, lse, ws, a)
    assert (ws[a:] == 0x5A).all()
    P.pbs_linear_xent_grad(dloss, x, w, 37, 301, 64, targets, lse, 0, dx, dw, P.PBS_FMT_BF16, ws, b)
    assert (ws[b:] == 0x5A).all()
    for got, want in ((loss, full["loss"]), (lse, full["lse"]), (dx, full["dx"]), (dw, full["dw"])):
        assert torch.equal(got[:len(want)], want) and (got[len(want):] == 5.0).all()


def test_other_stream_and_graph():
    x, w, targets, dloss = (t.cuda() for t in make(300, 1100, 128, seed=1, masked=0.3))
    ids, logits = (t.cuda() for t in teacher(300, 1100, 8, targets.cpu()))

    def step(**kw):
        loss, lse = PL.linear_xent(x, w, targets, **kw)
        dx, dw = PL.linear_xent_grad(dloss, x, w, targets, lse, piece=512, **kw)
        dl, ls = PL.linear_distill(x, w, ids, logits, 2.0, **kw)
        return loss, lse, dx, dw, dl, ls, *PL.linear_distill_grad(dloss, x, w, ids, logits, 2.0, ls, **kw)

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for s in (side, side.cuda_stream):
        got = step(stream=s)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = step()
        graphs.append((graph, outs))
    for k in range(4):
        x.copy_(x.flip(0))
        targets.copy_(targets.roll(k))
        dloss.mul_(0.5)
        want = step()
        for graph, outs in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for graph, outs in graphs:
            assert all(torch.equal(a, b) for a, b in zip(outs, want)), k


def test_two_streams_at_once():
    cases = [[t.cuda() for t in make(400, 3000, 256, seed=s, masked=0.2 * s)] for s in range(2)]
    want = [xent(*c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for (x, w, targets, dloss), s in zip(cases, streams):
            loss, lse = PL.linear_xent(x, w, targets, stream=s)
            dx, dw = PL.linear_xent_grad(dloss, x, w, targets, lse, stream=s)
            got.append(dict(loss=loss, lse=lse, dx=dx, dw=dw))
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(got, want))


def gpu_ref(x, w, targets, dloss):
    """The step in float64 on the GPU, for sizes that the host is too slow for."""
    z = x.double() @ w.double().t()
    lse = torch.logsumexp(z, 1)
    loss = lse - z.gather(1, targets[:, None])[:, 0]
    dz = z.sub_(lse[:, None]).exp_()
    dz.scatter_add_(1, targets[:, None], -torch.ones_like(targets, dtype=torch.float64)[:, None])
    dz.mul_(dloss.double()[:, None])
    dx, dw = dz @ w.double(), dz.t() @ x.double()
    # what bf16 dz may add: half a step of every term
    return loss, lse, (dx, dz, 2 ** -8 * (dz.abs_() @ w.double().abs())), dw


@pytest.mark.parametrize("T,V,H,piece", [(3, (1 << 21) + 70, 1024, 0), (8450, 262400, 64, 262400),
                                         (4200, 16500, 832, 8192)],
                         ids=["weight beyond 4 GiB", "piece beyond 4 GiB", "large tiles, three pieces"])
def test_large(T, V, H, piece):
    """A head of more than 4 GiB; a piece whose dz takes more than 4 GiB; pieces of 256 x 256 tiles."""
    g = torch.Generator(device="cuda").manual_seed(3)
    w = (torch.randn(V, H, device="cuda", generator=g) * 0.05).to(BF)
    x = torch.randn(T, H, device="cuda", generator=g).to(BF)
    targets = torch.randint(0, V, (T,), device="cuda", generator=g)
    targets[-1] = V - 1
    dloss = torch.full((T,), 1.0 / T, device="cuda")
    loss, lse = PL.linear_xent(x, w, targets)
    dx, dw = PL.linear_xent_grad(dloss, x, w, targets, lse, piece=piece)
    want_loss, want_lse, (want_dx, _, room), want_dw = gpu_ref(x, w, targets, dloss)
    # logits up to about 10 with sums of |x w| up to 64 (H = 1024): (H + 3) U 64 = 0.004 for the worst order of
    # additions, 1e-4 for 40 times that of a tree
    assert (loss - want_loss).abs().max() < 1e-4 and (lse - want_lse).abs().max() < 1e-4
    # dx: half a step of bf16 for every term and for the result, and 5 in 100 of it for dz's fp32 errors (about 1e-4
    # of q, where half a step is 4e-3); dw: the same halves, in the 2-norm of the whole
    assert ((dx - want_dx).abs() <= room * 1.05 + 2 ** -8 * want_dx.abs()).all()
    assert (dw - want_dw).norm() <= 2 ** -7 * want_dw.norm()


def test_norm_head_loss_and_back():
    """A step's end as it is used: norm, head, loss, gradients back through the norm, against autograd in 64 bits."""
    T, V, H = 200, 1500, 256
    x, w, targets, _ = make(T, V, H, seed=12, masked=0.25)
    gamma, beta = 1 + 0.1 * torch.randn(H), 0.1 * torch.randn(H)
    live = int((targets >= 0).sum())
    dloss = torch.full((T,), 1.0 / live)
    xg, wg, tg, gg, bg, dg = (t.cuda() for t in (x, w, targets, gamma, beta, dloss))
    y, mean, rstd = PL.layernorm(xg, gg, bg)
    loss, lse = PL.linear_xent(y, wg, tg)
    dy, dw = PL.linear_xent_grad(dg, y, wg, tg, lse, dw_dtype=F32)
    dx, dgamma, dbeta = PL.layernorm_grad(dy, xg, gg, mean, rstd)
    leaves = [t.double().requires_grad_() for t in (x, w, gamma, beta)]
    yr = torch.nn.functional.layer_norm(leaves[0], (H,), leaves[2], leaves[3], 1e-5)
    want = torch.nn.functional.cross_entropy(yr @ leaves[1].t(), targets, ignore_index=-100)
    grads = torch.autograd.grad(want, leaves)
    # y, dz and dy are each rounded to bf16 (2^-8 at most, each an independent error of a sum's terms); the norm of
    # their sum over the result's norm stays below the sum of the three and the last store's
    assert abs((loss.double().cpu() * dloss).sum() - want) < 2 ** -8 * want
    for name, got, ref in zip(("dx", "dw", "dgamma", "dbeta"), (dx, dw, dgamma, dbeta), grads):
        assert (got.double().cpu() - ref).norm() <= 4 * 2 ** -8 * ref.norm(), name


@pytest.mark.parametrize("T,V,H,top", [(1, 300, 64, 0), (37, 2003, 256, 7), (70, 9001, 512, 0), (129, 500, 64, 5),
                                       (300, 33001, 192, 0), (2100, 300, 64, 0), (4100, 1000, 128, 9)])
@pytest.mark.parametrize("masked", [0.0, 0.7])
def test_workspace_is_not_overrun(T, V, H, top, masked):
    """Exactly the bytes that pbs_linear_loss_bytes gives, what lies behind them untouched: partial products of dx and
    dW in as many splits as the live rows allow."""
    x, w, targets, dloss = make(T, V, H, seed=21, masked=masked)
    ids, logits = (t.cuda() for t in teacher(T, V, top or 1, targets))
    x, w, targets, dloss = (t.cuda() for t in (x, w, targets, dloss))
    a, b = P.pbs_linear_loss_bytes(T, V, H, top)
    lse = (PL.linear_distill(x, w, ids, logits, 2.0) if top else PL.linear_xent(x, w, targets))[1]
    ws = torch.full((b + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    if top:
        P.pbs_linear_distill_grad(dloss, x, w, T, V, H, ids, logits, P.PBS_FMT_F32, top, 2.0, lse, 0, dx, dw,
                                  P.PBS_FMT_BF16, ws, b)
        want = PL.linear_distill_grad(dloss, x, w, ids, logits, 2.0, lse)
    else:
        P.pbs_linear_xent_grad(dloss, x, w, T, V, H, targets, lse, 0, dx, dw, P.PBS_FMT_BF16, ws, b)
        want = PL.linear_xent_grad(dloss, x, w, targets, lse)
    assert (ws[b:] == 0x5A).all()
    assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])
