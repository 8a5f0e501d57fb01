"""The linear head's losses where every id of the vocabulary counts, and the gradients' paths that only large calls take,
against the formulas in 64 bits (on the GPU)."""
import pytest
import torch

from precision_block_scaled_amd import pipeline as PL
from tests.head_ref import head_ref, slots_of, stored
from tests.test_gpu_head import make, teacher
from tests.test_gpu_norm_rows import within

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


def same(a, b):
    return all(torch.equal(u, v) for u, v in zip(a, b))


# small tiles and large ones, joins of a few and of thousands of parts, one piece and several
@pytest.mark.parametrize("T,V,H,piece", [(64, 9001, 64, 0), (128, 33001, 128, 4096), (257, 513, 64, 0),
                                         (200, 33001, 192, 0), (900, 33001, 832, 0), (900, 33001, 832, 16384),
                                         (2000, 8100, 832, 0), (1100, (1 << 21) + 70, 1024, 0)])
def test_every_id_counts(T, V, H, piece):
    """Token t has the logit 64 at the ids v = t mod H and 0 at the others, so its n ids share all of the softmax: lse =
    64 + log n, and q = 1 / n at each of them (the others' e^-64 is past fp32).  All products are exact.  One id left out
    or counted twice, anywhere, moves lse by 1 / n, and dx and dw by whole terms."""
    k = torch.arange(T, device="cuda") % H
    v = torch.arange(V, device="cuda")
    x, w = torch.zeros(T, H, device="cuda", dtype=BF), torch.zeros(V, H, device="cuda", dtype=BF)
    x[torch.arange(T, device="cuda"), k] = 8
    w[v, v % H] = 8
    targets = (torch.arange(T, device="cuda") * 7919 + 5) % V
    targets[::2] = k[::2]                              # every other target is one of the token's n ids
    targets[-1] = V - 1
    n = ((V - 1 - k) // H + 1).double()
    hit = (targets % H == k).double()
    loss, lse = PL.linear_xent(x, w, targets)
    # sums of ones are exact; the logarithm of base 2 (one step at most), its product with log 2 and that constant
    # (a step each), the additions of the maximum in units of log 2 and its own product with 1 / log 2
    want = 64 + n.log()
    assert ((lse.double() - want).abs() <= 8 * U * want).all()
    assert ((loss.double() - (want - 64 * hit)).abs() <= 10 * U * want).all()
    assert (1 / n).min() > 8 * 10 * U * want.max()     # an id more or less would show
    dloss = torch.full((T,), 2.0 ** -6, device="cuda")
    dx, dw = PL.linear_xent_grad(dloss, x, w, targets, lse, piece=piece, dw_dtype=F32)
    want = torch.zeros(T, H, device="cuda", dtype=torch.float64)
    at = torch.arange(T, device="cuda")
    want[at, k] = 8 * 2.0 ** -6
    want[at, targets % H] -= 8 * 2.0 ** -6
    # q is off by lse's error, its rounding to bf16 by half a step of each term, the store by half a step
    assert ((dx.double() - want).abs() <= 8 * 2.0 ** -6 * (2.0 ** -7 + 2.0 ** -10)).all()
    if n.max() < 60:
        assert 1 / n.max() > 2 * (2.0 ** -7 + 2.0 ** -10)
    # dw: v's row has one column of q terms, of the tokens with k = v mod H, and its hits'
    tokens = torch.bincount(k, minlength=H).double()
    share = 8 * 2.0 ** -6 * tokens / ((V - 1 - torch.arange(H, device="cuda")) // H + 1)
    got = dw.double()
    got.index_put_((targets, k), torch.full((T,), 8 * 2.0 ** -6, device="cuda", dtype=torch.float64), accumulate=True)
    room = torch.zeros_like(got)
    room[v, v % H] = share[v % H] * (2.0 ** -8 + 2.0 ** -12)
    room.index_put_((targets, k), torch.full((T,), 8 * 2.0 ** -6 * 2.0 ** -8, device="cuda", dtype=torch.float64),
                    accumulate=True)
    got[v, v % H] -= share[v % H]
    assert (got.abs() <= room + 1e-20).all()


def check(got, want, dtype):
    for name, value in zip(("loss", "lse", "dx", "dw"), got):
        bound = stored(want["dw"], dtype) if name == "dw" else want[name]
        within(value, *bound, name)


def reference(x, w, slots, tau, dloss):
    return head_ref(x.cuda().double(), w.cuda().double(), [t.cuda() for t in slots], tau, dloss.cuda().double())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_products_apart_over_pieces(dtype):
    """So many tiles of dx that it and dW run apart, dx summed in fp32 over three pieces, the last one ragged; each
    gradient alone is the same."""
    T, V, H = 8300, 5000, 4096
    x, w, targets, dloss = make(T, V, H, seed=31, masked=0.2)
    want = reference(x, w, slots_of(targets), 1.0, dloss)
    x, w, targets, dloss = (t.cuda() for t in (x, w, targets, dloss))
    loss, lse = PL.linear_xent(x, w, targets)
    dx, dw = PL.linear_xent_grad(dloss, x, w, targets, lse, piece=2048, dw_dtype=dtype)
    check((loss, lse, dx, dw), want, dtype)
    assert not dx[targets < 0].any()
    again = PL.linear_xent_grad(dloss, x, w, targets, lse, piece=2048, dw_dtype=dtype)
    assert same(again, (dx, dw))
    assert torch.equal(PL.linear_xent_grad(dloss, x, w, targets, lse, piece=2048, need_dw=False)[0], dx)
    assert torch.equal(PL.linear_xent_grad(dloss, x, w, targets, lse, piece=2048, need_dx=False, dw_dtype=dtype)[1], dw)


@pytest.mark.parametrize("k,piece", [(9, 8192), (130, 8448)])
def test_distillation_in_pieces_of_large_tiles(k, piece):
    """256 x 256 tiles in both products of a distillation in pieces, whose slots fall into different ones."""
    T, V, H = 4100, 17000, 832
    x, w, targets, dloss = make(T, V, H, seed=32, masked=0.1)
    ids, logits = teacher(T, V, k, targets, seed=4)
    want = reference(x, w, slots_of(None, ids, logits, 2.0), 2.0, dloss)
    x, w, ids, logits, dloss = (t.cuda() for t in (x, w, ids, logits, dloss))
    loss, lse = PL.linear_distill(x, w, ids, logits, 2.0)
    dx, dw = PL.linear_distill_grad(dloss, x, w, ids, logits, 2.0, lse, piece=piece)
    check((loss, lse, dx, dw), want, BF)
    assert same(PL.linear_distill_grad(dloss, x, w, ids, logits, 2.0, lse, piece=piece), (dx, dw))
