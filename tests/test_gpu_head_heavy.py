"""The values of dz that a token's gradient hangs on, at its target or its teacher's likely ids, reach dx and dw with
what their rounding to bf16 left out."""
import pytest
import torch

from precision_block_scaled_amd import pipeline as PL
from tests.head_ref import head_ref, slots_of, stored
from tests.test_gpu_norm_rows import within

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
MOST_SHARED = 8                 # an id that is heavy for more tokens has its row of dw left as the product gave it


def make(T, V, H, seed, masked=0.0, crowd=()):
    """Rows of w are 0 but for every 16th id, from which the targets come: the softmax is spread over all ids, so that
    the rounding of all the other values of dz reaches little of dx and dw.  crowd: so many tokens share each of the
    first targets."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = 0.05 * torch.randn(V, H, device="cuda", generator=g)
    w[torch.arange(V, device="cuda") % 16 != 3 % V] = 0
    x = torch.randn(T, H, device="cuda", generator=g)
    held = torch.arange(3 % V, V, 16, device="cuda")
    targets = held[torch.randperm(max(T, len(held)), device="cuda", generator=g)[:T] % len(held)]
    at = 0
    for k, n in enumerate(crowd):
        targets[targets == held[k]] = held[len(crowd)]
        targets[at:at + n] = held[k]
        at += n
    order = torch.randperm(T, device="cuda", generator=g)
    targets = targets[order].contiguous()
    dloss = 0.5 + torch.rand(T, device="cuda", generator=g)
    out = torch.rand(T, device="cuda", generator=g) < masked
    return x.to(BF), w.to(BF), torch.where(out, -100, targets), dloss


def kept(ids, p, T, V, limit=1.1):
    """Masks of dz for dx and dw: the heavy values, and those whose id is heavy for few enough tokens."""
    heavy = (p > 0.2) & (ids >= 0)
    m = torch.zeros(T, V, dtype=torch.bool, device="cuda")
    rows = torch.arange(T, device="cuda")[:, None].expand_as(ids)
    m[rows[heavy], ids[heavy]] = True
    few = m.sum(0) <= MOST_SHARED
    return m, m & few & (T <= MOST_SHARED * V)


def check(got, want, dtype):
    for name in got:
        within(got[name], *(stored(want["dw"], dtype) if name == "dw" else want[name]), name)


def same(a, b):
    return all(torch.equal(u, v) for u, v in zip(a, b))


# dx through partial products and stored by its product; dw in one split and in several, in one piece and in several;
# small tiles and large ones; its rows set aside by token and by id
CASES = [(129, 5003, 64, 0, 0.0), (300, 2003, 320, 512, 0.3), (1000, 1000, 512, 0, 0.2), (2100, 300, 64, 0, 0.1),
         (600, 33001, 192, 16384, 0.0), (2000, 8100, 832, 0, 0.2), (4200, 16500, 832, 8192, 0.1), (8300, 1100, 2048, 0, 0.3)]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("T,V,H,piece,masked", CASES)
def test_cross_entropy_targets(T, V, H, piece, masked, dtype):
    x, w, targets, dloss = make(T, V, H, seed=T, masked=masked, crowd=(8, 9, 1, 30))
    slots = [t.cuda() for t in slots_of(targets.cpu())]
    want = head_ref(x.double(), w.double(), slots, 1.0, dloss.double(), kept(slots[0], slots[1], T, V))
    loss, lse = PL.linear_xent(x, w, targets)
    got = PL.linear_xent_grad(dloss, x, w, targets, lse, piece=piece, dw_dtype=dtype)
    check(dict(zip(("dx", "dw"), got)), want, dtype)
    for _ in range(3):
        assert same(PL.linear_xent_grad(dloss, x, w, targets, lse, piece=piece, dw_dtype=dtype), got)
    # alone, in other splits perhaps
    check(dict(dx=PL.linear_xent_grad(dloss, x, w, targets, lse, piece=piece, need_dw=False)[0]), want, dtype)
    alone = PL.linear_xent_grad(dloss, x, w, targets, lse, piece=piece, need_dx=False, dw_dtype=dtype)[1]
    check(dict(dw=alone), want, dtype)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("T,V,H,piece,masked", CASES + [(33000, 69, 1024, 0, 0.3)])
def test_distillation_likely_ids(T, V, H, piece, masked, dtype):
    """Tokens with one to four slots above 1/5, some of them twice, among slots below it."""
    x, w, targets, dloss = make(T, V, H, seed=T + 1, masked=masked)
    g = torch.Generator(device="cuda").manual_seed(T)
    k = 11
    ids = (targets[:, None] + 16 * torch.arange(k, device="cuda")) % V
    ids = torch.where(targets[:, None] < 0, -1, ids)
    p = torch.full((T, k), 0.004, device="cuda")
    p[0::4, 3] = 0.96
    p[1::4, 0:2] = 0.48
    p[2::4, [0, 5, 9]] = 0.32
    p[3::4, [1, 4, 7, 10]] = 0.24
    ids[2::8, 7] = ids[2::8, 5]                        # one likely id again, in a slot of little weight
    ids[6::8, 9] = ids[6::8, 5]                        # and in one of as much
    order = torch.rand(T, k, device="cuda", generator=g).argsort(1)
    ids, logits = ids.gather(1, order).contiguous(), (2 * p.log()).gather(1, order).contiguous()
    slots = [t.cuda() for t in slots_of(None, ids.cpu(), logits.cpu(), 2.0)]
    want = head_ref(x.double(), w.double(), slots, 2.0, dloss.double(), kept(slots[0], slots[1], T, V))
    loss, lse = PL.linear_distill(x, w, ids, logits, 2.0)
    got = PL.linear_distill_grad(dloss, x, w, ids, logits, 2.0, lse, piece=piece, dw_dtype=dtype)
    check(dict(zip(("dx", "dw"), got)), want, dtype)
    for _ in range(3):
        assert same(PL.linear_distill_grad(dloss, x, w, ids, logits, 2.0, lse, piece=piece, dw_dtype=dtype), got)


def test_gradients_are_as_near_as_their_store():
    """A step as it is met in training, in 2-norms: dx and dw are off by what their own rounding to bf16 takes, and a
    tenth more at most.  (Each value of dz below 1/5 of its token's weight is still rounded; their squares sum to
    a small part of the target's.)"""
    T, V, H = 1433, 20011, 1024
    g = torch.Generator(device="cuda").manual_seed(2)
    w = (0.02 * torch.randn(V, H, device="cuda", generator=g)).to(BF)
    targets = torch.randint(0, V, (T,), device="cuda", generator=g)
    x = torch.randn(T, H, device="cuda", generator=g)
    x = (x + 10 * torch.rand(T, 1, device="cuda", generator=g) / (0.02 ** 2 * H) * w[targets].float()).to(BF)
    dloss = torch.full((T,), 1.0 / T, device="cuda")
    loss, lse = PL.linear_xent(x, w, targets)
    got = PL.linear_xent_grad(dloss, x, w, targets, lse)
    z = x.double() @ w.double().t()
    dz = torch.softmax(z, 1).scatter_add_(1, targets[:, None], -torch.ones(T, 1, dtype=torch.float64, device="cuda"))
    dz *= dloss.double()[:, None]
    for value, want in zip(got, (dz @ w.double(), dz.t() @ x.double())):
        store = (want.to(BF).double() - want).norm()
        assert (value.double() - want).norm() <= 1.1 * store


def test_infinite_weight_of_a_token():
    """A dloss whose dz overflows bf16 alone: infinity stays infinity, and no NaN comes of what it left out."""
    T, V, H = 200, 1000, 64
    x, w, targets, dloss = make(T, V, H, seed=3)
    x = torch.zeros_like(x)
    x[:, 0] = 1
    dloss[7] = 3.4e38
    lse = PL.linear_xent(x, w, targets)[1]
    dx, dw = PL.linear_xent_grad(dloss, x, w, targets, lse, dw_dtype=F32)
    assert not dw[targets[7], 0].isnan() and dw[targets[7], 0] < -3e38


@pytest.mark.parametrize("T,V,H", [(1000, 5003, 64), (3000, 33001, 192)])
def test_most_tokens_on_one_id(T, V, H):
    """Most targets are one id and a few others, in the lanes of many waves: their lists hold them all once, whatever
    the order, and the ids of a few tokens beside them get theirs."""
    x, w, targets, dloss = make(T, V, H, seed=5, crowd=(T // 2, T // 4, 8, 7, 2))
    slots = [t.cuda() for t in slots_of(targets.cpu())]
    want = head_ref(x.double(), w.double(), slots, 1.0, dloss.double(), kept(slots[0], slots[1], T, V))
    lse = PL.linear_xent(x, w, targets)[1]
    got = PL.linear_xent_grad(dloss, x, w, targets, lse, dw_dtype=F32)
    check(dict(zip(("dx", "dw"), got)), want, F32)
    ids = torch.stack([targets, (targets + 16) % V, targets, (targets + 32) % V], 1).contiguous()
    logits = torch.log(torch.tensor([0.26, 0.3, 0.14, 0.3], device="cuda")).expand(T, 4).contiguous()
    slots = [t.cuda() for t in slots_of(None, ids.cpu(), logits.cpu(), 1.0)]
    want = head_ref(x.double(), w.double(), slots, 1.0, dloss.double(), kept(slots[0], slots[1], T, V))
    lse = PL.linear_distill(x, w, ids, logits, 1.0)[1]
    got = PL.linear_distill_grad(dloss, x, w, ids, logits, 1.0, lse, dw_dtype=F32)
    check(dict(zip(("dx", "dw"), got)), want, F32)
    for _ in range(5):
        assert same(PL.linear_distill_grad(dloss, x, w, ids, logits, 1.0, lse, dw_dtype=F32), got)
