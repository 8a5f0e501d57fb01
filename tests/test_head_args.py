"""The linear head's losses: what the calls refuse before anything is enqueued, and the 64-bit reference against
differences (CPU)."""
import os

import pytest
import torch

import precision_block_scaled_amd as P
from precision_block_scaled_amd import pipeline as PL
from tests.head_ref import head_ref, slots_of

FAKE = 1 << 40          # a non-null, aligned address never dereferenced
BF, F32 = P.PBS_FMT_BF16, P.PBS_FMT_F32
needs_lib = pytest.mark.skipif(not os.path.exists(P.lib_path), reason="libpbs.so not built")

SIZES = [(2, dict(tokens=-1)), (2, dict(tokens=(1 << 24) + 1)), (2, dict(vocab=0)), (2, dict(vocab=(1 << 22) + 1)),
         (2, dict(hidden=0)), (2, dict(hidden=96)), (2, dict(hidden=65600)), (2, dict(tokens=1 << 24, vocab=1 << 22))]
COMMON = SIZES + [(1, dict(x=None)), (1, dict(w=None)), (1, dict(x=FAKE + 2)), (1, dict(w=FAKE + 8)),
                  (1, dict(lse=None)), (1, dict(lse=FAKE + 2)), (1, dict(ws=None)), (1, dict(ws=FAKE + 16)),
                  (1, dict(n=1000))]
LOSS = [(1, dict(loss=None)), (1, dict(loss=FAKE + 1))]
GRAD = [(1, dict(dloss=None)), (1, dict(dloss=FAKE + 2)), (1, dict(piece=-1)), (1, dict(dx=None, dw=None)),
        (1, dict(dx=FAKE + 8)), (1, dict(dw=FAKE + 4)), (3, dict(dw_fmt=P.PBS_FMT_E4M3))]
XENT = [(1, dict(targets=None)), (1, dict(targets=FAKE + 4))]
TEACHER = [(1, dict(top_ids=None)), (1, dict(top_logits=None)), (1, dict(top_ids=FAKE + 4)),
           (1, dict(top_logits=FAKE + 2)), (3, dict(top_fmt=P.PBS_FMT_E5M2)), (2, dict(top=0)), (2, dict(top=1025)),
           (1, dict(tau=0.0)), (1, dict(tau=-1.0)), (1, dict(tau=float("nan"))), (1, dict(tau=float("inf")))]


def args(change):
    a = dict(x=FAKE, w=FAKE, tokens=8, vocab=100, hidden=64, targets=FAKE, top_ids=FAKE, top_logits=FAKE, top_fmt=F32,
             top=4, tau=1.0, loss=FAKE, lse=FAKE, dloss=FAKE, piece=0, dx=FAKE, dw=FAKE, dw_fmt=BF, ws=FAKE, n=1 << 62)
    assert set(change) <= set(a)
    return {**a, **change}


def refused(status, fn, *a):
    with pytest.raises(P.PBSError) as e:
        fn(*a)
    assert e.value.status == status, str(e.value)


@needs_lib
@pytest.mark.parametrize("status,change", COMMON + LOSS + XENT)
def test_xent_refuses(status, change):
    a = args(change)
    refused(status, P.pbs_linear_xent, *(a[k] for k in "x w tokens vocab hidden targets loss lse ws n".split()), 0)


@needs_lib
@pytest.mark.parametrize("status,change", COMMON + GRAD + XENT)
def test_xent_grad_refuses(status, change):
    a = args(change)
    refused(status, P.pbs_linear_xent_grad,
            *(a[k] for k in "dloss x w tokens vocab hidden targets lse piece dx dw dw_fmt ws n".split()), 0)


@needs_lib
@pytest.mark.parametrize("status,change", COMMON + LOSS + TEACHER)
def test_distill_refuses(status, change):
    a = args(change)
    refused(status, P.pbs_linear_distill,
            *(a[k] for k in "x w tokens vocab hidden top_ids top_logits top_fmt top tau loss lse ws n".split()), 0)


@needs_lib
@pytest.mark.parametrize("status,change", COMMON + GRAD + TEACHER)
def test_distill_grad_refuses(status, change):
    a = args(change)
    refused(status, P.pbs_linear_distill_grad,
            *(a[k] for k in ("dloss x w tokens vocab hidden top_ids top_logits top_fmt top tau lse piece dx dw dw_fmt "
                             "ws n").split()), 0)


@needs_lib
def test_workspace_bytes():
    for status, change in SIZES + [(2, dict(top=-1)), (2, dict(top=1025)), (1, dict(piece=-5))]:
        a = args(change)
        refused(status, P.pbs_linear_loss_bytes, a["tokens"], a["vocab"], a["hidden"], a["top"], a["piece"])
    loss, grad = P.pbs_linear_loss_bytes(8192, 131072, 4096)
    # the loss keeps two numbers per 64 to 128 logits, and a gathered x
    assert loss < 8192 * 131072 * 8 / 64 + 2 * 8192 * 4096 + (1 << 20)
    # a piece of 4096 ids at a time: its dz, dx sums, a gathered x and what splits may take
    small = P.pbs_linear_loss_bytes(8192, 131072, 4096, 0, 4096)[1]
    assert small < grad and small < 8192 * 4096 * (2 + 2 + 4 * 4)
    # a piece of more than the vocabulary is the vocabulary, whatever the number
    assert P.pbs_linear_loss_bytes(300, 5000, 64, 0, (1 << 63) - 1) == P.pbs_linear_loss_bytes(300, 5000, 64, 0, 5000)
    # one byte short is refused
    a = args(dict(n=P.pbs_linear_loss_bytes(8, 100, 64)[0] - 1))
    refused(1, P.pbs_linear_xent, *(a[k] for k in "x w tokens vocab hidden targets loss lse ws n".split()), 0)


def test_pipeline_refuses():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(10, 64, dtype=torch.bfloat16)
    t, f = torch.zeros(4, dtype=torch.int64), torch.zeros(4)
    ids, logits = torch.zeros(4, 3, dtype=torch.int64), torch.zeros(4, 3)
    for bad in (lambda: PL.linear_xent(x, w, t),                            # not on a GPU
                lambda: PL.linear_xent(x.float(), w, t), lambda: PL.linear_xent(x, w.half(), t),
                lambda: PL.linear_xent(x, w[:, :32], t), lambda: PL.linear_xent(x[:, ::2], w[:, ::2], t),
                lambda: PL.linear_xent(x, w, t[:3]), lambda: PL.linear_xent(x, w, t.int()),
                lambda: PL.linear_xent(x, w, None), lambda: PL.linear_xent(x, w, t.repeat(2)[::2]),
                lambda: PL.linear_xent_grad(f[0].expand(4), x, w, t, f),
                lambda: PL.linear_xent_grad(f.double(), x, w, t, f),
                lambda: PL.linear_xent_grad(f, x, w, t, f[:2]), lambda: PL.linear_xent_grad(f, x, w, t, None),
                lambda: PL.linear_distill(x, w, ids[:, 0], logits), lambda: PL.linear_distill(x, w, ids.int(), logits),
                lambda: PL.linear_distill(x, w, ids, logits[:, :2]),
                lambda: PL.linear_distill(x, w, ids, logits.half()),
                lambda: PL.linear_distill(x, w, ids[:, :0], logits[:, :0]),
                lambda: PL.linear_distill_grad(f, x, w, ids[:3], logits[:3], 1.0, f)):
        with pytest.raises(ValueError):
            bad()


def test_reference_gradients_against_differences():
    g = torch.Generator().manual_seed(1)
    x, w = (torch.randn(n, 64, generator=g, dtype=torch.float64) * s for n, s in ((5, 1.0), (9, 0.2)))
    c = torch.randn(5, generator=g, dtype=torch.float64)
    targets = torch.tensor([3, -100, 0, 8, 3])
    ids = torch.tensor([[1, 2, -1], [0, 0, 4], [-1, -1, -1], [8, 7, 6], [5, -1, 5]])
    logits = torch.randn(5, 3, generator=g)
    for slots, tau in ((slots_of(targets), 1.0), (slots_of(None, ids, logits, 2.0), 2.0)):
        ref = head_ref(x, w, slots, tau, c)
        for t, name in ((x, "dx"), (w, "dw")):
            for at in ((0, 3), (1, 5), (2, 7), (4, 63)):
                ends = []
                for h in (1e-5, -1e-5):
                    moved = t.clone()
                    moved[at] += h
                    args = (moved if t is x else x, moved if t is w else w)
                    ends.append((head_ref(*args, slots, tau)["loss"][0] * c).sum())
                assert abs((ends[0] - ends[1]) / 2e-5 - ref[name][0][at]) < 1e-8


@needs_lib
def test_default_piece_is_a_gib_of_dz():
    """Without a piece the workspace is at most 1 GiB of dz (one or two terms, rows in whole tiles) and what the rest
    takes: x and dx of the tokens in 2 and 4 bytes, 64 MiB of splits and lists.  More than 2^18 tokens take 2048 ids all
    the same."""
    for tokens, vocab in ((1, 1 << 21), (1, 1 << 22), (17, 1 << 22), (100, 1 << 21), (128, 1 << 22), (129, 1 << 22),
                          (1000, 1 << 20), (20000, 1 << 18), (200000, 1 << 14), (1 << 18, 1 << 14)):
        most = (1 << 30) + (64 << 20) + (2 + 4) * tokens * 64
        assert P.pbs_linear_loss_bytes(tokens, vocab, 64)[1] <= most, (tokens, vocab)
    dz = 2 * (1 << 20) * 2048
    assert dz <= P.pbs_linear_loss_bytes(1 << 20, 5000, 64)[1] < dz + (1 << 30)


@needs_lib
def test_workspace_of_small_gradients():
    """Partial products take 16 splits of the tiles that a call has (128 x 128, whole rows of dx and dW) and no more."""
    for tokens, vocab, hidden, top in ((37, 2003, 256, 7), (1, 300, 64, 0), (100, 5000, 4096, 0), (700, 131, 64, 0)):
        rows, ids = (-(-n // 256) * 256 for n in (tokens, vocab))
        most = 16 * 4 * hidden * (rows + ids)                    # splits of dx and dW
        most += 4 * rows * ids + 2 * tokens * hidden             # dz, x of the live tokens
        most += tokens * (20 + 8 * (top + 3)) + 16 * 256         # lists, slots, alignment
        assert P.pbs_linear_loss_bytes(tokens, vocab, hidden, top)[1] <= most, (tokens, vocab, hidden)
