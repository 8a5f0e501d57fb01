"""Refusals of the orthogonalisation and Muon's update, on the CPU: nothing is enqueued."""
import os

import pytest
import torch

import precision_block_scaled_amd as P
from precision_block_scaled_amd import pipeline as PL

pytestmark = pytest.mark.skipif(not os.path.exists(P.lib_path), reason="libpbs.so is not built")

BF, F32 = P.PBS_FMT_BF16, P.PBS_FMT_F32
A = 1 << 20                     # addresses that no call reads
STEPS = PL.MUON_STEPS
ORTHO = dict(x=A, x_fmt=F32, ldx=96, x_batch_stride=96 * 64, batch=2, rows=64, cols=96, coefficients=STEPS, eps=1e-7, y=2 * A,
             ldy=96, y_batch_stride=96 * 64, workspace=3 * A, workspace_bytes=1 << 30, stream=0)
BAD = [
    (dict(x_fmt=P.PBS_FMT_E4M3), 3, "BF16 or F32"), (dict(x=None), 1, "x is null"), (dict(y=None), 1, "y is null"),
    (dict(x=A + 2), 1, "aligned"), (dict(y=2 * A + 1), 1, "aligned"), (dict(batch=-1), 2, "batch"), (dict(batch=65536), 2, "batch"),
    (dict(rows=-1), 2, "sides"), (dict(rows=40000, cols=40000), 2, "sides"), (dict(cols=(1 << 20) + 1), 2, "sides"),
    (dict(batch=60000, rows=1 << 14, cols=1 << 14), 2, "too many"), (dict(ldx=-1), 2, "strides"),
    (dict(ldy=95), 2, "overlap"), (dict(y_batch_stride=0), 2, "overlap"), (dict(y_batch_stride=96 * 63), 2, "overlap"),
    (dict(ldy=192, y_batch_stride=97), 2, "overlap"), (dict(coefficients=()), 1, "steps"), (dict(coefficients=STEPS * 13), 1, "steps"),
    (dict(coefficients=((float("nan"), 0, 0),)), 1, "not finite"), (dict(coefficients=((1e30, 0, 0),)), 1, "range"),
    (dict(coefficients=((10.0, 0, 0),) * 5), 1, "range"), (dict(eps=-1.0), 1, "eps"), (dict(eps=float("nan")), 1, "eps"),
    (dict(workspace=None), 1, "workspace"), (dict(workspace=3 * A + 128), 1, "workspace"), (dict(workspace_bytes=100), 1, "workspace"),
    (dict(y=A), 1, "another type"), (dict(y=3 * A), 1, "workspace's memory"),
]


@pytest.mark.parametrize("change,status,text", BAD, ids=lambda v: str(v)[:40])
def test_orthogonalize_refusals(change, status, text):
    with pytest.raises(P.PBSError, match=text) as e:
        P.pbs_orthogonalize(**{**ORTHO, **change})
    assert e.value.status == status


MUON = dict(w=A, w_fmt=BF, ldw=96, w_batch_stride=96 * 64, momentum=2 * A, m_fmt=F32, ldm=96, m_batch_stride=96 * 64, grad=3 * A,
            g_fmt=BF, grad_transposed=0, ldg=96, g_batch_stride=96 * 64, batch=2, rows=64, cols=96, beta=0.95, nesterov=1, lr=0.02,
            lr_factor=None, weight_decay=0.1, scale=1.0, coefficients=STEPS, eps=1e-7, workspace=4 * A, workspace_bytes=1 << 30,
            stream=0)
MUON_BAD = [
    (dict(w_fmt=P.PBS_FMT_E5M2), 3, "w must"), (dict(m_fmt=7), 3, "momentum must"), (dict(g_fmt=P.PBS_FMT_E2M1), 3, "grad must"),
    (dict(w=None), 1, "w is null"), (dict(momentum=None), 1, "momentum is null"), (dict(grad=None), 1, "grad is null"),
    (dict(w=2 * A), 1, "apart"), (dict(grad=A), 1, "apart"), (dict(momentum=3 * A), 1, "apart"), (dict(momentum=4 * A), 1, "workspace's"),
    (dict(beta=-0.1), 1, "beta"), (dict(beta=1.1), 1, "beta"), (dict(beta=float("nan")), 1, "beta"), (dict(lr=float("inf")), 1, "lr"),
    (dict(weight_decay=float("nan")), 1, "lr"), (dict(scale=float("inf")), 1, "lr"), (dict(lr_factor=A + 2), 1, "lr_factor"),
    (dict(ldw=90), 2, "overlap"), (dict(m_batch_stride=96), 2, "overlap"), (dict(workspace_bytes=0), 1, "workspace"),
    (dict(coefficients=((100.0, 100.0, 100.0),) * 3), 1, "range"), (dict(rows=1 << 21), 2, "sides"),
]


@pytest.mark.parametrize("change,status,text", MUON_BAD, ids=lambda v: str(v)[:40])
def test_muon_refusals(change, status, text):
    with pytest.raises(P.PBSError, match=text) as e:
        P.pbs_muon(**{**MUON, **change})
    assert e.value.status == status


def test_nothing_to_do():
    """An empty batch or matrix needs no pointers."""
    for change in (dict(batch=0), dict(rows=0), dict(cols=0)):
        assert P.pbs_orthogonalize_bytes(*({**dict(batch=2, rows=64, cols=96), **change}).values()) == 0
        P.pbs_orthogonalize(**{**ORTHO, **change, "x": None, "y": None, "workspace": None, "workspace_bytes": 0})
        P.pbs_muon(**{**MUON, **change, "w": None, "momentum": None, "grad": None, "workspace": None, "workspace_bytes": 0})


def test_python_refusals():
    x = torch.zeros(4, 6)
    for t in (x[0], x.double(), x[:, ::2], torch.zeros(2, 2, 4, 6)):
        with pytest.raises(ValueError):
            PL.orthogonalize(t)
    with pytest.raises(ValueError):
        PL.orthogonalize(x, y=x)
    with pytest.raises(ValueError):
        PL.orthogonalize(x, y=torch.zeros(6, 4, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        PL.orthogonalize(x.bfloat16()[:, :4], y=x.bfloat16()[:, :5])
    for change in (dict(w=x.t()), dict(momentum=x[:3]), dict(momentum=x.double()), dict(grad=x.t()), dict(grad=torch.zeros(4, 12)[:, ::2]),
                   dict(lr=torch.zeros(2)), dict(lr=torch.zeros(1, dtype=torch.float64)), dict(grad=x.half())):
        with pytest.raises(ValueError):
            PL.muon(**{**dict(w=x, momentum=x.clone(), grad=x.clone(), lr=0.1), **change})
    with pytest.raises(ValueError, match="on the GPU"):
        PL.orthogonalize(x)
    with pytest.raises(ValueError, match="on the GPU"):
        PL.muon(x, x.clone(), x.clone(), 0.1)
    with pytest.raises(ValueError, match="for each step"):
        P.pbs_orthogonalize(**{**ORTHO, "coefficients": ((1.0, 2.0),)})


@pytest.mark.parametrize("change", [dict(ldy=128), dict(ldx=128, x_batch_stride=128 * 64), dict(y_batch_stride=96 * 65),
                                    dict(x_batch_stride=0)], ids=str)
def test_in_place_with_other_strides(change):
    """Rows that are written where other rows are still to be read."""
    same = dict(x_fmt=BF, y=A, y_batch_stride=96 * 64)
    if "ldy" in change:
        change = dict(change, y_batch_stride=128 * 64)
    with pytest.raises(P.PBSError, match="other strides") as e:
        P.pbs_orthogonalize(**{**ORTHO, **same, **change})
    assert e.value.status == 1


def test_coefficients_that_change_in_place():
    """A step's numbers are taken as they are at the call, whatever holds them."""
    a = torch.tensor(1.5)
    steps = ((a, -0.5, 0.0),)
    first, n = P._triples(steps)
    assert n == 1 and list(first) == [1.5, -0.5, 0.0]
    a.fill_(2.0)
    assert list(P._triples(steps)[0]) == [2.0, -0.5, 0.0]
    assert list(P._triples(torch.tensor([[1.0, 2.0, 3.0]]))[0]) == [1.0, 2.0, 3.0]


def test_workspaces_hold_what_is_used():
    """Small matrices need none to speak of; short sides their Gram matrices' tiles and a copy in 64 bits; the others two X and a
    few matrices of the shorter side, 16 bits each."""
    need = P.pbs_orthogonalize_bytes
    assert need(65535, 64, 256) <= 256 and need(1, 33, 65) <= 256
    assert need(65535, 3, 5) <= 65535 * (2 * 16 * 16 * 8 + 3 * 5 * 8 + 8) + 4 * 256
    assert need(1, 16, 4096) <= 33 * 16 * 16 * 8 + 16 * 4096 * 8 + 4 * 256
    assert need(1, 64, 1 << 20) <= 16 * 10 * 256 * 8 + 64 * 64 * 8 + (64 << 20) * 8 + 4 * 256
    assert need(1, 4096, 4096) <= (8 + 2 * 2) * 4096 ** 2 + (1 << 20)
    assert need(1, 4096, 16384) <= 8 * 4096 * 16384 + 5 * 2 * 4096 ** 2 + (1 << 20)
