"""Layer norm: what the calls refuse, before anything is enqueued (CPU)."""
import os

import pytest
import torch

import precision_block_scaled_amd as P
from precision_block_scaled_amd import pipeline as PL
from tests.norm_ref import norm_grad_ref, norm_ref

FAKE = 1 << 40          # a non-null, aligned address never dereferenced
BF, F32 = P.PBS_FMT_BF16, P.PBS_FMT_F32

needs_lib = pytest.mark.skipif(not os.path.exists(P.lib_path), reason="libpbs.so not built")


def _expect(status, fn, *args):
    with pytest.raises(P.PBSError) as e:
        fn(*args)
    assert e.value.status == status, str(e.value)


def forward(x=FAKE, x_fmt=BF, rows=4, cols=64, ldx=64, gamma=None, beta=None, w_fmt=BF, eps=1e-5, y=FAKE, y_fmt=BF,
            ldy=64, mean=None, rstd=None, amax=None):
    return (x, x_fmt, rows, cols, ldx, gamma, beta, w_fmt, eps, y, y_fmt, ldy, mean, rstd, amax, 0)


def grad(dy=FAKE, y_fmt=BF, lddy=64, x=FAKE, x_fmt=BF, ldx=64, rows=4, cols=64, gamma=None, w_fmt=BF, mean=FAKE,
         rstd=FAKE, dx=FAKE, lddx=64, dgamma=FAKE, dbeta=FAKE, ws=FAKE, n=1 << 30):
    return (dy, y_fmt, lddy, x, x_fmt, ldx, rows, cols, gamma, w_fmt, mean, rstd, dx, lddx, dgamma, dbeta, ws, n, 0)


@needs_lib
@pytest.mark.parametrize("status,change", [
    (3, dict(x_fmt=P.PBS_FMT_E4M3)), (3, dict(y_fmt=P.PBS_FMT_E2M1)), (3, dict(w_fmt=P.PBS_FMT_E5M2)),
    (2, dict(rows=-1)), (2, dict(cols=0)), (2, dict(cols=(1 << 24) + 1, ldx=1 << 25, ldy=1 << 25)),
    (2, dict(ldx=63)), (2, dict(ldy=63)), (2, dict(ldx=0)), (2, dict(ldx=-64)),
    (1, dict(x=None)), (1, dict(y=None)), (1, dict(x=FAKE + 1)), (1, dict(x=FAKE + 2, x_fmt=F32)),
    (1, dict(y=FAKE + 2, y_fmt=F32)), (1, dict(gamma=FAKE + 1)), (1, dict(beta=FAKE + 2, w_fmt=F32)),
    (1, dict(mean=FAKE + 2)), (1, dict(rstd=FAKE + 1)), (1, dict(amax=FAKE + 2)),
    # y on x's memory in another type or with other rows: not in place
    (1, dict(y=FAKE, y_fmt=F32)), (1, dict(y=FAKE, ldy=65)),
    (1, dict(eps=-1.0)), (1, dict(eps=float("nan"))), (1, dict(eps=float("inf")))])
def test_layernorm_refuses(status, change):
    _expect(status, P.pbs_layernorm, *forward(**change))


@needs_lib
@pytest.mark.parametrize("status,change", [
    (3, dict(x_fmt=P.PBS_FMT_E4M3)), (3, dict(y_fmt=P.PBS_FMT_E4M3)), (3, dict(w_fmt=7)),
    (2, dict(rows=-1)), (2, dict(cols=0)), (2, dict(lddy=63)), (2, dict(ldx=1)), (2, dict(lddx=63)),
    (1, dict(dy=None)), (1, dict(x=None)), (1, dict(mean=None)), (1, dict(rstd=None)),
    (1, dict(dy=FAKE + 1)), (1, dict(dx=FAKE + 1)), (1, dict(dgamma=FAKE + 2)), (1, dict(dbeta=FAKE + 2)),
    (1, dict(ws=None)), (1, dict(ws=FAKE + 8)), (1, dict(n=0)), (1, dict(n=2 * 64 * 4 - 1)),
    # dx on x's or dy's memory in another type or with other rows
    (1, dict(x=FAKE, lddx=65)), (1, dict(dy=FAKE, y_fmt=F32, x=2 * FAKE)), (1, dict(dy=FAKE, lddx=65, x=2 * FAKE))])
def test_layernorm_grad_refuses(status, change):
    _expect(status, P.pbs_layernorm_grad, *grad(**change))


@needs_lib
def test_layernorm_grad_bytes():
    assert P.pbs_layernorm_grad_bytes(4, 64) >= 2 * 64 * 4
    assert P.pbs_layernorm_grad_bytes(0, 1) >= 0
    _expect(2, P.pbs_layernorm_grad_bytes, 4, 0)
    _expect(2, P.pbs_layernorm_grad_bytes, -1, 64)


def test_pipeline_refuses():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for bad in (lambda: PL.layernorm(x),                                   # not on a GPU
                lambda: PL.layernorm(x.half()), lambda: PL.layernorm(x[0]), lambda: PL.layernorm(x.t()),
                lambda: PL.layernorm(x[:, :0]), lambda: PL.layernorm(x[:1].expand(4, 64)),
                lambda: PL.layernorm(x, torch.ones(63)), lambda: PL.layernorm(x, torch.ones(64, dtype=torch.half)),
                lambda: PL.layernorm(x, torch.ones(64), torch.ones(64).bfloat16()),
                lambda: PL.layernorm(x, torch.ones(128)[::2]),
                lambda: PL.layernorm(x, amax=torch.zeros(2)), lambda: PL.layernorm(x, amax=torch.zeros(1).double()),
                lambda: PL.layernorm(x, y=x, out_dtype=torch.float32),
                lambda: PL.layernorm_grad(x[:3], x, None, torch.zeros(4), torch.zeros(4)),
                lambda: PL.layernorm_grad(x, x, None, torch.zeros(3), torch.zeros(4)),
                lambda: PL.layernorm_grad(x, x, None, torch.zeros(4), None),
                lambda: PL.layernorm_grad(x, x, None, torch.zeros(4), torch.zeros(4).bfloat16())):
        with pytest.raises(ValueError):
            bad()


def test_reference_gradient_against_differences():
    """The 64-bit reference itself: its gradients against central differences of its forward pass."""
    g = torch.Generator().manual_seed(5)
    x, c = (torch.randn(3, 11, generator=g, dtype=torch.float64) for _ in range(2))
    gamma, beta = (torch.randn(11, generator=g, dtype=torch.float64) for _ in range(2))
    eps, h = 1e-3, 1e-5

    def value(x, gamma, beta):
        return (norm_ref(x, gamma, beta, eps, torch.float32)[0] * c).sum()

    mu, r = (norm_ref(x, gamma, beta, eps, torch.float32)[i] for i in (2, 4))
    dx, _, dg, _, db, _ = norm_grad_ref(c, x, gamma, mu, r, torch.float32)
    for t, want, at in ((x, dx, (1, 4)), (x, dx, (2, 10)), (gamma, dg, (3,)), (beta, db, (7,))):
        up, down = t.clone(), t.clone()
        up[at] += h
        down[at] -= h
        args = [[u if v is t else v for v in (x, gamma, beta)] for u in (up, down)]
        assert abs((value(*args[0]) - value(*args[1])) / (2 * h) - want[at]) < 1e-7
