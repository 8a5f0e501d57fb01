"""Which steps the orthogonalisation takes, on the CPU: an empty batch goes through all checks of the coefficients."""
import os

import pytest

import precision_block_scaled_amd as P
from precision_block_scaled_amd import pipeline as PL

pytestmark = pytest.mark.skipif(not os.path.exists(P.lib_path), reason="libpbs.so is not built")

# Polynomials of steps whose range shrinks from [1e-3, 1], as the Polar Express paper (Amsel et al., 2025) tabulates them:
# largest values 1.99, 1.97, 1.87, 1.56, 1.12, 1.00, 1.00, each reached again at the end of its range, on a rise of 12 times it
RISING = ((8.28721201814563, -23.595886519098837, 17.300387312530933), (4.107059111542203, -2.9478499167379106, 0.5448431082926601),
          (3.9486908534822946, -2.908902115962949, 0.5518191394370137), (3.3184196573706015, -2.488488024314874, 0.51004894012372),
          (2.300652019954817, -1.6689039845747493, 0.4188073119525673), (1.891301407787398, -1.2679958271945868, 0.37680408948524835),
          (1.875, -1.25, 0.375))


def within(steps, f=1.01):
    """The steps with their arguments a little within their ranges, but for the last."""
    return tuple((a / f, b / f ** 3, c / f ** 5) for a, b, c in steps[:-1]) + steps[-1:]


def take(steps):
    P.pbs_orthogonalize(None, P.PBS_FMT_F32, 96, 0, 0, 64, 96, steps, 1e-7, None, 96, 0, None, 0, 0)


@pytest.mark.parametrize("steps", [within(RISING), within(RISING)[:4], within(RISING) + RISING[-1:] * 57, RISING[:3],
                                   PL.MUON_STEPS, PL.MUON_STEPS[:1] * 64, ((1.5, -0.5, 0.0),) * 64, ((1.875, -1.25, 0.375),) * 64,
                                   ((8.0, -20.0, 13.0),) * 2, ((0.0, 0.0, 0.0),), ((0.0, 0.0, 1.0),) * 4, ((1.0, 0.0, 0.0),) * 64,
                                   ((4000.0, 0.0, 0.0),), ((1.0, 0.0, 4000.0),), ((-2.0, 1.0, 0.0),) * 40], ids=lambda s: str(len(s)))
def test_taken(steps):
    take(steps)


@pytest.mark.parametrize("steps,at", [(RISING, 5), (((5000.0, 0.0, 0.0),), 0), (((70.0, 0.0, 0.0),) * 2, 1), (((60.0, 0.0, 0.0),) * 3, 2),
                                      (((0.0, 1e38, -1e38),), 0), (((1.0, -2e4, 2e4),), 0), (((3.0, 0.0, 0.0),) * 20, 4),
                                      (((1.5, -0.5, 0.0), (2.5, 0.0, 0.0), (1.5, -0.5, 0.0), (1.5, -0.5, 0.0), (1.5, -0.5, 0.0)), 4)],
                         ids=lambda s: str(s)[:30])
def test_refused(steps, at):
    """Steps that carry a singular value of [0, 1], or one that roundings have moved by 2^-10, or its square, past 4096."""
    with pytest.raises(P.PBSError, match=rf"step {at}\)") as e:
        take(steps)
    assert e.value.status == 1
