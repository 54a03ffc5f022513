"""GPU: sigmoid scores of logits so low that fp32 holds them as denormals or not at all, in the form of
one block, of a warp and of four lanes per token."""
import math

import pytest
import torch

import fused_reference as R

pytestmark = pytest.mark.gpu

# scores e^l / (1 + e^l) from normal numbers through fp32's denormals (e^-89 .. e^-103.9) to below them
ROWS = [[-88, -89, -90, -91, -95], [-95, -96, -97, -98, -99], [-100, -101, -100, -102, -103], [-103, -104, -110, -103, -200],
        [-150, -151, -149, -150, -699], [-690, -650.5, -660, -640, -699], [-705, -1, -800, -2, -95], [0, -95, -103, 5, -120],
        [-701, -800, -900, -5000, -702], [-89, -math.inf, -95, -math.inf, -math.inf]]


def _logits(T, E, dtype):
    x = torch.full((T, E), -math.inf, dtype=dtype)
    at = torch.randperm(E, generator=torch.Generator().manual_seed(E))[:5]
    x[:, at] = torch.tensor(ROWS, dtype=dtype).repeat(T // len(ROWS) + 1, 1)[:T]
    return x


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("T,E", [(10, 5), (100, 5), (100, 70), (10, 300), (6500, 70)])
@pytest.mark.parametrize("renorm", [True, False])
def test_sigmoid_scores_of_low_logits(lib, dtype, T, E, renorm):
    """Renormalised, weights depend on the differences of the logits, not on their level; else they are the
    fp32 score.  Two exponentials (a unit and the argument's half unit each), a quotient, the sum of 3 and its
    quotient: 2^-16 relative is far more; a denormal is off by two units of 2^-149 and its rounding."""
    x = _logits(T, E, dtype)
    r = lib.moe_route(x.cuda(), 3, scoring="sigmoid", renormalize=renorm)
    torch.cuda.synchronize()
    w, experts, offsets, rows, positions = R.route64(x, 3, "sigmoid", renorm)
    assert r.experts.tolist() == experts and r.offsets.tolist() == offsets
    assert r.rows.tolist() == rows and r.positions.tolist() == positions
    w = torch.tensor(w, dtype=torch.float64)
    got = r.weights.double().cpu()
    assert ((got - w).abs() <= 2.0 ** -16 * w + 3 * 2.0 ** -149).all()
    if renorm:
        live = torch.tensor([max(row) > -700 for row in x.tolist()])
        assert ((got.sum(1) - live.double()).abs() <= 2.0 ** -20).all()
