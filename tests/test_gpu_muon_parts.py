"""The Newton-Schulz products in every tile on operands whose lo parts count (tests/muon_parts.py), and on values of any size."""
import math

import pytest
import torch

from tests import muon_parts as parts
from tests import muon_ref as ref
from tests import test_gpu_muon as muon

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def zs():
    import sharded_mixed_precision_rank_amd as zs

    return zs


@pytest.mark.parametrize("batch,rows,cols", parts.SIZES)
def test_products_keep_both_parts(zs, batch, rows, cols):
    u = torch.stack([parts.sparse_signs(rows, cols, 10 * rows + k, "cuda") for k in range(batch)])
    ws = muon.Guarded(zs, rows, cols, batch)
    out = torch.empty_like(u)
    again = (1.0, 0.0, 0.0)
    for coefs in parts.coefficients(rows, cols):
        wants = [parts.expected(v, coefs) for v in u]
        # alone, and behind a step that leaves X as it is, so through the parts that a step writes for the next one: another
        # 1.25 of 2^-22 and two roundings of 2^-24 for each factor of X (one in X, where `most` is as much; three in S X and five
        # in S^2 X, where it is 15 of 2^-22 and more)
        for steps in ([coefs], [again, coefs]):
            out.fill_(math.nan)
            zs.orthogonalize(u, out, ws.t, steps=len(steps), coefs=steps)
            for got, (want, most) in zip(out, wants):
                assert parts.off_by(got, want, most * (1 if len(steps) == 1 else 2)) <= 1, (coefs, len(steps))
    assert ws.untouched_outside()


@pytest.mark.parametrize("batch,rows,cols", [(1, 2006, 2006), (1, 1774, 9504), (1, 2818, 2818), (3, 2702, 2702), (1, 4090, 4096), (1, 11424, 672),
                                             (1, 5150, 5100)])
def test_default_steps_in_large_tiles(zs, batch, rows, cols):
    """Values of any size, one step, two and all five, against 64 bits."""
    x = muon.gradients(rows, batch, rows, cols)
    out = torch.empty_like(x)
    for steps in (1, 2, 5):
        zs.orthogonalize(x, out, steps=steps)
        for i in {0, batch - 1}:
            assert muon.off(out[i], ref.steps_of(x[i], steps)) <= ref.bound(steps, rows, cols), steps


@pytest.mark.parametrize("shape", [(11424, 672), (3, 5288, 2644), (2818, 2818)])
@pytest.mark.parametrize("nesterov", [False, True])
def test_the_update_in_large_tiles(zs, shape, nesterov):
    """Master and working copy from the last product's tiles of 192 and 256, turned and not, bit for bit."""
    muon.test_reduce_muon(zs, shape, 2, nesterov)


@pytest.mark.parametrize("rows,cols,stated", [(128, 128, 1.1e-6), (1001, 517, 2.4e-6), (4096, 4096, 3.2e-6), (11008, 4096, 4.5e-6)])
def test_five_default_steps_are_as_near_as_the_header_says(zs, rows, cols, stated):
    """Relative to the result's norm; a tenth more for other values than the header's."""
    x = muon.gradients(rows + cols, rows, cols)
    out = torch.empty_like(x)
    zs.orthogonalize(x, out)
    want = ref.steps_of(x)
    assert ((out.double() - want).norm() / want.norm()).item() <= 1.1 * stated
