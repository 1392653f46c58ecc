"""The tolerances of tests/muon_parts.py on the CPU: an emulation of the parts' products stays inside them, and is outside as soon
as one product leaves out one part."""
import shutil

import pytest

from tests import muon_parts as parts
from tests.tile_choice import Choices

LOST = {0: ["x lo add"], 1: ["x lo gram", "x lo apply", "s lo add", "b lo apply"], 2: ["s lo poly"]}  # by the coefficients that show it


@pytest.mark.parametrize("rows,cols", [(96, 120), (300, 200), (672, 1300), (1000, 1030), (200, 9000)])
def test_a_lost_part_is_seen(rows, cols):
    u = parts.sparse_signs(rows, cols, 1, "cpu")
    for k, coefs in enumerate(parts.coefficients(rows, cols)):
        want, most = parts.expected(u, coefs)
        assert parts.off_by(parts.emulated(u, coefs), want, most) <= 1
        for part in LOST[k]:
            assert parts.off_by(parts.emulated(u, coefs, {part}), want, most) > 2, (coefs, part)


@pytest.mark.parametrize("batch,rows,cols", parts.SIZES)
def test_the_sizes_have_lo_parts(batch, rows, cols):
    """About as large a share of the hi parts as where a lost one is seen above, with 3.5 to 50 times the tolerance (X's 2.0e-4 at 672
    rows, S's 2.1e-4 at 300 x 200)."""
    _, x, s = parts.entries(rows, cols)
    assert x >= 1.7e-4 and s >= 1.3e-4


@pytest.mark.skipif(shutil.which("g++") is None, reason="no g++")
def test_the_sizes_reach_every_tile(tmp_path):
    choices = Choices(str(tmp_path))
    reached = {"gram": set(), "poly": set(), "apply": set()}
    turned = set()
    for batch, rows, cols in parts.SIZES:
        for product, (side, splits) in choices.orthogonalize(rows, cols, batch).items():
            reached[product].add((side, splits > 1))
            if product == "apply" and rows > cols:
                turned.add(side)
    for product in ("gram", "poly", "apply"):
        assert {side for side, _ in reached[product]} == {32, 64, 128, 192, 256}, (product, reached[product])
    assert {side for side, split in reached["gram"] if split} >= {128, 192, 256} and (192, True) in reached["poly"]
    assert turned >= {192, 256}
