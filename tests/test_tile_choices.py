"""Which kernels the sizes of the GPU tests reach, by the rules that the launches go by: a change of a rule that takes a
kernel out of those tests fails here."""
import shutil

import pytest

from tests import test_gpu_glu, test_gpu_muon
from tests.tile_choice import Choices

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="no g++")


@pytest.fixture(scope="module")
def choices(tmp_path_factory):
    return Choices(str(tmp_path_factory.mktemp("choices")))


def parametrized(test):
    """The sizes of a test's parametrisation whose values are tuples or lists of whole numbers."""
    return [m.args[1] for m in test.pytestmark if m.name == "parametrize" and isinstance(m.args[1][0], tuple)
            and all(isinstance(v, int) for v in m.args[1][0])][0]


@pytest.mark.parametrize("op,test,kernels", [
    ("forward", test_gpu_glu.test_forward_of_whole_numbers, {"few", "64x32", "64", "128", "192", "256"}),
    ("input", test_gpu_glu.test_input_grad_of_whole_numbers, {"split", "32", "64x128", "128", "128 near", "256"}),
    ("weight", test_gpu_glu.test_weight_grad_of_whole_numbers, {"64", "128", "128 near", "256"})])
def test_every_kernel_of_the_gated_block_is_tested(choices, op, test, kernels):
    """In the layouts with rows on 4-byte boundaries, and in the one without."""
    assert {choices.glu(op, *s) for s in parametrized(test)} == kernels
    assert {choices.glu(op, *s, direct=False) for s in parametrized(test)} == {"any", "through"}


def test_every_tile_of_the_orthogonalised_update_is_tested(choices):
    """With sums of whole numbers: each tile in each product that takes it, split sums too."""
    sizes = [(*s, 1) for s in parametrized(test_gpu_muon.test_exact_products)]
    sizes += [(*s, 1) for s in parametrized(test_gpu_muon.test_exact_products_of_large_matrices)]
    sizes += [(r, c, b) for b, r, c in parametrized(test_gpu_muon.test_exact_products_of_stacks)]
    reached = {}
    for s in sizes:
        for product, (side, splits) in choices.orthogonalize(*s).items():
            reached.setdefault(product, set()).add((side, splits > 1))
    assert {side for side, _ in reached["gram"]} == {32, 64, 128, 192, 256} == {side for side, split in reached["gram"] if split}
    assert {side for side, _ in reached["poly"]} == {32, 64, 128, 192, 256}
    assert {side for side, _ in reached["apply"]} == {32, 64, 128, 192, 256}


def test_large_products_keep_the_direct_loads(choices):
    """However many small tiles the outputs are (800,000 tokens: 8.8e9 outputs), as long as large ones fit a grid; past that
    the kernel that goes round."""
    for op in ("forward", "input", "weight"):
        for M, N, K in ((800_000, 11008, 4096), (800_000, 11008, 64), (4_000_000, 4096, 1376), (300_000, 32768, 64)):
            assert choices.glu(op, M, N, K) in ("128", "128 near", "192", "256"), (op, M, N, K)
        assert choices.glu(op, 2 ** 31 - 1, 2 ** 31 - 1, 64) == "any"
