"""The listings of the kernels that load to LDS, the gated block's and the orthogonalised update's: what the compiler does
not keep for asm statements, and what must not be in them."""
import os
import re
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from sharded_mixed_precision_rank_amd import build
from tests.test_q8_contract import CSRC, too_early

FILES = ("zs_glu_gemm.hip", "zs_muon.hip")


@pytest.fixture(scope="module")
def listings(tmp_path_factory):
    if shutil.which("hipcc") is None:
        pytest.skip("no hipcc")
    to = tmp_path_factory.mktemp("listings")

    def make(name):
        out = str(to / (name + ".s"))
        subprocess.run(["hipcc", *build.FLAGS, "-S", "--cuda-device-only", "-x", "hip", os.path.join(CSRC, name), "-o", out], check=True,
                       stdout=subprocess.DEVNULL, stderr=subprocess.DEVNULL)
        return open(out, encoding="utf-8").read()

    with ThreadPoolExecutor(len(FILES)) as pool:
        return dict(zip(FILES, pool.map(make, FILES)))


@pytest.mark.parametrize("name", FILES)
def test_no_load_takes_a_descriptor_just_written_by_a_vector_instruction(listings, name):
    assert listings[name].count(" lds\n") > 100
    assert not too_early(listings[name])


@pytest.mark.parametrize("name", FILES)
def test_no_packed_fp32_instructions_and_no_spills(listings, name):
    for word in ("v_pk_add_f32", "v_pk_mul_f32", "v_pk_fma_f32", "scratch_load", "scratch_store"):
        assert word not in listings[name]


OTHERS = ("zs_glu_rows.hip", "zs_muon_small.hip")


@pytest.fixture(scope="module")
def all_listings(listings, tmp_path_factory):
    to = tmp_path_factory.mktemp("others")

    def make(name):
        out = str(to / (name + ".s"))
        flags = [f for f in build.FLAGS if f != "-shared"]
        subprocess.run(["hipcc", *flags, "-S", "--cuda-device-only", "-x", "hip", os.path.join(CSRC, name), "-o", out], check=True,
                       stdout=subprocess.DEVNULL, stderr=subprocess.DEVNULL)
        return open(out, encoding="utf-8").read()

    with ThreadPoolExecutor(len(OTHERS)) as pool:
        return {**listings, **dict(zip(OTHERS, pool.map(make, OTHERS)))}


def spills(listing):
    """{kernel: (vector registers spilled, scalar ones, bytes of scratch)}, from the listing's metadata."""
    out = {}
    for block in listing.split("amdhsa.kernels:")[1].split("- .agpr_count:")[1:]:
        number = lambda key: int(re.search(rf"\.{key}:\s+(\d+)", block).group(1))  # noqa: E731
        name = re.search(r"\.name:\s+(\S+)", block).group(1)
        out[name] = (number("vgpr_spill_count"), number("sgpr_spill_count"), number("private_segment_fixed_size"))
    return out


@pytest.mark.parametrize("name", FILES + OTHERS)
def test_no_vector_spills_and_few_scalar_ones(all_listings, name):
    """Spilled scalar registers go to lanes of vector registers, without a trace among the scratch instructions.  glu_any, the
    kernel of few tiles with rows at any address, holds the addresses and bounds of four stages that way."""
    found = spills(all_listings[name])
    assert found
    for kernel, (vector, scalar, scratch) in found.items():
        assert vector == 0 and scratch == 0, kernel
        assert scalar <= (128 if "glu_any" in kernel else 4), (kernel, scalar)
    for word in ("v_pk_add_f32", "v_pk_mul_f32", "v_pk_fma_f32"):
        assert word not in all_listings[name]
