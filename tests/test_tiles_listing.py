"""The listings of the kernels that load to LDS, the gated block's and the orthogonalised update's: what the compiler does
not keep for asm statements, and what must not be in them."""
import os
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
