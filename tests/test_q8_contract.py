"""The 8-bit training operators on the CPU: what their sources, header and argument checks promise."""
import os
import random
import re
import shutil
import subprocess

import pytest

import sharded_mixed_precision_rank_amd as zs
from sharded_mixed_precision_rank_amd import build

LIB = zs.library()
A = 0x7F0000000000  # never dereferenced: every call here fails before any HIP call
MB = 1 << 20
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sharded_mixed_precision_rank_amd", "csrc")


def inline_asm():
    """(file, text) of every asm statement of the library's device sources, up to its closing bracket."""
    for name in sorted(os.listdir(CSRC)):
        if not name.endswith((".hip", ".h")):
            continue
        src = open(os.path.join(CSRC, name), encoding="utf-8").read()
        for m in re.finditer(r"\basm\s*(?:volatile\s*)?\(", src):
            depth, i = 1, m.end()
            quoted = False
            while depth:
                c = src[i]
                if c == '"' and src[i - 1] != "\\":
                    quoted = not quoted
                elif not quoted:
                    depth += (c == "(") - (c == ")")
                i += 1
            yield name, src[m.end():i - 1]


def test_loads_to_lds_take_m0_as_an_operand():
    """A statement that writes m0 by itself, without the compiler's knowledge, could land between the compiler's own
    write and its use; and a load to LDS has to have m0 from somewhere."""
    found = 0
    for name, text in inline_asm():
        template = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', text.split(" : ")[0]))
        for instruction in template.replace("\\t", "").split("\\n"):
            assert not re.match(r"\s*\w+\s+m0\b", instruction), (name, instruction)
            if re.search(r"\blds$", instruction):
                assert '"{m0}"' in text, (name, instruction)
                found += 1
    assert found == 2


def _scalars(text):
    """Numbers of the scalar registers named in an instruction's operands."""
    out = set()
    for lo, hi, one in re.findall(r"\bs\[(\d+):(\d+)\]|\bs(\d+)\b", text):
        out |= {int(one)} if one else set(range(int(lo), int(hi) + 1))
    return out


def too_early(listing):
    """Memory instructions that read a scalar register less than five wait states after a vector instruction wrote it
    (in the listing's order; a label starts afresh)."""
    written, bad = [], []
    for line in listing.splitlines():
        text = line.split(";")[0].strip()
        if re.match(r"^[\w.$]+:", text):
            written = []
        if not text or text.startswith(".") or text.endswith(":"):
            continue
        op, _, operands = text.partition(" ")
        if op.startswith(("buffer_", "global_", "flat_", "scratch_")):
            used = _scalars(operands)
            if any(used & regs for _, regs in written):
                bad.append(text)
        states = int(operands, 0) + 1 if op == "s_nop" else 1
        written = [(age + states, regs) for age, regs in written if age + states < 5]
        if op.startswith("v_"):
            regs = _scalars(operands.split(",")[0])
            if regs:
                written.append((0, regs))
    return bad


def test_too_early_finds_what_it_looks_for():
    early = "k:\n\tv_readfirstlane_b32 s4, v0\n\ts_mov_b32 m0, s9\n\ts_nop 0\n\tbuffer_load_dwordx4 v1, s[4:7], 0 offen lds\n"
    assert len(too_early(early)) == 1
    assert not too_early(early.replace("s_nop 0", "s_nop 3")) and not too_early(early.replace("s4, v0", "s8, v0"))


@pytest.mark.skipif(shutil.which("hipcc") is None, reason="no hipcc")
def test_no_load_takes_a_descriptor_just_written_by_a_vector_instruction(tmp_path):
    """The compiler keeps that distance for its own instructions, not for those in asm statements: the listing of the
    kernels that load to LDS."""
    out = str(tmp_path / "gemm.s")
    flags = [f for f in build.FLAGS if f != "-shared"]
    subprocess.run(["hipcc", *flags, "-S", "--cuda-device-only", "-x", "hip", os.path.join(CSRC, "zs_q8_gemm.hip"), "-o", out],
                   check=True, stdout=subprocess.DEVNULL, stderr=subprocess.DEVNULL)
    listing = open(out, encoding="utf-8").read()
    assert listing.count(" lds\n") > 100
    assert not too_early(listing)


def _shared(a, b):
    """Whether two matrices (base, rows, bytes a row, pitch) share a byte, by their bytes."""
    bytes_of = lambda base, rows, width, pitch: {base + r * pitch + k for r in range(rows) for k in range(width)}  # noqa: E731
    return bool(bytes_of(*a) & bytes_of(*b))


def test_a_single_row_may_lie_between_the_rows_of_a_matrix():
    """An output is refused where it shares a byte with an input, not where it lies in a gap between its rows.  One
    token's product y beside the weight's rows; w_scales is y itself, so that every call is refused before it launches
    anything, and the message says for which of the two."""
    rng = random.Random(1)
    met = {False: 0, True: 0}
    for _ in range(4000):
        n, k = rng.randint(1, 6), rng.randint(1, 12)
        ld = k + rng.choice((0, 1, rng.randint(1, 40)))
        at = A + rng.randint(-40, n * ld + 8) // 4 * 4
        status = LIB.zs_q8_matmul(A + MB, k, A + 2 * MB, A, ld, at, 1, n, k, 0, at, 0, n, None)
        message = LIB.zs_last_error().decode()
        want = _shared((at, 1, 2 * n, 2 * n), (A, n, k, ld))
        assert zs.STATUS[status] == "ZS_ERR_ALIAS", message
        assert ("overlaps w_codes" in message) == want, (n, k, ld, at - A, message)
        assert want or "overlaps w_scales" in message
        met[want] += 1
    assert min(met.values()) > 300


def test_a_vector_may_lie_between_the_rows_of_a_matrix():
    """The scales somewhere about x's rows; the column factors are the scales themselves, which is refused last."""
    rng = random.Random(2)
    met = {False: 0, True: 0}
    for _ in range(4000):
        rows, cols = rng.randint(2, 6), rng.randint(1, 12)
        ld = cols + rng.choice((0, 1, rng.randint(1, 40)))
        at = A + rng.randint(-40, rows * ld * 2 + 8) // 4 * 4
        status = LIB.zs_q8_save(A, 0, ld, rows, cols, at, 0, A + MB, cols, at, None)
        message = LIB.zs_last_error().decode()
        want = _shared((at, 1, 4 * rows, 4 * rows), (A, rows, 2 * cols, 2 * ld))
        assert zs.STATUS[status] == "ZS_ERR_ALIAS", message
        assert ("scales overlaps x" in message) == want, (rows, cols, ld, at - A, message)
        assert want or "scales overlaps col_scale" in message
        met[want] += 1
    assert min(met.values()) > 300


def test_rows_at_different_distances_are_refused_where_their_ranges_meet():
    """Two matrices of several rows: told apart where their rows lie at the same distance, refused otherwise."""
    codes = dict(x=A + 64, T=4, K=16)
    for ld_y, want in ((32, "ZS_ERR_ALIAS"), (64, "ZS_ERR_ALIAS")):
        status = LIB.zs_q8_matmul(codes["x"], 128, A + MB, A + 2 * MB, 16, A, 4, 8, 16, 0, A, 0, ld_y, None)
        message = LIB.zs_last_error().decode()
        assert zs.STATUS[status] == want
        assert ("overlaps x_codes" in message) == (ld_y != 64), message
