"""Checks of the compiled gfx950 device code of linear attention and of the
processing of logits (no GPU needed; needs hipcc): the properties that
test_device_code_serving.py checks of its kernels."""
import os
import re
import shutil
import subprocess

import pytest

from kda_chunked_delta_amd import build as kbuild
from test_device_code import SCC_READERS, SCC_WRITERS, mfma_shape_changes
from test_device_code_serving import kernels, unawaited_lds_loads

SOURCES = ("linear_attention.hip", "logits.hip")


@pytest.fixture(scope="module")
def linear_asm(tmp_path_factory):
    if not os.path.exists(kbuild.HIPCC) and shutil.which("hipcc") is None:
        pytest.skip("hipcc not available")
    out = tmp_path_factory.mktemp("isa")
    flags = [f for f in kbuild.FLAGS if f not in ("-shared", "-fPIC")]
    texts = {}
    for src in SOURCES:
        dst = str(out / (src + ".s"))
        subprocess.run([kbuild.HIPCC, *flags, "--cuda-device-only", "-S", "-o", dst,
                        os.path.join(kbuild.HERE, "csrc", src)], check=True,
                       stdout=subprocess.DEVNULL, stderr=subprocess.DEVNULL)
        texts[src] = open(dst).read().split("\n")
    return texts


@pytest.mark.parametrize("out,nt", [(1, 0), (1, 1), (0, 0)])
def test_every_operand_wavefront_waits_for_its_lds_loads(linear_asm, out, nt):
    """The four operand wavefronts load q, k and v straight into LDS; each has to
    wait for its own loads before the barrier that publishes them."""
    name = "la_prefillILb%dELb%dE" % (out, nt)
    body = next(b for n, b in kernels(linear_asm["linear_attention.hip"]).items() if name in n)
    found, checked = unawaited_lds_loads(body)
    assert checked >= 4 and not found, found


def test_inline_asm_does_not_break_live_scc(linear_asm):
    for src, lines in linear_asm.items():
        for i, line in enumerate(lines):
            if ";;#ASMSTART" not in line:
                continue
            j = next(j for j in range(i, len(lines)) if ";;#ASMEND" in lines[j])
            assert not any(SCC_WRITERS.match(x) or SCC_READERS.match(x) for x in lines[i + 1:j]), (src, i + 1)


def test_mfma_accumulators_keep_their_shape(linear_asm):
    found, checked = mfma_shape_changes(linear_asm["linear_attention.hip"])
    assert checked > 0 and not found, found[:3]


def test_no_spills_and_no_packed_fp32(linear_asm):
    for src, lines in linear_asm.items():
        for i, line in enumerate(lines):
            assert not re.match(r"^\s*(scratch_(load|store)|v_pk_(add|mul|fma)_f32)", line), (src, i + 1, line)


def test_uniform_loads_are_not_made_lane_by_lane(linear_asm):
    """A buffer descriptor that the compiler cannot see to be the same in all lanes is
    loaded through in a loop over its values (a readfirstlane, compares and a branch)."""
    lines = linear_asm["linear_attention.hip"]
    for i, line in enumerate(lines):
        if re.search(r"^\s*buffer_(load|store)", line):
            assert not any("s_and_saveexec" in x for x in lines[max(0, i - 2):i]) or \
                not any("v_readfirstlane" in x for x in lines[max(0, i - 10):i]), i + 1
