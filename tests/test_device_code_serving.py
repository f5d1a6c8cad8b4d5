"""Checks of the compiled gfx950 device code of the gated delta rule, the state
pool's pages and beam selection (no GPU needed; needs hipcc): the properties
that test_device_code.py checks of the KDA kernels, and the waits for
direct-to-LDS loads in the gated delta prefill."""
import os
import re
import shutil
import subprocess

import pytest

from kda_chunked_delta_amd import build as kbuild
from test_device_code import SCC_READERS, SCC_WRITERS, mfma_shape_changes

SOURCES = ("gated_delta.hip", "state_pool.hip", "beam_select.hip")


@pytest.fixture(scope="module")
def serving_asm(tmp_path_factory):
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


def kernels(lines):
    """{symbol: lines} of the functions."""
    out, name = {}, None
    for line in lines:
        m = re.match(r"^(_ZN\w+):", line)
        if m:
            name = m.group(1)
            out[name] = []
        elif line.startswith(".Lfunc_end"):
            name = None
        if name:
            out[name].append(line)
    return out


def unawaited_lds_loads(lines):
    """Barriers that a direct-to-LDS load may reach without a wait in the source:
    going down the text, a load that is followed by an inline-asm barrier with no
    inline-asm vmcnt wait between. Also the number of barriers behind such loads."""
    found, checked, pending, inline = [], 0, None, False
    for i, line in enumerate(lines):
        if ";;#ASMSTART" in line:
            inline = True
        elif ";;#ASMEND" in line:
            inline = False
        elif re.search(r"^\s*buffer_load\w*\s.*\blds\b", line):
            pending = (i, False)
        elif inline and "vmcnt(" in line and pending:
            pending = (pending[0], True)
        elif "s_barrier" in line and pending:
            checked += 1
            if not pending[1]:
                found.append((i + 1, pending[0] + 1))
            pending = None
    return found, checked


@pytest.mark.parametrize("out", [1, 0])
def test_every_operand_wavefront_waits_for_its_lds_loads(serving_asm, out):
    """The four operand wavefronts load q, k and v straight into LDS, one
    interval before the chunk's first use; each has to wait for the last
    interval's loads itself before the barrier that publishes them. (One that
    leaves this to the compiler's wait for its later register loads depends on
    those not being scheduled first.)"""
    body = next(b for n, b in kernels(serving_asm["gated_delta.hip"]).items() if "gd_prefillILb%dE" % out in n)
    found, checked = unawaited_lds_loads(body)
    assert checked >= 4 and not found, found


def test_wait_check_catches_a_missing_wait():
    text = ["buffer_load_dwordx4 v1, s[0:3], 0 offen lds", ";;#ASMSTART", "s_waitcnt vmcnt(6)", ";;#ASMEND", "s_barrier",
            "buffer_load_dwordx4 v1, s[0:3], 0 offen lds", "s_waitcnt vmcnt(6)", "s_barrier", "s_barrier"]
    assert unawaited_lds_loads(text) == ([(8, 6)], 2)


def test_inline_asm_does_not_break_live_scc(serving_asm):
    for src, lines in serving_asm.items():
        for i, line in enumerate(lines):
            if ";;#ASMSTART" not in line:
                continue
            j = next(j for j in range(i, len(lines)) if ";;#ASMEND" in lines[j])
            assert not any(SCC_WRITERS.match(x) or SCC_READERS.match(x) for x in lines[i + 1:j]), (src, i + 1)


def test_mfma_accumulators_keep_their_shape(serving_asm):
    found, checked = mfma_shape_changes(serving_asm["gated_delta.hip"])
    assert checked > 0 and not found, found[:3]


def test_no_spills_and_no_packed_fp32(serving_asm):
    for src, lines in serving_asm.items():
        for i, line in enumerate(lines):
            assert not re.match(r"^\s*(scratch_(load|store)|v_pk_(add|mul|fma)_f32)", line), (src, i + 1, line)
