"""Host-side tests (no GPU) of the size limits of the gated delta rule, the state
pool's pages and beam selection: HIP launches fewer than 2^32 threads, and what
would need more is refused by the checks of arguments."""
import ctypes
import os
import subprocess
import sys

import pytest

import kda_chunked_delta_amd as kda

OK, INVALID = 0, 1
AT = [(1 << 50) + (i << 42) for i in range(10)]  # compared only, 4 TiB apart


# threads of a workgroup: 512 per (unit, head), 768 per (segment, head) whose end state is formed, 8 x 512 per
# (segmented sequence, head)
@pytest.mark.parametrize("lengths,H,seg,fits", [
    ([1] * 65535, 128, 0, True), ([1] * 65536, 128, 0, False), ([1] * 63, 1 << 17, 0, True),
    ([1] * 64, 1 << 17, 0, False), ([32 * 43], 1 << 17, 1, True), ([32 * 44], 1 << 17, 1, False),
    ([64] * 7, 1 << 17, 1, True), ([64] * 8, 1 << 17, 1, False)])
def test_prefill_units(kda_lib, lengths, H, seg, fits):
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    make = lambda: kda.plan_gated_delta_host(cu, H, 256, seg > 0, seg)
    if fits:
        assert make().info()["n_units"] >= len(lengths)
    else:
        with pytest.raises(kda.KDAError, match="work units") as e:
            make()
        assert e.value.status == INVALID


@pytest.mark.parametrize("n,H,fits", [((1 << 24) - 1, 1, True), (1 << 24, 1, False), ((1 << 19) - 1, 32, True),
                                      (1 << 19, 32, False)])
def test_decode_sequences(kda_lib, n, H, fits):
    a = AT
    st = kda_lib.kda_gated_delta_decode_validate(n, 1, H, H, 128, 128, a[0], a[1], a[2], a[3], a[4], 1.0, a[5], 7, a[6],
                                                 a[7])
    assert st == (OK if fits else INVALID)


@pytest.mark.parametrize("page,beams,batch,fits", [(65536, 64, 65535, True), (65536, 64, 65536, False),
                                                   (16, 1, (1 << 24) - 1, True), (16, 1, 1 << 24, False),
                                                   (16400, 2, 1 << 22, False), (16384, 2, 1 << 22, True)])
def test_reordered_parts(kda_lib, page, beams, batch, fits):
    pool = kda.Pool(AT[0], 0, page, 1, 10)
    st = kda_lib.kda_beam_reorder_validate(ctypes.byref(pool), AT[1], AT[2], AT[3], batch, beams)
    assert st == (OK if fits else INVALID)


@pytest.mark.parametrize("B,W,V,n,fits", [((1 << 24) - 1, 1, 8, 1, True), (1 << 24, 1, 8, 1, False),
                                          ((1 << 18) - 1, 64, 64, 64, True), (1 << 18, 64, 64, 64, False),
                                          ((1 << 20) - 1, 1, 131072, 32, True), (1 << 20, 1, 131072, 32, False),
                                          ((1 << 18) - 1, 1, 131072, 33, True), (1 << 18, 1, 131072, 33, False)])
def test_selected_chunks(kda_lib, B, W, V, n, fits):
    """Chunks of 8192 logits, or of 2048 for more than 32 candidates."""
    a = AT
    need = kda_lib.kda_beam_select_workspace_bytes(B, W, V, n)
    st = kda_lib.kda_beam_select_validate(B, W, V, n, a[0], 1, V, a[1], None, -1, a[2], a[3], a[4], None, a[5], need)
    assert st == (OK if fits else INVALID)


OUT_OF_MEMORY = """
import ctypes, resource, sys
import kda_chunked_delta_amd as kda
kda.plan_gated_delta_host([0, 4096], 1, 256, True, 1)
size = lambda: int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
before = size()
resource.setrlimit(resource.RLIMIT_AS, (before + (200 << 20),) * 2)
cu, h = (ctypes.c_int32 * 2)(0, 1 << 28), ctypes.c_void_p()
st = kda.lib().kda_plan_gated_delta_host(256, cu, 1, 1, 128, 128, 1, 1, ctypes.byref(h))
print(st, bool(h), size() - before >> 20, kda.lib().kda_last_error().decode())
"""


def test_a_plan_that_runs_out_of_memory_gives_it_back(kda_lib):
    """Eight million segments of a chunk in 200 MiB: an error, and nothing kept."""
    r = subprocess.run([sys.executable, "-c", OUT_OF_MEMORY], capture_output=True, text=True, timeout=100,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    status, plan, kept, message = r.stdout.strip().split(" ", 3)
    assert int(status) == INVALID and plan == "False" and "memory" in message, (r.stdout, r.stderr)
    assert int(kept) < 32, r.stdout


@pytest.mark.parametrize("tokens", [(1 << 31) - 1, (1 << 31) - 31, (1 << 31) - 32])
@pytest.mark.parametrize("seg", [0, 1 << 22])
def test_plan_of_the_longest_prompt(kda_lib, tokens, seg):
    """Chunks whose end lies beyond 2^31 - 1 tokens."""
    p = kda.plan_gated_delta_host([0, tokens], 1, 256, seg > 0, seg)
    chunks = -(-tokens // 32)
    assert sum(u["n_chunks"] for u in p.units()) == chunks == p.info()["total_chunks"]
    assert p.info()["max_unit_chunks"] == max(u["n_chunks"] for u in p.units())
