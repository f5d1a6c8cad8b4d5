"""How kda_logits_process cuts a call into workgroups (csrc/logits_launch.h), as a
host program of its own (no GPU needed; needs hipcc)."""
import os
import shutil
import subprocess

import pytest

from kda_chunked_delta_amd import build as kbuild

MAIN = r"""
#include <cstdio>
#include "logits_launch.h"
int main() {
    int rows, vocab, max_tokens, n_bias, tokens, penalty;
    static float f;
    static int32_t t;
    while (scanf("%d %d %d %d %d %d", &rows, &vocab, &max_tokens, &n_bias, &tokens, &penalty) == 6) {
        kda::LogitsArgs a{};
        a.x.rows = rows;
        a.x.vocab = vocab;
        a.x.max_tokens = max_tokens;
        a.x.n_bias = n_bias;
        a.x.tokens = tokens ? &t : nullptr;
        a.x.presence = penalty ? &f : nullptr;
        kda::split_logits(&a);
        printf("%d %d %d %d %d\n", a.chunk, a.splits, a.lists, a.threads, a.lds);
    }
}
"""


@pytest.fixture(scope="module")
def split(tmp_path_factory):
    if not os.path.exists(kbuild.HIPCC) and shutil.which("hipcc") is None:
        pytest.skip("hipcc not available")
    out = tmp_path_factory.mktemp("split")
    src, exe = out / "main.hip", out / "main"
    src.write_text(MAIN)
    subprocess.run([kbuild.HIPCC, "--cuda-host-only", "-std=c++17", "-I" + os.path.join(kbuild.ROOT, "include"),
                    "-I" + os.path.join(kbuild.HERE, "csrc"), "-o", str(exe), str(src)], check=True,
                   stdout=subprocess.DEVNULL, stderr=subprocess.DEVNULL)

    def call(cases):
        text = "\n".join(" ".join(str(int(c.get(n, d))) for n, d in
                                  (("rows", 1), ("vocab", 1), ("max_tokens", 0), ("n_bias", 0), ("tokens", 0),
                                   ("penalty", 1))) for c in cases)
        lines = subprocess.run([str(exe)], input=text, check=True, capture_output=True, text=True).stdout.split("\n")
        names = ("chunk", "splits", "lists", "threads", "lds")
        return [dict(zip(names, map(int, line.split()))) for line in lines[:len(cases)]]

    return call


LISTS = [dict(), dict(n_bias=8192), dict(tokens=1, max_tokens=1), dict(tokens=1, max_tokens=4096),
         dict(tokens=1, max_tokens=4097, n_bias=1), dict(tokens=1, max_tokens=(1 << 14) - 1),
         dict(tokens=1, max_tokens=1 << 14), dict(tokens=1, max_tokens=(1 << 30) - 1)]
MOST = (1 << 31) - 1


@pytest.mark.parametrize("rows,vocab", [(1, 1), (3, 4097), (512, 8192), (511, 16384), (256, 131072), (1, MOST), (15, MOST),
                                        (1, MOST - 2047), (1, MOST - 2048), (1, MOST - 4096), (1, MOST - 8192),
                                        (1, MOST - 16384), ((1 << 23) - 1, 4096), ((1 << 22) - 1, 8192)])
def test_the_chunks_of_a_row_cover_it(split, rows, vocab):
    cases = [dict(rows=rows, vocab=vocab, **x) for x in LISTS]
    for case, a in zip(cases, split(cases)):
        assert a["chunk"] > 0 and a["chunk"] % 32 == 0 and a["splits"] > 0, (case, a)
        assert (a["splits"] - 1) * a["chunk"] < vocab <= a["splits"] * a["chunk"], (case, a)
        assert rows * a["splits"] * a["threads"] < 1 << 32, (case, a)
        assert 0 < a["lds"] <= 65536, (case, a)
        # many workgroups at the largest chunk are not cut finer
        assert rows * -(-vocab // 16384) < 512 or a["chunk"] >= 8192, (case, a)


@pytest.mark.parametrize("n_bias", [0, 1, 64])
@pytest.mark.parametrize("length", [1, 4096, 4097, 1 << 14, (1 << 30) - 1])
def test_a_history_without_penalties_takes_no_room(split, n_bias, length):
    """It is not looked at, so the call is cut as one without it."""
    sizes = dict(rows=256, vocab=131072, n_bias=n_bias)
    without, with_it = split([sizes, dict(sizes, tokens=1, max_tokens=length, penalty=0)])
    assert with_it == without
