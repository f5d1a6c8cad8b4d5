"""Sizes that the C ABI's 32 bits do not hold are refused by the Python binding (no GPU needed)."""
import pytest
import torch

import kda_chunked_delta_amd as kda

W = 1 << 32  # an int32 argument would take W + 5 for 5


@pytest.mark.parametrize("kw", [dict(H=W + 1), dict(cu=[0, W + 5]), dict(cu=[0, 5, W + 9]), dict(n_cus=W + 256),
                                dict(seg=W + 4), dict(H=1 << 31), dict(cu=[-W, 5])])
def test_linear_attention_plans(kda_lib, kw):
    a = dict(dict(cu=[0, 5], H=1, n_cus=256, seg=0), **kw)
    with pytest.raises(ValueError, match="below 2\\^31"):
        kda.plan_linear_attention_host(a["cu"], a["H"], a["n_cus"], "auto", a["seg"])


def test_rows_of_lists_and_logits():
    long = torch.empty(1, W + 5, dtype=torch.int32, device="meta")
    for t in (long, long.expand(3, -1)):
        with pytest.raises(ValueError, match="below 2\\^31"):
            kda._rows("tokens", t, torch.int32, t.shape[:-1], -1)
