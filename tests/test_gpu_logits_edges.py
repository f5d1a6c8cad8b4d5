"""GPU tests of the processing of logits at the ends of its sizes."""
import pytest
import torch

import kda_chunked_delta_amd as kda

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("V", [(1 << 31) - 1, (1 << 31) - 8191])
def test_the_largest_vocabulary(V):
    x = torch.zeros(1, V, dtype=torch.bfloat16, device=DEV)  # 4 GiB
    t = torch.tensor([[5, V - 1, V // 2, V // 2]], dtype=torch.int32, device=DEV)
    one = torch.ones(1, device=DEV)
    kda.logits_process(x, tokens=t, frequency=one, out=x)
    assert x[0, t[0].long()].tolist() == [-1.0, -1.0, -2.0, -2.0]
    x[0, t[0].long()] = 0.0
    assert not x.any()
