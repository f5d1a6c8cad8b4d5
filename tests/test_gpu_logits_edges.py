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


def test_sizes_of_more_than_32_bits_are_refused():
    """An int32 would take them for small ones, and the call do a small part of its work."""
    W = 1 << 32
    x = torch.zeros(2, 100, dtype=torch.bfloat16, device=DEV)
    one = torch.ones(2, device=DEV)
    long = torch.empty(1, W + 5, dtype=torch.bfloat16, device=DEV)  # 8 GiB
    tall = torch.empty(W + 2, 1, dtype=torch.bfloat16, device=DEV)
    for bad in (long, tall):
        with pytest.raises(ValueError):
            kda.logits_process(bad)
    del long, tall
    t = torch.empty(1, W + 5, dtype=torch.int32, device=DEV)  # 16 GiB
    with pytest.raises(ValueError):
        kda.logits_process(x, tokens=t.expand(2, -1), presence=one)
