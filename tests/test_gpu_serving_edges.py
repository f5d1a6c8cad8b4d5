"""GPU tests of what the gated delta rule, the state pool's pages and beam
selection state about their limits: the bound of the selection's log-sum-exp."""
import pytest
import torch

import kda_chunked_delta_amd as kda

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def say(*a):
    print(*a, flush=True)


# ---------------------------------------------------------------------------
# the selection's log-sum-exp
# ---------------------------------------------------------------------------
# One logit m in every `step` and equal ones y between, a few below it: whatever
# one term is off by, all are, and every chunk of the row has the same maximum,
# so nothing averages out. The score is chosen so that the first candidate's
# value is next to zero, where the fp32 result resolves it: what is left is the
# error of the log-sum-exp, stated as 2e-7 (its terms are off by 2^-23 for
# exp2's last bit and 2^-24 for one fp32 addition, 1.8e-7).
@pytest.mark.parametrize("dtype,m,y", [
    (torch.float32, 8.217265, 0.21694326), (torch.float32, 8.5000005, 0.4999996), (torch.float32, 9.1, 0.3),
    (torch.float32, 3.3, -0.0123), (torch.float32, 7.7, -0.30000004), (torch.float32, -0.7, -8.8999996),
    (torch.float32, -40.3, -48.7), (torch.float32, 47.9, 39.77), (torch.float32, 48.1, 40.2),
    (torch.float32, 60.3, 52.1), (torch.float32, -60.3, -68.7), (torch.float32, 300.1, 291.3),
    (torch.float32, 1e-3, -1e-3), (torch.bfloat16, 8.0, -4.8e-7), (torch.bfloat16, 9.0, 0.0021),
    (torch.bfloat16, 0.004, -8.0), (torch.float16, 8.0, -4.8e-7), (torch.float16, 8.6, 1.7e-4)])
@pytest.mark.parametrize("B,V,step", [(2, 5000, 2048), (2, 32000, 2048), (32, 131072, 8192)])
def test_log_sum_exp_of_equal_logits(dtype, m, y, B, V, step):
    say("case equal logits", dtype, m, y, B, V)
    x = torch.full((B, 2, V), y, dtype=torch.float32).to(dtype)
    x[..., ::step] = m
    k = -(-V // step)
    a, b = x[0, 0, 0].double(), x[0, 0, 1].double()
    log = torch.log(k + (V - k) * torch.exp(b - a))
    s = log.float().expand(B, 2).contiguous()
    score, parent, token, _ = kda.beam_select(x.to(DEV), s.to(DEV), n=3)
    want = (s[0, 0].double() - log).item()
    off = (score.cpu().double() - want).abs().max().item()
    say("  off by %.2e" % off)
    assert off <= 2e-7 + 2.0 ** -24 * abs(want)
    # equal candidates of equal beams: by beam, then by token
    assert parent.tolist() == [[0] * 3] * B and token.tolist() == [[0, step, 2 * step]] * B
