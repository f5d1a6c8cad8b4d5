"""GPU tests of how far the states and outputs of linear attention may be from the
exact ones, where a coarser arithmetic than the stated one would show: long
sequences with slow decays, decays without new tokens, few tokens alone.

The exact values are closed sums in 64 bits: S = sum over t of e^(decay behind t) k_t v_t^T."""
import math

import pytest
import torch

import kda_chunked_delta_amd as kda

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
D = 128


def tokens(T, H, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return [torch.randn(T, H, D, generator=gen, device=DEV, dtype=torch.bfloat16) for _ in range(3)]


def end_state(k, v, g):
    """The state after all tokens, from zero, with one log-decay per head."""
    T = k.shape[0]
    behind = torch.arange(T - 1, -1, -1, device=DEV).double()
    return torch.stack([(torch.exp(g[h].double() * behind)[:, None] * k[:, h].double()).t().contiguous()
                        @ v[:, h].double() for h in range(k.shape[1])])


# A decay per token and how far the state may be off as a whole, as a factor: the fp32
# sums round it without a preferred sign, 16384 elements of it, which leaves 3e-8; the
# weights of the tokens and the decay of a chunk are exponentials, off by 2^-23, of a
# log-decay that is rounded to 2^-24, each counting once whatever the length: 5e-7 in all.
# A state that decays by a few steps of its last bit per chunk (4e-8 a token: 11 to 21 of
# them) is rounded to whole ones, which favours one sign by at most 1/8 of a step in
# those: 2048 times 1e-9, of which a growing state remembers half.
SLOW = [(-4e-8, 2e-6), (-1e-6, 5e-7), (-1e-5, 5e-7), (-3e-5, 5e-7), (-3e-4, 5e-7)]


def slow_decays(plan_args, T=65536):
    q, k, v = tokens(T, len(SLOW), seed=1)
    g = torch.tensor([x for x, _ in SLOW], device=DEV)
    plan = kda.plan_linear_attention([0, T], len(SLOW), *plan_args, device=DEV)
    _, s = kda.linear_attention_prefill(q, k, v, g, cu_seqlens=[0, T], plan=plan, output_final_state=True)
    want = end_state(k, v, g)
    err = s[0].double() - want
    for h, (x, most) in enumerate(SLOW):
        norm = want[h].norm()
        off, gain = (err[h].norm() / norm).item(), ((err[h] * want[h]).sum() / norm.square()).item()
        print("  %8.0e a token: off %.2e, as a factor %+.2e" % (x, off, gain), flush=True)
        # seven roundings of each element a chunk, at most 2^-24 of it and 2^-24 / sqrt(3) in the
        # mean, over 2048 chunks of a state that grows with their root: 2.9e-6, and its factor
        assert off <= 4e-6 and abs(gain) <= most, x


def test_slow_decays_of_long_sequences():
    slow_decays((False,))


@pytest.mark.parametrize("seg", [0, 1, 8])
def test_slow_decays_of_segments(seg):
    """Up to 2048 of them: the merge rounds a state once per segment, the decay between two counts like a chunk's."""
    slow_decays((True, seg))


# The decay of a chunk of 32 tokens on both sides of 1/2, of 1 and of 2, and zero.
@pytest.mark.parametrize("of_chunk", [0.49, 0.4999, 0.5, 0.5001, 0.51, 0.75, 0.999, 1.0, 1.001, 1.5, 1.999, 2.0, 2.001,
                                      2.1, 1e-9, 0.0])
def test_decays_without_new_tokens(of_chunk):
    T = 32 * 12 + 7
    q, k, v = tokens(T, 2, seed=2)
    v.zero_()
    g = torch.full((2,), math.log(of_chunk) / 32 if of_chunk else -math.inf, device=DEV)
    s0 = torch.randn(1, 2, D, D, device=DEV)
    _, s = kda.linear_attention_prefill(q, k, v, g, initial_state=s0, output_final_state=True, use_intracard_cp=False)
    total = (g.double() * T)[None, :, None, None]
    want = torch.exp(total) * s0.double()
    # 13 chunks: an exponential (2^-23) and a rounding (2^-24) each; the log-decay is rounded to 2^-24 twice
    tol = 13 * 1.5 * 2.0 ** -23 + total.abs().max().item() * 2.0 ** -23 if of_chunk else 0.0
    off = (s.double() - want).abs()
    if of_chunk != 1e-9:  # whose twelfth power is zero in 32 bits
        assert (off <= tol * want.abs() + 1e-45).all()
    else:
        assert not s.any()


def test_a_decay_between_segments_below_the_smallest_fp32_number():
    """A state that has grown keeps a part of such a decay: e^80 of it, e^-96 and e^40 in a row, by segments."""
    T = 192
    q, k, v = tokens(3 * T, 1, seed=5)
    v[T:] = 0
    g = torch.empty(3 * T, 1, device=DEV)
    g[:T], g[T:2 * T], g[2 * T:] = 80 / T, -96 / T, 40 / T
    behind = g.double().flip(0).cumsum(0).flip(0) - g.double()
    want = (torch.exp(behind) * k[:, 0].double()).t().contiguous() @ v[:, 0].double()
    plan = kda.plan_linear_attention([0, 3 * T], 1, True, 6, device=DEV)
    _, s = kda.linear_attention_prefill(q, k, v, g, cu_seqlens=[0, 3 * T], plan=plan, output_final_state=True)
    # log-decays of 216 in all, rounded as such, as multiples of log2(e) and to sums, 2^-24 each
    assert (s[0, 0].double() - want).norm() <= 216 * 3 * 2.0 ** -24 * want.norm()


# ---------------------------------------------------------------------------
# segments whose early tokens come back
# ---------------------------------------------------------------------------
def growing(T=384):
    """Segments of 384 tokens, by chunks: a decay of e^-115 over the last four, growth of e^77 before and of e^38
    in what follows them. Only the tokens before the decay have values, so that all of the state passes it."""
    q, k, v = tokens(3 * T, 2, seed=3)
    g = torch.zeros(3 * T, 2, device=DEV)
    g[:256], g[256:384], g[384:512] = 0.3, -0.9, 0.3
    g[:, 1] *= 0.5
    v[256:] = 0
    return q, k, v, g


def test_growth_before_a_strong_decay_in_a_segment():
    q, k, v, g = growing()
    behind = g.double().flip(0).cumsum(0).flip(0) - g.double()
    want = torch.stack([(torch.exp(behind[:, h])[:, None] * k[:, h].double()).t().contiguous() @ v[:, h].double()
                        for h in range(2)])
    for mode, seg in ((False, 0), (True, 12), (True, 6)):
        plan = kda.plan_linear_attention([0, len(q)], 2, mode, seg, device=DEV)
        o, s = kda.linear_attention_prefill(q, k, v, g, cu_seqlens=[0, len(q)], plan=plan, output_final_state=True)
        off = ((s[0].double() - want).norm(dim=(1, 2)) / want.norm(dim=(1, 2))).tolist()
        print("  segments of %d chunks: off %.2e %.2e" % (seg, *off), flush=True)
        # log-decays of 230 in all, rounded as such (2^-24), as multiples of log2(e) (2^-24) and to sums (2^-24)
        assert max(off) <= 230 * 3 * 2.0 ** -24, (seg, off)


@pytest.mark.parametrize("seg", [0, 12])
def test_a_log_decay_that_is_nan_reaches_the_end_from_everywhere(seg):
    q, k, v = tokens(1200, 2, seed=4)
    g = torch.full((1200, 2), -2.0, device=DEV)  # a segment's end state is that of its last few chunks
    for at in (3, 500, 1199):
        x = g.clone()
        x[at, 1] = math.nan
        plan = kda.plan_linear_attention([0, 1200], 2, seg > 0, seg, device=DEV)
        _, s = kda.linear_attention_prefill(q, k, v, x, cu_seqlens=[0, 1200], plan=plan, output_final_state=True)
        assert torch.isfinite(s[0, 0]).all() and s[0, 1].isnan().all(), at


# ---------------------------------------------------------------------------
# what the computed operands keep
# ---------------------------------------------------------------------------
def halves(x, n):
    """The sum of x's first n bf16 parts, each the rounding of what the ones before leave."""
    total = torch.zeros_like(x)
    for _ in range(n):
        total = total + (x - total).bfloat16().to(x.dtype)
    return total


@pytest.mark.parametrize("T,seg", [(32, 0), (23, 0), (64, 1), (96, 1)])
def test_a_token_enters_a_state_with_all_its_bits(T, seg):
    """In the norm: the weights are exponentials (2^-23) of log-decays below 1 that are rounded (2^-23), times v (2^-24),
    in sums with six roundings a chunk, 2^-24 / sqrt(3) in the mean; the decay between chunks (2^-23) and its sum."""
    g = torch.tensor([-0.003, -0.01, -0.007, -0.0301], device=DEV)
    q, k, v = tokens(T, 4, seed=6)
    plan = kda.plan_linear_attention([0, T], 4, seg > 0, seg, device=DEV)
    _, s = kda.linear_attention_prefill(q, k, v, g, cu_seqlens=[0, T], plan=plan, output_final_state=True)
    want = end_state(k, v, g)
    tol = 7e-7
    off = ((s[0].double() - want).norm(dim=(1, 2)) / want.norm(dim=(1, 2))).max().item()
    # what two parts of the weighted v would leave, with everything else exact
    w = torch.exp(g.double()[None] * torch.arange(T - 1, -1, -1, device=DEV).double()[:, None])[..., None] * v.double()
    two = torch.stack([k[:, h].double().t().contiguous() @ halves(w, 2)[:, h] for h in range(4)])
    coarse = ((two - want).norm(dim=(1, 2)) / want.norm(dim=(1, 2))).min().item()
    print("  off %.2e, with two parts %.2e" % (off, coarse), flush=True)
    assert off <= tol and coarse > 2 * tol


@pytest.mark.parametrize("at", [0, 5, 15, 16, 20])
def test_a_product_of_q_and_k_reaches_an_output_with_more_than_eight_bits(at):
    """One key alone, so that an output row is one product times its v: a rounding of the product scales the row.
    Rounding the row's 128 outputs looks like a factor of at most 2^-8 / sqrt(3) times sqrt(3 / 128) in the mean."""
    T, H, scale = 32, 16, 0.7301
    q, k, v = tokens(T, H, seed=7)
    k[:at], k[at + 1:] = 0, 0
    o, _ = kda.linear_attention_prefill(q, k, v, torch.zeros(H, device=DEV), scale=scale)
    A = scale * (q.double() * k[at].double()).sum(-1)[at:]  # [tokens, H]
    want = A[..., None] * v[at].double()
    factor = lambda x: (((x - want) * want).sum(-1) / want.square().sum(-1)).square().mean().sqrt().item()
    off, coarse = factor(o[at:].double()), factor((halves(A, 1)[..., None] * v[at].double()).bfloat16().double())
    print("  off %.2e, with one part %.2e" % (off, coarse), flush=True)
    assert not o[:at].any()
    assert off <= 2.0 ** -8 / 128 ** 0.5 * 1.2 and coarse > 2 * 2.0 ** -8 / 128 ** 0.5


def test_slow_decays_of_long_generations():
    """A state is rounded once a token: 2^-24 / sqrt(3) in the mean over 4096 of them and a state that grows with
    their root, 1.6e-6, and with no preferred sign but where it decays by a few steps of its last bit (17 at -1e-6:
    1 / 8 of a step in those, half of 4096 times 7e-10)."""
    T = 4096
    decays = [(-1e-6, 2e-6), (-1e-5, 5e-7), (-3e-5, 5e-7), (-1e-4, 5e-7), (-1e-3, 5e-7)]
    q, k, v = tokens(T, len(decays), seed=8)
    g = torch.tensor([x for x, _ in decays], device=DEV)
    s = torch.zeros(1, len(decays), D, D, device=DEV)
    kda.linear_attention_decode(q[None], k[None], v[None], g, s)
    want = end_state(k, v, g)
    err = s[0].double() - want
    for h, (x, most) in enumerate(decays):
        norm = want[h].norm()
        off, gain = (err[h].norm() / norm).item(), ((err[h] * want[h]).sum() / norm.square()).item()
        print("  %8.0e a token: off %.2e, as a factor %+.2e" % (x, off, gain), flush=True)
        assert off <= 3e-6 and abs(gain) <= most, x
