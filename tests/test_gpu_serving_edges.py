"""GPU tests of what the gated delta rule, the state pool's pages and beam
selection state about their limits: the bound of the selection's log-sum-exp,
the largest launches, the timing of a window with every kernel in it, how far a
value that is not finite reaches, and the order of candidates at -inf."""
import pytest
import torch

import kda_chunked_delta_amd as kda
from kda_inputs import draw, draw_decode

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


# ---------------------------------------------------------------------------
# the largest launches: just below 2^32 threads
# ---------------------------------------------------------------------------
def test_prefill_of_65535_one_token_prompts():
    """From a zero state, o = beta (q . k) v: one rounding, and the level of fp32 states."""
    N, H = 65535, 128
    say("case prefill, 65535 x 128 units")
    gen = torch.Generator(device=DEV).manual_seed(1)
    q = torch.randn(N, 1, 128, generator=gen, device=DEV).bfloat16()
    v = torch.empty(N, H, 128, dtype=torch.bfloat16, device=DEV).normal_(generator=gen)
    g, beta = torch.full((N, H), -0.5, device=DEV), torch.rand(N, H, generator=gen, device=DEV)
    o, _ = kda.gated_delta_prefill(q, q, v, g, beta, cu_seqlens_host=list(range(N + 1)), use_intracard_cp=False,
                                   scale=1 / 128)
    for i in (0, 1, 40000, N - 1):
        want = (q[i].double() ** 2).sum() / 128 * beta[i].double()[:, None] * v[i].double()
        assert ((o[i].double() - want).abs() <= (2.0 ** -8 + 1e-5) * want.abs()).all(), i


def test_decode_of_2_24_minus_1_sequences():
    """Only the first and the last have a slot; the outputs of the others are zero."""
    N = (1 << 24) - 1
    say("case decode, 2^24 - 1 sequences")
    gen = torch.Generator(device=DEV).manual_seed(2)
    x = torch.empty(N, 1, 128, dtype=torch.bfloat16, device=DEV).normal_(std=0.1, generator=gen)
    g, beta = torch.full((N, 1), -0.1, device=DEV), torch.full((N, 1), 0.5, device=DEV)
    slots = torch.full((N,), -1, dtype=torch.int32, device=DEV)
    slots[0], slots[-1] = 1, 0
    pool = torch.randn(2, 1, 128, 128, generator=gen, device=DEV)
    state = pool.flip(0).contiguous()
    o = kda.gated_delta_decode(x, x, x, g, beta, pool, slots=slots)
    two = [t[[0, N - 1]].contiguous() for t in (x, x, x, g, beta)]
    want = kda.gated_delta_decode(*two, state)
    assert torch.equal(o[[0, N - 1]], want) and torch.equal(pool, state.flip(0))
    o[0] = o[-1] = 0.0
    assert not o.any()


def test_selection_and_reordering_of_2_24_minus_1_rows():
    B, V = (1 << 24) - 1, 8
    say("case selection, 2^24 - 1 rows")
    x = torch.zeros(B, 1, V, dtype=torch.bfloat16, device=DEV)
    best = torch.arange(B, device=DEV) * 7 % V
    x.view(B, V).scatter_(1, best[:, None], 1.0)
    _, parents, tokens, _ = kda.beam_select(x, torch.zeros(B, 1, device=DEV), n=1)
    assert torch.equal(tokens[:, 0], best.int()) and not parents.any()
    say("case reordering, 2^24 - 2 beams")
    B //= 2
    pool = torch.arange(2 * B * 4, dtype=torch.int32, device=DEV).view(2 * B, 4)
    slots = torch.arange(2 * B, dtype=torch.int32, device=DEV).view(B, 2)
    new = kda.beam_reorder(pool, slots, torch.ones_like(slots))  # both beams continue the second
    assert torch.equal(new, slots.flip(1))
    odd = torch.arange(1, 2 * B, 2, device=DEV)
    want = (odd[:, None] * 4 + torch.arange(4, device=DEV)).int()
    assert torch.equal(pool.view(B, 2, 4), want[:, None].expand(B, 2, 4))


def test_copy_of_large_pages_with_many_pairs():
    """1024 pairs take parts of 128 bytes, more of them than one launch has workgroups."""
    say("case copy, 520 MiB pages")
    pool = torch.randint(0, 1 << 30, (3, 130 << 20), dtype=torch.int32, device=DEV,
                         generator=torch.Generator(device=DEV).manual_seed(4))
    old = pool.clone()
    src, dst = torch.full((2, 1024), -1, dtype=torch.int32, device=DEV).unbind(0)
    src[5], dst[5], src[1000], dst[1000] = 0, 2, 2, 0
    kda.pool_copy(pool, src, dst)
    assert torch.equal(pool, old[[2, 1, 0]])
    # the same with the pages' bytes spread over layers
    layers = old.view(3, 13, 10 << 20).transpose(0, 1).contiguous()
    want = layers[:, [2, 1, 0]]
    kda.pool_copy(layers, src, dst, page_dim=1)
    assert torch.equal(layers, want)


# ---------------------------------------------------------------------------
# per-kernel timing
# ---------------------------------------------------------------------------
def test_timing_lists_every_kernel_of_a_serving_window():
    """A server's window runs more than twenty kernels by name; none is dropped."""
    say("case timing")
    H, d = 2, draw([700], 2, seed=1, device=DEV)
    cu, xs = d["cu_seqlens_host"], [d[x] for x in ("q", "k", "v", "g", "beta")]
    one = draw_decode(1, H, seed=2, device=DEV)
    tok = [one[x] for x in ("q", "k", "v", "g", "beta")]
    pool, used = torch.zeros(6, H, 128, 128, device=DEV), torch.tensor([True] * 3 + [False] * 3, device=DEV)
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)
    state = d["initial_state"].clone()
    plans = [kda.plan(cu, H, device=DEV), kda.plan_segments(cu, H, 4, device=DEV), kda.plan_split(cu, H, [20], 4, device=DEV),
             kda.plan_warm_cp(cu, H, 8, 2, device=DEV)]
    gated = kda.plan_gated_delta(cu, H, True, 4, device=DEV)
    ctx = kda.context(DEV)
    ctx.set_timing(True)
    try:
        ctx.timing()
        for p in plans:
            kda.prefill(*xs[:4], xs[4].bfloat16(), cu_seqlens_host=cu, plan=p, output_final_state=True)
        kda.decode(*tok, state)
        kda.gated_delta_prefill(*xs[:3], xs[3][..., 0].contiguous(), xs[4], cu_seqlens_host=cu, plan=gated)
        kda.gated_delta_decode(*tok[:3], tok[3][..., 0].contiguous(), tok[4], state)
        kda.beam_select(torch.zeros(1, 2, 50, device=DEV), torch.zeros(1, 2, device=DEV))
        kda.beam_reorder(pool, i(0, 1).view(1, 2), i(1, 1).view(1, 2))
        kda.pool_copy(pool, i(0), i(1))
        kda.pool_fork(pool, used, i(0))
        kda.pool_free(used, i(1))
        kda.pool_compact(pool, used)
        t = ctx.timing()
    finally:
        ctx.set_timing(False)
    want = ["decode", "gated_delta_segments", "gated_delta_merge", "gated_delta", "gated_delta_decode", "beam_rows",
            "beam_pick", "beam_reorder", "pool_copy", "pool_fork_plan", "pool_move", "pool_free", "pool_compact_plan"]
    assert len(t) > 20 and not [n for n in want if n not in t], sorted(t)
    assert t["pool_move"][1] == 2 and all(ms > 0 and n > 0 for ms, n in t.values())


# ---------------------------------------------------------------------------
# values that are not finite
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("seg", [0, 1])
def test_prefill_with_a_value_that_is_not_finite(value, seg):
    """One in v reaches its own value column of its head from its chunk of 32 on;
    one in k its head from there on. Every other result keeps its bits."""
    say("case not finite", value, seg)
    d = draw([100, 70], 3, seed=11, device=DEV)
    xs = [d[x] for x in ("q", "k", "v", "g", "beta")]
    xs[3] = xs[3][..., 0].contiguous()
    plan = kda.plan_gated_delta(d["cu_seqlens_host"], 3, seg > 0, seg, device=DEV)
    run = lambda: kda.gated_delta_prefill(*xs, cu_seqlens_host=d["cu_seqlens_host"], plan=plan,
                                          initial_state=d["initial_state"], output_final_state=True)
    o, s = run()
    for at, column in ((2, 7), (1, None)):
        old = xs[at].clone()
        xs[at][45, 1, 7] = value
        o2, s2 = run()
        xs[at].copy_(old)
        hit_o, hit_s = torch.zeros_like(o, dtype=torch.bool), torch.zeros_like(s, dtype=torch.bool)
        hit_o[32:100, 1, slice(None) if column is None else slice(column, column + 1)] = True
        hit_s[0, 1, :, slice(None) if column is None else slice(column, column + 1)] = True
        assert torch.equal(o2[~hit_o], o[~hit_o]) and torch.equal(s2[~hit_s], s[~hit_s])
        tail = o2[45:100, 1] if column is None else o2[45:100, 1, column]
        assert not torch.isfinite(tail).any() and not torch.isfinite(s2[hit_s]).any()
        again, s3 = run()  # nothing of it is left behind
        assert torch.equal(again, o) and torch.equal(s3, s)


@pytest.mark.parametrize("V", [40, 9000, 300000])
def test_order_of_candidates_at_minus_infinity(V):
    """A beam at score -inf gives its tokens in order; a finite one, with logits
    at +inf that share the row, the others by logit."""
    say("case -inf", V)
    gen = torch.Generator(device=DEV).manual_seed(V)
    x = torch.randperm(V, generator=gen, device=DEV).float().sub(V // 2).view(1, 1, V).repeat(2, 2, 1)
    x[1, :, [30, 11]] = float("inf")
    score = torch.tensor([[-float("inf"), -float("inf")], [-1.0, -float("inf")]], device=DEV)
    s, parents, tokens, _ = kda.beam_select(x, score, n=6)
    assert not parents.any()
    assert tokens[0].tolist() == list(range(6)) and torch.isneginf(s[0]).all()
    rest = x[1, 0].clone()
    rest[[30, 11]] = -float("inf")
    assert tokens[1].tolist() == [11, 30] + rest.argsort(descending=True)[:4].tolist()
    want = torch.tensor(-1.0 - 0.6931471805599453, dtype=torch.float64)
    assert ((s[1, :2].cpu().double() - want).abs() <= 2e-7 + 2.0 ** -24 * want.abs()).all()
    assert torch.isneginf(s[1, 2:]).all()
