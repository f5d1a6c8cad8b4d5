"""GPU parity of the gated delta rule (one log-decay per token and head) with
the per-token recurrence in 64 bits: chunked prefill, segmented prefill, and
decode of one or several tokens.

Tolerances, relative to the norm of the exact result. fp32 states: the state
and every computed operand go into products as hi + lo bf16 pairs (2^-18 of
their value, at most), three such operands meet on the way of one token into
the state, and steps add up at random over the tokens a state remembers: 1e-5
bounds 2.6 * 2^-18. Decode is fp32 throughout: 128-term sums, 2e-6. bf16
results add one rounding, at most 2^-8 of each value."""
import math

import pytest
import torch

import kda_chunked_delta_amd as kda
from kda_inputs import draw

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
D = 128
STATE_TOL, DECODE_TOL, HALF = 1e-5, 2e-6, 2.0 ** -8


def say(*a):
    print(*a, flush=True)


def make(lengths, H, seed, qk_heads=None, state_std=0.1, g_scale=1.0, g_mul=1.0, beta=torch.float32):
    d = draw(lengths, H, seed=seed, state_std=state_std, g_scale=g_scale, device=DEV, qk_heads=qk_heads)
    d["g"] = (g_mul * d["g"][:, :, 0]).contiguous()
    d["beta"] = d["beta"].to(beta)
    return d


def recurrence(q, k, v, g, beta, cu, s0, scale=1.0):
    """fp64, token by token (on the device: elementwise products and sums)."""
    rep = v.shape[1] // k.shape[1]
    q, k = (x.double().repeat_interleave(rep, 1) for x in (q, k))
    v, g, beta = v.double(), g.double(), beta.double()
    H = v.shape[1]
    out = torch.zeros(v.shape, dtype=torch.float64, device=v.device)
    S = torch.zeros(len(cu) - 1, H, D, D, dtype=torch.float64, device=v.device)
    if s0 is not None:
        S.copy_(s0)
    for i in range(len(cu) - 1):
        s = S[i]
        for t in range(cu[i], cu[i + 1]):
            s = s * torch.exp(g[t])[:, None, None]
            e = v[t] - (s * k[t][:, :, None]).sum(1)
            s = s + (beta[t][:, None] * k[t])[:, :, None] * e[:, None, :]
            out[t] = scale * (s * q[t][:, :, None]).sum(1)
        S[i] = s
    return out, S


def close(name, got, want, tol):
    g, w = got.double(), want.double()
    assert torch.isfinite(g).all(), name
    err, norm = (g - w).norm().item(), w.norm().item()
    say("  %-8s rel %.2e (tolerance %.2e)" % (name, err / norm if norm else err, tol))
    assert err <= tol * norm, (name, err, norm)
    if got.dtype == torch.bfloat16:  # element by element: one rounding, and the fp32-level error
        rms = norm / math.sqrt(max(1, w.numel()))
        assert ((g - w).abs() <= HALF * w.abs() + 40 * STATE_TOL * (rms + w.abs())).all(), name


def run(d, mode="auto", state=None, scale=1.0, **kw):
    s0 = d["initial_state"]
    if state is not None and s0 is not None:
        s0 = s0.to(state)
    o, s = kda.gated_delta_prefill(d["q"], d["k"], d["v"], d["g"], d["beta"], cu_seqlens=d["cu_seqlens"],
                                   cu_seqlens_host=d["cu_seqlens_host"], initial_state=s0, output_final_state=True,
                                   use_intracard_cp=mode, scale=scale, state_dtype=state, **kw)
    torch.cuda.synchronize()
    return o, s


def check(d, scale=1.0, state=torch.float32, **kw):
    s0 = d["initial_state"]
    o_ref, s_ref = recurrence(d["q"], d["k"], d["v"], d["g"], d["beta"], d["cu_seqlens_host"],
                              None if s0 is None else s0.to(state), scale)
    o, s = run(d, state=state, scale=scale, **kw)
    close("out", o, o_ref, STATE_TOL + HALF / 2)
    close("state", s, s_ref, STATE_TOL + (HALF / 2 if state == torch.bfloat16 else 0))


@pytest.mark.parametrize("lengths", [[1], [2], [15], [16], [17], [31], [32], [33], [64], [95],
                                     [0, 5, 0, 31, 48, 0], [3, 100, 257]])
def test_prefill_lengths(lengths):
    say("case lengths", lengths)
    check(make(lengths, 3, seed=sum(lengths) + 1), mode=False)


@pytest.mark.parametrize("H,Hk", [(1, 1), (5, 5), (12, 4), (6, 1), (32, 16)])
@pytest.mark.parametrize("beta", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("state", [torch.float32, torch.bfloat16])
def test_prefill_heads_and_types(H, Hk, beta, state):
    say("case H %d Hk %d beta %s state %s" % (H, Hk, beta, state))
    check(make([70, 33], H, seed=H + Hk, qk_heads=Hk, beta=beta), scale=0.7, state=state, mode=False)


# slow decay (a long memory), the plain one, and decays whose products leave fp32's range inside a chunk
@pytest.mark.parametrize("g_mul", [0.0, 0.001, 0.05, 1.0, 8.0, 60.0])
def test_prefill_decay_range(g_mul):
    say("case g x", g_mul)
    check(make([300, 77], 4, seed=5, g_mul=g_mul, state_std=None if g_mul == 1.0 else 0.1), mode=False)


def test_prefill_forgets_at_minus_infinity():
    """g = -inf forgets everything before its token, exactly."""
    d = make([90], 2, seed=8)
    d["g"][37] = float("-inf")
    check(d, mode=False)
    o, s = run(d, mode=False)
    d["initial_state"] = 50.0 + d["initial_state"]
    o2, s2 = run(d, mode=False)
    assert torch.equal(o[37:], o2[37:]) and torch.equal(s, s2) and not torch.equal(o[:37], o2[:37])


def test_prefill_repeated_keys_and_unit_beta():
    """beta = 1 and one key for all tokens: every step replaces the value of that key."""
    d = make([100], 2, seed=9)
    d["k"][:] = d["k"][:1]
    d["beta"][:] = 1.0
    check(d, mode=False)


def test_prefill_zero_tokens_keeps_states():
    d = make([0, 0], 3, seed=4)
    o, s = run(d, mode=False)
    assert o.shape == (0, 3, D) and torch.equal(s, d["initial_state"])
    d["initial_state"] = None
    assert torch.count_nonzero(run(d, mode=False)[1]) == 0


@pytest.mark.parametrize("lengths,H,seg", [([700], 2, 4), ([64], 1, 1), ([65], 3, 1), ([1000, 40, 0, 333], 2, 3),
                                           ([1500], 1, 7)])
@pytest.mark.parametrize("g_mul", [0.002, 1.0])
def test_segmented_prefill(lengths, H, seg, g_mul):
    say("case segments of %d chunks, lengths %s, g x %g" % (seg, lengths, g_mul))
    d = make(lengths, H, seed=sum(lengths), g_mul=g_mul)
    plan = kda.plan_gated_delta(d["cu_seqlens_host"], H, True, seg, device=DEV)
    assert plan.info()["uses_cp"] == 1
    check(d, plan=plan)
    check(d, plan=plan, state=torch.bfloat16)


def test_segmented_prefill_in_place_and_auto():
    """final_state = initial_state with segments; AUTO segments a long few-head prompt."""
    d = make([9000], 2, seed=3, g_mul=0.01)
    assert kda.plan_gated_delta(d["cu_seqlens_host"], 2, "auto", device=DEV).info()["uses_cp"] == 1
    o, s = run(d)
    state = d["initial_state"].clone()
    o2, s2 = kda.gated_delta_prefill(d["q"], d["k"], d["v"], d["g"], d["beta"], initial_state=state,
                                     final_state=state)
    torch.cuda.synchronize()
    assert s2 is state and torch.equal(o, o2) and torch.equal(s, s2)
    o_ref, s_ref = recurrence(d["q"], d["k"], d["v"], d["g"], d["beta"], [0, 9000], d["initial_state"])
    close("out", o, o_ref, STATE_TOL + HALF / 2)
    close("state", s, s_ref, STATE_TOL)


def test_prefill_equals_kda_prefill_with_the_decay_on_every_channel():
    d = make([200, 61], 4, seed=12)
    o, s = run(d, mode=False)
    g = d["g"][:, :, None].expand(-1, -1, D).contiguous()
    o2, s2 = kda.prefill(d["q"], d["k"], d["v"], g, d["beta"], cu_seqlens_host=d["cu_seqlens_host"],
                         initial_state=d["initial_state"], output_final_state=True)
    assert torch.allclose(o.float(), o2.float(), atol=1e-2, rtol=1e-2)
    assert torch.allclose(s, s2, atol=1e-2, rtol=1e-2)


def test_prefill_carry_and_repeat_bitwise():
    """A prompt in two calls, cut at a chunk border, gives the bits of one call; so does a repetition."""
    d = make([128 + 51], 3, seed=21, g_mul=0.1)
    o, s = run(d, mode=False)
    o2, s2 = run(d, mode=False)
    assert torch.equal(o, o2) and torch.equal(s, s2)
    part = lambda a, b: [x[a:b].contiguous() for x in (d["q"], d["k"], d["v"], d["g"], d["beta"])]
    oa, sa = kda.gated_delta_prefill(*part(0, 128), initial_state=d["initial_state"], output_final_state=True,
                                     use_intracard_cp=False)
    ob, sb = kda.gated_delta_prefill(*part(128, 179), initial_state=sa, output_final_state=True,
                                     use_intracard_cp=False)
    assert torch.equal(torch.cat([oa, ob]), o) and torch.equal(sb, s)


def test_prefill_4d_batch():
    d = make([40] * 3, 2, seed=6)
    o, s = run(d, mode=False)
    four = lambda x: x.view(3, 40, *x.shape[1:])
    o4, s4 = kda.gated_delta_prefill(*map(four, (d["q"], d["k"], d["v"], d["g"], d["beta"])),
                                     initial_state=d["initial_state"], output_final_state=True,
                                     use_intracard_cp=False)
    assert torch.equal(o4.view_as(o), o) and torch.equal(s4, s)


# ---------------------------------------------------------------------------
# decode
# ---------------------------------------------------------------------------
def decode_case(N, T, H, Hk, seed):
    d = make([T] * N, H, seed=seed, qk_heads=Hk)
    for x in ("q", "k", "v", "g", "beta"):
        d[x] = d[x].view(N, T, *d[x].shape[1:])
    return d


@pytest.mark.parametrize("N,T,H,Hk", [(1, 1, 1, 1), (3, 1, 5, 5), (7, 2, 12, 4), (64, 1, 32, 32), (5, 9, 6, 1),
                                      (2, 40, 3, 3), (80, 1, 32, 16)])
def test_decode(N, T, H, Hk):
    say("case decode", N, T, H, Hk)
    d = decode_case(N, T, H, Hk, seed=N + 10 * T + H)
    flat = [d[x].reshape(N * T, *d[x].shape[2:]) for x in ("q", "k", "v", "g", "beta")]
    o_ref, s_ref = recurrence(*flat, [i * T for i in range(N + 1)], d["initial_state"], 0.8)
    state = d["initial_state"].clone()
    args = [d[x] for x in ("q", "k", "v", "g", "beta")]
    if T == 1 and N % 2:
        args = [x.squeeze(1) for x in args]
    o = kda.gated_delta_decode(*args, state, scale=0.8)
    assert o.shape == args[2].shape
    close("out", o.reshape(o_ref.shape), o_ref, DECODE_TOL + HALF / 2)
    close("state", state, s_ref, DECODE_TOL)


def test_decode_tokens_at_once_are_the_bits_of_one_by_one():
    d = decode_case(6, 5, 4, 2, seed=2)
    a, b = d["initial_state"].clone(), d["initial_state"].clone()
    args = [d[x] for x in ("q", "k", "v", "g", "beta")]
    o = kda.gated_delta_decode(*args, a)
    for t in range(5):
        o1 = kda.gated_delta_decode(*[x[:, t].contiguous() for x in args], b)
        assert torch.equal(o1, o[:, t])
    assert torch.equal(a, b)


def test_decode_slots_skip_and_leave_others():
    N, H, P = 6, 4, 9
    d = decode_case(N, 2, H, H, seed=61)
    pool = torch.randn(P, H, D, D, device=DEV)
    before = pool.clone()
    slots = torch.tensor([7, 2, -1, 0, 9, 4], dtype=torch.int32, device=DEV)
    args = [d[x] for x in ("q", "k", "v", "g", "beta")]
    o = kda.gated_delta_decode(*args, pool, slots=slots)
    live = [0, 1, 3, 5]
    state = before[slots[live].long()].contiguous()
    o2 = kda.gated_delta_decode(*[x[live].contiguous() for x in args], state)
    assert torch.equal(o[live], o2) and torch.equal(pool[slots[live].long()], state)
    assert torch.count_nonzero(o[[2, 4]]) == 0
    rest = [1, 3, 5, 6, 8]
    assert torch.equal(pool[rest], before[rest])


def test_decode_empty():
    d = decode_case(2, 1, 3, 3, seed=1)
    s = d["initial_state"].clone()
    args = [d[x][:0] for x in ("q", "k", "v", "g", "beta")]
    assert kda.gated_delta_decode(*args, s[:0]).shape == (0, 1, 3, D)
    args = [d[x][:, :0].contiguous() for x in ("q", "k", "v", "g", "beta")]
    assert kda.gated_delta_decode(*args, s).shape == (2, 0, 3, D) and torch.equal(s, d["initial_state"])


def test_decode_continues_prefill():
    d = make([20, 1, 75], 4, seed=33, qk_heads=2)
    cu = d["cu_seqlens_host"]
    last = torch.tensor([c - 1 for c in cu[1:]], device=DEV)
    head = torch.tensor([t for i in range(3) for t in range(cu[i], cu[i + 1] - 1)], device=DEV)
    xs = [d[x] for x in ("q", "k", "v", "g", "beta")]
    _, s = kda.gated_delta_prefill(*[x[head] for x in xs], cu_seqlens=[0, 19, 19, 93],
                                   initial_state=d["initial_state"], output_final_state=True)
    o = kda.gated_delta_decode(*[x[last] for x in xs], s)
    o_ref, s_ref = recurrence(*xs, cu, d["initial_state"])
    close("out", o, o_ref[last], STATE_TOL + HALF / 2)
    close("state", s, s_ref, STATE_TOL)


# ---------------------------------------------------------------------------
# streams and graphs
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("seg", [0, 4])
def test_graph_replay_on_another_stream(seg):
    """Prefill and decode captured together, replayed between eager work, each replay against the eager result."""
    d = make([400, 33], 2, seed=14, g_mul=0.05)
    plan = kda.plan_gated_delta(d["cu_seqlens_host"], 2, seg > 0, seg, device=DEV)
    plan.cu_device()
    one = decode_case(2, 1, 2, 2, seed=15)
    tok = [one[x].squeeze(1) for x in ("q", "k", "v", "g", "beta")]

    def step(state):
        o, s = kda.gated_delta_prefill(d["q"], d["k"], d["v"], d["g"], d["beta"], plan=plan,
                                       cu_seqlens_host=d["cu_seqlens_host"], initial_state=state, final_state=state)
        return o, kda.gated_delta_decode(*tok, s)

    eager = d["initial_state"].clone()
    state = d["initial_state"].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            o, o1 = step(state)
    torch.cuda.synchronize()
    for _ in range(3):
        want = step(eager)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(o1, want[1]) and torch.equal(state, eager)


def test_capture_refuses_what_would_break_it():
    """Without a plan, with device cu_seqlens alone, or with a table that is not on the device yet."""
    d = make([70, 41], 2, seed=77)
    xs = [d[x] for x in ("q", "k", "v", "g", "beta")]
    plan = kda.plan_gated_delta([0, 70, 111], 2, device=DEV)
    cu = torch.tensor([0, 70, 111], dtype=torch.int32, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for kw in (dict(cu_seqlens=[0, 70, 111]), dict(cu_seqlens=cu), dict(cu_seqlens=[0, 70, 111], plan=plan)):
            with pytest.raises(ValueError, match="capture"):
                kda.gated_delta_prefill(*xs, **kw)
        o, _ = kda.gated_delta_prefill(*xs, cu_seqlens=cu, cu_seqlens_host=[0, 70, 111], plan=plan)
    want, _ = kda.gated_delta_prefill(*xs, cu_seqlens=cu)
    for _ in range(3):
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want)


def test_two_streams_at_once():
    ds = [make([600], 2, seed=s, g_mul=0.05) for s in (1, 2)]
    plan = kda.plan_gated_delta([0, 600], 2, True, 4, device=DEV)
    want = [run(d, plan=plan) for d in ds]
    streams = [torch.cuda.Stream() for _ in ds]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for d, s in zip(ds, streams):
            with torch.cuda.stream(s):
                got.append(kda.gated_delta_prefill(d["q"], d["k"], d["v"], d["g"], d["beta"], plan=plan,
                                                   initial_state=d["initial_state"], output_final_state=True))
    torch.cuda.synchronize()
    for i, (o, s) in enumerate(got):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(s, want[i % 2][1])


# ---------------------------------------------------------------------------
# offsets beyond 32 bits
# ---------------------------------------------------------------------------
def test_decode_of_a_slot_beyond_4_gib():
    """A pool of 8.4 GiB: the slots behind 2^31 elements give the bits of a small pool."""
    H, P = 32, 4200
    say("case decode, slots beyond 2^31 elements")
    d = decode_case(3, 2, H, H, seed=71)
    args = [d[x] for x in ("q", "k", "v", "g", "beta")]
    pool = torch.zeros(P, H, D, D, device=DEV)
    slots = torch.tensor([P - 1, 4097, 2049], dtype=torch.int32, device=DEV)
    pool[slots.long()] = d["initial_state"]
    state = d["initial_state"].clone()
    o = kda.gated_delta_decode(*args, pool, slots=slots)
    want = kda.gated_delta_decode(*args, state)
    assert torch.equal(o, want) and torch.equal(pool[slots.long()], state)
    pool[slots.long()] = 0.0
    assert torch.count_nonzero(pool) == 0


def test_prefill_tokens_beyond_4_gib():
    """262250 tokens of 64 heads (4.3 GB of v): the prompts behind the long one give
    the bits of a batch of their own. Segmented outputs are off the unsegmented
    ones by a rounding each, half a bf16 step (2^-8 of the value), and the
    states' tolerance."""
    H, Hk, lengths = 64, 1, [262000, 100, 33, 117]
    say("case prefill beyond 4 GiB")
    cu = [sum(lengths[:i]) for i in range(len(lengths) + 1)]
    gen = torch.Generator(device=DEV).manual_seed(5)
    q, k = (torch.nn.functional.normalize(torch.randn(cu[-1], Hk, D, generator=gen, device=DEV), dim=-1).bfloat16()
            for _ in range(2))
    v = torch.empty(cu[-1], H, D, dtype=torch.bfloat16, device=DEV).normal_(generator=gen)
    g = -0.2 * torch.rand(cu[-1], H, generator=gen, device=DEV)
    beta = torch.rand(cu[-1], H, generator=gen, device=DEV)
    tail = [x[cu[1]:].contiguous() for x in (q, k, v, g, beta)]
    want, sw = kda.gated_delta_prefill(*tail, cu_seqlens=[c - cu[1] for c in cu[1:]], output_final_state=True,
                                       use_intracard_cp=False)
    for cp in (False, True):
        o, s = kda.gated_delta_prefill(q, k, v, g, beta, cu_seqlens=cu, output_final_state=True,
                                       plan=kda.plan_gated_delta(cu, H, cp, 512 if cp else 0, device=DEV))
        assert torch.equal(o[cu[1]:], want) and torch.equal(s[1:], sw)
        if not cp:
            first, s_first = o[:cu[1]], s[:1]
        else:
            close("state", s[:1], s_first.double(), 2 * STATE_TOL)
            assert (o[:cu[1]].float() - first.float()).abs().max() <= (2 * HALF + 2 * STATE_TOL) * first.float().abs().max()
