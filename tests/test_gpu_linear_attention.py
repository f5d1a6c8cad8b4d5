"""GPU parity of linear attention (one log-decay per token and head, or per head)
with the per-token recurrence in 64 bits: chunked prefill, segmented prefill, and
decode of one or several tokens.

Tolerances. fp32 states, relative to the norm of the exact one: a token enters
with 24 bits, times a weight of 2^-22 (an exponential), and the running decay is an
fp32 product over the chunks that a state remembers, 2^-22 of each: 1e-5 bounds 40 of
them (decays that let more count are close to one, and rounded to 2^-24). Decode is fp32 throughout: 128-term sums,
2e-6. Outputs of the prefill are rounded twice to bf16 (the copy of the state,
the output), each by at most HALF = 2^-8 of its value; the decayed q . k products
are pairs, 2^-17. So one output is off by at most HALF of itself and of what it
would be with all signs positive; and over many independent outputs each rounding
has an rms of HALF / sqrt(3) at most: sqrt(2 / 3) HALF in the norm, held to HALF.
Outputs of the decode are rounded once."""
import math

import pytest
import torch

import kda_chunked_delta_amd as kda

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
D = 128
STATE_TOL, DECODE_TOL, HALF = 1e-5, 2e-6, 2.0 ** -8


def say(*a):
    print(*a, flush=True)


def make(lengths, H, seed, Hk=None, decay="token", states=True):
    gen = torch.Generator().manual_seed(seed)
    Hk = H if Hk is None else Hk
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    Tt = cu[-1]

    def normal(*shape):
        return torch.randn(*shape, generator=gen)

    if decay == "head":  # one per head, among them none at all
        g = -torch.exp2(-torch.arange(H).float())
        g[H - 1] = 0.0
    elif decay == "growth":
        g = 0.05 * normal(Tt, H)
    else:
        g = -torch.nn.functional.softplus(normal(Tt, H)) * {"token": 0.1, "strong": 30.0, "weak": 1e-4}[decay]
    d = dict(q=normal(Tt, Hk, D).bfloat16(), k=normal(Tt, Hk, D).bfloat16(), v=normal(Tt, H, D).bfloat16(), g=g)
    d = {n: x.to(DEV) for n, x in d.items()}
    d["s0"] = normal(len(lengths), H, D, D).to(DEV) if states else None
    d["cu_host"], d["cu"] = cu, torch.tensor(cu, dtype=torch.int32, device=DEV)
    return d


def recurrence(q, k, v, g, cu, s0, scale=1.0):
    """fp64, token by token. Also what the outputs would be with all signs positive."""
    rep = v.shape[1] // k.shape[1]
    q, k = (x.double().repeat_interleave(rep, 1) for x in (q, k))
    v, g = v.double(), g.double()
    gam = torch.exp(g if g.dim() == 2 else g.expand(v.shape[:2]))
    H = v.shape[1]
    out, mag = (torch.zeros(v.shape, dtype=torch.float64, device=v.device) for _ in range(2))
    S = torch.zeros(len(cu) - 1, H, D, D, dtype=torch.float64, device=v.device)
    if s0 is not None:
        S.copy_(s0)
    for i in range(len(cu) - 1):
        s, a = S[i], S[i].abs()
        for t in range(cu[i], cu[i + 1]):
            kv = k[t][:, :, None] * v[t][:, None, :]
            s = gam[t][:, None, None] * s + kv
            a = gam[t][:, None, None] * a + kv.abs()
            out[t] = scale * (s * q[t][:, :, None]).sum(1)
            mag[t] = abs(scale) * (a * q[t].abs()[:, :, None]).sum(1)
        S[i] = s
    return out, S, mag


def near(name, got, want, tol):
    g, w = got.double(), want.double()
    assert torch.isfinite(g).all(), name
    err, norm = (g - w).norm().item(), w.norm().item()
    say("  %-8s rel %.2e (tolerance %.2e)" % (name, err / norm if norm else err, tol))
    assert err <= tol * norm, (name, err, norm)
    return g - w


def check_prefill(d, o, s, scale=1.0, what=""):
    s0 = d["s0"]
    want, S, mag = recurrence(d["q"], d["k"], d["v"], d["g"], d["cu_host"], s0, scale)
    if want.numel():
        err = near("o " + what, o, want, HALF)
        assert (err.abs() <= HALF * want.abs() + HALF * 1.01 * mag).all()
    if s is not None:
        near("state " + what, s, S, STATE_TOL if s.dtype == torch.float32 else HALF)
        if s.dtype == torch.bfloat16:
            assert ((s.double() - S).abs() <= HALF * S.abs() + 40 * STATE_TOL * S.square().mean().sqrt()).all()


def prefill(d, mode="auto", scale=1.0, **kw):
    o, s = kda.linear_attention_prefill(d["q"], d["k"], d["v"], d["g"], cu_seqlens=d["cu"], cu_seqlens_host=d["cu_host"],
                                        initial_state=d["s0"], output_final_state=True, use_intracard_cp=mode,
                                        scale=scale, **kw)
    torch.cuda.synchronize()
    return o, s


@pytest.mark.parametrize("decay", ["token", "strong", "weak", "head", "growth"])
@pytest.mark.parametrize("lengths,H,Hk", [([1], 1, 1), ([31], 3, 1), ([32], 2, 2), ([33], 1, 1), ([64, 65], 4, 2),
                                          ([0, 1, 33, 7, 129, 0], 6, 2), ([300], 2, 2)])
def test_prefill(lengths, H, Hk, decay):
    d = make(lengths, H, seed=sum(lengths) + H, Hk=Hk, decay=decay, states=len(lengths) % 2 == 0)
    say(lengths, H, Hk, decay)
    check_prefill(d, *prefill(d, scale=0.7), scale=0.7)


def test_bf16_states():
    d = make([40, 0, 97], 4, seed=3, Hk=2)
    d["s0"] = d["s0"].bfloat16()
    o, s = prefill(d)
    assert s.dtype == torch.bfloat16
    check_prefill(d, o, s)
    assert torch.equal(s[1], d["s0"][1])
    d["s0"] = None
    o, s = prefill(d, state_dtype=torch.bfloat16)
    assert s.dtype == torch.bfloat16
    check_prefill(d, o, s)


@pytest.mark.parametrize("seg", [1, 3, 4])
@pytest.mark.parametrize("decay", ["token", "strong", "head", "weak"])
@pytest.mark.parametrize("state", [torch.float32, torch.bfloat16, None])
def test_segments(seg, decay, state):
    lengths, H = [290, 0, 1, 33, 32 * seg, 32 * seg + 1], 4
    d = make(lengths, H, seed=seg, Hk=2, decay=decay, states=state is not None)
    if state is not None:
        d["s0"] = d["s0"].to(state)
    plan = kda.plan_linear_attention(d["cu_host"], H, True, seg, device=DEV)
    assert plan.info()["uses_cp"] == 1
    say(seg, decay, state)
    o, s = prefill(d, plan=plan, state_dtype=state)
    check_prefill(d, o, s, what="cut")
    # again, with the states updated in place
    if state is not None:
        s0 = d["s0"].clone()
        o2, s2 = kda.linear_attention_prefill(d["q"], d["k"], d["v"], d["g"], cu_seqlens=d["cu"], plan=plan,
                                              cu_seqlens_host=d["cu_host"], initial_state=s0, final_state=s0)
        assert s2 is s0 and torch.equal(s2, s) and torch.equal(o2, o)
    whole, _ = prefill(d, mode=False, state_dtype=state)
    # the states that the outputs read differ by STATE_TOL at most, which flips some of their roundings
    near("whole", o, whole, HALF)


def test_auto_segments_long_prompts():
    d = make([9000], 2, seed=5, decay="weak")
    assert kda.plan_linear_attention(d["cu_host"], 2, "auto", device=DEV).info()["uses_cp"] == 1
    check_prefill(d, *prefill(d))


def test_forgetting():
    """A log-decay of -inf (or one whose exponential is zero) forgets the state exactly, wherever it stands."""
    d = make([100], 2, seed=6)
    at = [0, 31, 32, 50, 99]
    d["g"][at] = torch.tensor([-math.inf, -1e30], device=DEV)
    check_prefill(d, *prefill(d))
    cut = make([100], 2, seed=6)
    cut["g"][50] = -math.inf
    o, s = prefill(cut)
    tail = {n: cut[n][50:].contiguous() for n in "qkv"}
    g = cut["g"][50:].clone()
    g[0] = 0.0
    want, S, mag = recurrence(tail["q"], tail["k"], tail["v"], g, [0, 50], None)
    near("state", s, S, STATE_TOL)
    assert ((o[50:].double() - want).abs() <= HALF * want.abs() + 1.01 * HALF * mag).all()


def test_a_prompt_in_parts():
    d = make([179], 3, seed=8)
    o, s = prefill(d)
    part = lambda a, b: [d[n][a:b].contiguous() for n in ("q", "k", "v", "g")]
    oa, sa = kda.linear_attention_prefill(*part(0, 128), initial_state=d["s0"], output_final_state=True)
    ob, sb = kda.linear_attention_prefill(*part(128, 179), initial_state=sa, output_final_state=True)
    # cut between chunks, the parts do what the whole does
    assert torch.equal(torch.cat([oa, ob]), o) and torch.equal(sb, s)


def test_batched_form():
    d = make([40, 40], 2, seed=9)
    o, s = prefill(d)
    four = lambda x: x.view(2, 40, *x.shape[1:])
    out = torch.empty_like(four(d["v"]))
    o4, s4 = kda.linear_attention_prefill(*map(four, (d["q"], d["k"], d["v"], d["g"])), initial_state=d["s0"],
                                          output_final_state=True, out=out)
    assert o4.data_ptr() == out.data_ptr() and torch.equal(o4.view_as(o), o) and torch.equal(s4, s)
    h = make([40, 40], 2, seed=9, decay="head")
    o, _ = prefill(h)
    o4, none = kda.linear_attention_prefill(*map(four, (h["q"], h["k"], h["v"])), h["g"], initial_state=h["s0"])
    assert none is None and torch.equal(o4.view_as(o), o)


def test_a_decay_per_head_is_that_decay_for_every_token():
    d = make([70, 5], 3, seed=10, decay="head")
    o, s = prefill(d)
    d["g"] = d["g"].expand(75, 3).contiguous()
    o2, s2 = prefill(d)
    assert torch.equal(o, o2) and torch.equal(s, s2)


def test_values_that_are_not_finite_stay_in_their_head_and_sequence():
    d = make([70, 80], 3, seed=11)
    o, s = prefill(d)
    for bad in (math.nan, math.inf):
        x = {n: t.clone() if isinstance(t, torch.Tensor) else t for n, t in d.items()}
        x["v"][70 + 40, 1, 5] = bad
        o2, s2 = prefill(x)
        assert torch.equal(o2[:, [0, 2]], o[:, [0, 2]]) and torch.equal(o2[:70], o[:70])
        assert torch.equal(o2[70:102], o[70:102])  # the chunks before it
        assert torch.equal(s2[0], s[0]) and torch.equal(s2[1, [0, 2]], s[1, [0, 2]])
        keep = [c for c in range(D) if c != 5]
        assert torch.equal(o2[..., keep], o[..., keep]) and torch.equal(s2[..., keep], s[..., keep])
        assert not torch.isfinite(s2[1, 1, :, 5]).any()


# ---------------------------------------------------------------------------
# decode
# ---------------------------------------------------------------------------
def tokens(N, T, H, Hk, seed, fixed=False):
    d = make([T] * N, H, seed, Hk=Hk, decay="head" if fixed else "token")
    x = [d[n].view(N, T, *d[n].shape[1:]) for n in "qkv"]
    return x + [d["g"] if fixed else d["g"].view(N, T, H)], d


@pytest.mark.parametrize("fixed", [False, True])
@pytest.mark.parametrize("N,T,H,Hk", [(1, 1, 1, 1), (3, 1, 4, 2), (2, 5, 3, 1), (17, 2, 2, 2), (40, 1, 60, 60)])
def test_decode(N, T, H, Hk, fixed):
    args, d = tokens(N, T, H, Hk, seed=N + T, fixed=fixed)
    state = d["s0"].clone()
    o = kda.linear_attention_decode(*args, state, scale=0.8)
    want, S, _ = recurrence(d["q"], d["k"], d["v"], d["g"], d["cu_host"], d["s0"], 0.8)
    near("state", state, S, DECODE_TOL)
    err = near("o", o.view_as(want), want, HALF)
    rms = want.square().mean().sqrt()
    assert (err.abs() <= HALF * want.abs() + 40 * DECODE_TOL * (rms + want.abs())).all()
    # several tokens at once are so many calls
    again = d["s0"].clone()
    for t in range(T):
        o1 = kda.linear_attention_decode(*[x[:, t].contiguous() for x in args[:3]],
                                         args[3] if fixed else args[3][:, t].contiguous(), again, scale=0.8)
        assert torch.equal(o1, o[:, t])
    assert torch.equal(again, state)


def test_decode_slots():
    args, d = tokens(5, 2, 3, 3, seed=20)
    pool = torch.randn(9, 3, D, D, generator=torch.Generator().manual_seed(1)).to(DEV)
    before = pool.clone()
    slots = torch.tensor([7, -1, 0, 9, 3], dtype=torch.int32, device=DEV)
    o = kda.linear_attention_decode(*args, pool, slots=slots)
    live = torch.tensor([0, 2, 4], device=DEV)
    state = before[slots[live].long()].clone()
    o2 = kda.linear_attention_decode(*[x[live].contiguous() for x in args], state)
    assert torch.equal(o[live], o2) and not o[[1, 3]].any()
    before[slots[live].long()] = state
    assert torch.equal(pool, before)


def test_nothing_to_decode():
    args, d = tokens(2, 1, 3, 3, seed=21)
    s = d["s0"].clone()
    assert kda.linear_attention_decode(*[x[:0] for x in args], s[:0]).shape == (0, 1, 3, D)
    assert kda.linear_attention_decode(*[x[:, :0].contiguous() for x in args], s).shape == (2, 0, 3, D)
    assert torch.equal(s, d["s0"])


def test_prefill_then_decode():
    d = make([20, 1, 75], 2, seed=22)
    want, S, _ = recurrence(d["q"], d["k"], d["v"], d["g"], d["cu_host"], None)
    last = [c - 1 for c in d["cu_host"][1:]]
    head = [i for i in range(96) if i not in last]
    xs = [d[n] for n in ("q", "k", "v", "g")]
    _, s = kda.linear_attention_prefill(*[x[head] for x in xs], cu_seqlens=[0, 19, 19, 93], output_final_state=True)
    o = kda.linear_attention_decode(*[x[last] for x in xs], s)
    near("state", s, S, STATE_TOL)
    # the state's error reaches an output through 128 terms of its own norm
    near("o", o, want[last], HALF)


# ---------------------------------------------------------------------------
# graphs, streams, sizes, refusals
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("seg", [0, 2])
def test_graph(seg):
    d = make([150, 64, 3], 2, seed=30)
    plan = kda.plan_linear_attention(d["cu_host"], 2, seg > 0, seg, device=DEV)
    tok, _ = tokens(3, 1, 2, 2, seed=31)

    def step():
        o, s = kda.linear_attention_prefill(d["q"], d["k"], d["v"], d["g"], cu_seqlens=d["cu"], plan=plan,
                                            cu_seqlens_host=d["cu_host"], initial_state=d["s0"], output_final_state=True)
        return o, kda.linear_attention_decode(*tok, s), s

    want = [x.clone() for x in step()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(torch.equal(a, b) for a, b in zip(step(), want))
        for x in got:
            x.zero_()
    # other inputs in the same buffers
    other = make([150, 64, 3], 2, seed=32)
    for n in ("q", "k", "v", "g", "s0"):
        d[n].copy_(other[n])
    want = [x.clone() for x in step()]
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_streams():
    plan = kda.plan_linear_attention([0, 600], 2, True, 4, device=DEV)
    ds = [make([600], 2, seed=40 + i) for i in range(2)]
    want = [prefill(d, plan=plan) for d in ds]
    streams = [torch.cuda.Stream() for _ in ds]
    for _ in range(5):
        got = []
        for d, st in zip(ds, streams):
            with torch.cuda.stream(st):
                got.append(kda.linear_attention_prefill(d["q"], d["k"], d["v"], d["g"], plan=plan, cu_seqlens=d["cu"],
                                                        cu_seqlens_host=d["cu_host"], initial_state=d["s0"],
                                                        output_final_state=True))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))


def test_offsets_beyond_32_bits():
    """The last sequence of a batch whose tensors pass 4 GiB, and a slot as far into a pool, against the same alone."""
    H, lengths = 256, [65000, 1500, 70]  # 65 KiB of q a token
    gen = torch.Generator(device=DEV).manual_seed(50)
    Tt = sum(lengths)
    q, k, v = (torch.randn(Tt, H, D, generator=gen, device=DEV, dtype=torch.bfloat16) for _ in range(3))
    g = -0.1 * torch.rand(Tt, H, generator=gen, device=DEV)
    cu = [0, 65000, 66500, 66570]
    tail = [x[65000:].contiguous() for x in (q, k, v, g)]
    want, sw = kda.linear_attention_prefill(*tail, cu_seqlens=[0, 1500, 1570], output_final_state=True,
                                            use_intracard_cp=False)
    for cp in (False, True):
        o, s = kda.linear_attention_prefill(q, k, v, g, cu_seqlens=cu, output_final_state=True,
                                            plan=kda.plan_linear_attention(cu, H, cp, 512 if cp else 0, device=DEV))
        assert torch.equal(o[65000:], want) and torch.equal(s[1:], sw)
    del q, k, v, g, o
    pool = torch.zeros(300, H, D, D, device=DEV)  # 5 GB, 1.26e9 elements
    args = [x[:1] for x in tail]
    pool[299] = sw[0]
    state = sw[:1].clone()
    slots = torch.tensor([299], dtype=torch.int32, device=DEV)
    o = kda.linear_attention_decode(*args, pool, slots=slots)
    assert torch.equal(o, kda.linear_attention_decode(*args, state)) and torch.equal(pool[299], state[0])
    assert not pool[:299].any()


def test_refusals():
    d = make([40], 4, seed=60, Hk=2)
    q, k, v, g = (d[n] for n in "qkvg")
    call = kda.linear_attention_prefill
    for bad in (dict(q=q.half()), dict(k=k[:39]), dict(v=v[:, :3].contiguous()), dict(g=g[:, :2].contiguous()),
                dict(g=g[0, :2].contiguous()), dict(g=g.double()), dict(q=q.transpose(0, 1)), dict(k=k.cpu()),
                dict(cu_seqlens=[0, 39]), dict(cu_seqlens=[0, 20, 10, 40]), dict(initial_state=d["s0"][:, :2]),
                dict(initial_state=d["s0"], final_state=d["s0"].bfloat16()), dict(out=torch.empty_like(v).float()),
                dict(plan=kda.plan_linear_attention([0, 40], 2, device=DEV)),
                dict(state_dtype=torch.float16)):
        with pytest.raises(ValueError):
            call(**{**dict(q=q, k=k, v=v, g=g), **bad})
    with pytest.raises(kda.KDAError):  # a plan of another operator
        call(q, k, v, g, plan=kda.plan_gated_delta([0, 40], 4, device=DEV))
    with pytest.raises(kda.KDAError):
        kda.gated_delta_prefill(q, k, v, g, torch.ones_like(g), plan=kda.plan_linear_attention([0, 40], 4, device=DEV))
    with pytest.raises(kda.KDAError):
        call(q, k, v, g, out=v)
    with pytest.raises(kda.KDAError):
        call(q, k, v, g, scale=math.nan)
    plan = kda.plan_linear_attention([0, 7, 40], 4, device=DEV)
    cu = torch.tensor([0, 7, 40], dtype=torch.int32, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for kw in (dict(cu_seqlens=[0, 8, 40]), dict(cu_seqlens=d["cu"]), dict(plan=plan, cu_seqlens=[0, 7, 40])):
            with pytest.raises(ValueError):
                call(q, k, v, g, **kw)
        o, _ = call(q, k, v, g, cu_seqlens=cu, cu_seqlens_host=[0, 7, 40], plan=plan)
    graph.replay()
    torch.cuda.synchronize()
    want, _ = call(q, k, v, g, cu_seqlens=cu)
    assert torch.equal(o, want)
    args, t = tokens(3, 1, 4, 2, seed=61)
    s = t["s0"]
    dec = kda.linear_attention_decode
    for bad in (dict(q=args[0].half()), dict(k=args[1][:2]), dict(g=args[3][:, :, :2].contiguous()),
                dict(state=s.bfloat16()), dict(state=s[:2]), dict(slots=torch.zeros(2, dtype=torch.int32, device=DEV)),
                dict(out=torch.empty_like(args[2]).float())):
        with pytest.raises(ValueError):
            dec(**{**dict(zip(("q", "k", "v", "g"), args)), "state": s, **bad})
