"""GPU tests of the processing of logits against the definition, row by row in
64 bits.

Tolerance. The kernel computes in fp32: up to five operations, each off by at
most 2^-24 of its result, whose magnitudes the sum of the terms' bounds; then one
rounding to the logits' type, half a step of the result. Logits that nothing
applies to keep their bits."""
import pytest
import torch

import kda_chunked_delta_amd as kda

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
NEG = float("-inf")
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def make(R, V, L, K, dtype, seed, mask=True):
    gen = torch.Generator().manual_seed(seed)
    d = dict(logits=(3.0 * torch.randn(R, V, generator=gen)).to(dtype))
    if L:
        # few distinct tokens, so that they repeat; padding and tokens outside the vocabulary among them
        few = torch.randint(0, V, (R, max(1, L // 3)), generator=gen)
        t = few.gather(1, torch.randint(0, few.shape[1], (R, L), generator=gen))
        t[torch.rand(R, L, generator=gen) < 0.1] = -1
        t[:, L // 2] = V
        t[:, L // 3] = V - 1
        d.update(tokens=t.int(), lengths=torch.randint(0, L + 1, (R,), generator=gen).int(),
                 prompt_lengths=torch.randint(0, L + 1, (R,), generator=gen).int(),
                 repetition=0.7 + torch.rand(R, generator=gen), frequency=torch.rand(R, generator=gen) - 0.3,
                 presence=torch.rand(R, generator=gen) - 0.3)
        d["lengths"][0] = L
        if R > 2:
            d["lengths"][1], d["lengths"][2] = -3, L + 5
            d["prompt_lengths"][0], d["prompt_lengths"][2] = -1, L // 2
    if K:
        bt = torch.randint(0, V, (R, K), generator=gen)
        bt[:, -1] = bt[:, 0]  # the same token twice: the last entry counts
        bt[:, K // 2] = -1
        if L:
            bt[:, K // 3] = d["tokens"][:, 0].clamp(0, V - 1)
        d.update(bias_tokens=bt.int(), bias=2.0 * torch.randn(R, K, generator=gen))
    if mask:
        words = -(-V // 32)
        m = torch.randint(-2**31, 2**31, (R, words), generator=gen)
        some = torch.rand(R, words, generator=gen)
        m[some < 0.3] = -1
        m[some > 0.8] = 0
        m[0] = 0  # a row without an allowed token
        if R > 1:
            m[1] = -1
        d["allowed"] = m.int()
    return {n: x.to(DEV) for n, x in d.items()}


def reference(d):
    """(values in 64 bits, how far the kernel's may be off)"""
    x = d["logits"].double().cpu()
    off = torch.zeros_like(x)
    get = lambda n, r: d[n][r].double().cpu() if n in d else None
    R, V = x.shape
    eps = torch.finfo(d["logits"].dtype).eps / 2
    tiny = torch.finfo(d["logits"].dtype).tiny * eps  # half a step of the smallest numbers
    for r in range(R):
        if "tokens" in d:
            t = d["tokens"][r].cpu().tolist()
            n = min(max(int(d["lengths"][r]), 0), len(t)) if "lengths" in d else len(t)
            p = int(d["prompt_lengths"][r]) if "prompt_lengths" in d else 0
            every, past = {}, {}
            for i, tok in enumerate(t[:n]):
                if 0 <= tok < V:
                    every[tok] = 1
                    if i >= p:
                        past[tok] = past.get(tok, 0) + 1
            if "repetition" in d:
                f = get("repetition", r)
                for tok in every:
                    x[r, tok] = x[r, tok] / f if x[r, tok] > 0 else x[r, tok] * f
                    off[r, tok] += x[r, tok].abs()
            if "frequency" in d or "presence" in d:
                f = get("frequency", r) if "frequency" in d else 0.0
                pr = get("presence", r) if "presence" in d else 0.0
                for tok, m in past.items():
                    x[r, tok] -= f * m + pr
                    off[r, tok] += 3 * (abs(f * m) + abs(pr) + x[r, tok].abs())
        if "bias" in d:
            last = {}
            for j, tok in enumerate(d["bias_tokens"][r].tolist()):
                if 0 <= tok < V:
                    last[tok] = j
            for tok, j in last.items():
                x[r, tok] += get("bias", r)[j]
                off[r, tok] += get("bias", r)[j].abs() + x[r, tok].abs()
        if "allowed" in d:
            bits = (d["allowed"][r].cpu()[:, None] >> torch.arange(32)) & 1
            gone = bits.reshape(-1)[:V] == 0
            x[r, gone] = NEG
            off[r, gone] = 0
    fine = torch.isfinite(x)
    tol = torch.where(fine & (off > 0), 2.0 ** -24 * off + eps * x.abs() + tiny, 0.0)
    return x, tol


def check(d, out, name=""):
    want, tol = reference(d)
    got = out.double().cpu()
    same = got == want  # infinities, and what nothing applies to
    err = torch.where(same, 0.0, (got - want).abs())
    worst = (err / tol.clamp(min=1e-300)).where(~same, torch.zeros(())).max().item() if err.numel() else 0.0
    print("  %-20s largest error %.2f of its tolerance" % (name, worst), flush=True)
    assert (same | (err <= tol)).all(), name


def run(d, **kw):
    out = kda.logits_process(**d, **kw)
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("R,V,L,K", [(1, 1, 1, 1), (3, 5, 7, 2), (4, 31, 9, 3), (2, 2048, 40, 4), (5, 2049, 200, 9),
                                     (3, 8200, 1000, 300), (70, 65541, 70, 5)])
def test_everything(R, V, L, K, dtype):
    d = make(R, V, L, K, TYPES[dtype], seed=R + V)
    out = run(d)
    assert out.shape == (R, V) and out.dtype == TYPES[dtype] and out.stride(0) * out.element_size() % 128 == 0
    check(d, out, "new")
    place = d["logits"].clone()
    got = run({**d, "logits": place}, out=place)
    assert got is place and torch.equal(place, out)


@pytest.mark.parametrize("parts", [("repetition",), ("frequency",), ("presence",), ("repetition", "presence"), ("bias",),
                                   ("allowed",), ("frequency", "bias"), ("bias", "allowed"), ()])
@pytest.mark.parametrize("lists", [(), ("lengths", "prompt_lengths"), ("prompt_lengths",)])
def test_parts(parts, lists):
    full = make(4, 3001, 120, 7, torch.float32, seed=len(parts))
    keep = set(parts) | {"logits"} | ({"bias_tokens"} if "bias" in parts else set())
    if set(parts) & {"repetition", "frequency", "presence"}:
        keep |= {"tokens"} | set(lists)
    d = {n: x for n, x in full.items() if n in keep}
    check(d, run(d), "+".join(parts))
    place = d["logits"].clone()
    check(d, run({**d, "logits": place}, out=place), "in place")


def test_no_new_rounding_without_a_reason():
    """Logits that nothing applies to keep their bits: NaN, infinities, zeros with a sign, subnormal numbers."""
    for dtype in TYPES.values():
        x = torch.randn(3, 1000, device=DEV).to(dtype)
        tiny = torch.finfo(dtype).tiny / 4
        x[:, 5:11] = torch.tensor([float("nan"), float("inf"), NEG, -0.0, tiny, -tiny], device=DEV).to(dtype)
        t = torch.tensor([[20], [21], [-1]], dtype=torch.int32, device=DEV)
        one = torch.ones(3, device=DEV)
        out = kda.logits_process(x, tokens=t, presence=one)
        bits = torch.int32 if dtype == torch.float32 else torch.int16
        same = out.contiguous().view(bits) == x.view(bits)
        assert same.sum() == 3 * 1000 - 2 and not same[0, 20] and not same[1, 21]


def test_values_that_are_not_finite():
    x = torch.tensor([[float("nan"), float("inf"), NEG, 1.0, float("nan"), float("inf"), NEG, 2.0]], device=DEV)
    t = torch.tensor([[0, 1, 2, 3]], dtype=torch.int32, device=DEV)
    two = torch.full((1,), 2.0, device=DEV)
    allowed = torch.tensor([[0b10001111]], dtype=torch.int32, device=DEV)  # NaN and infinities behind the mask
    for dtype in TYPES.values():
        out = kda.logits_process(x.to(dtype), tokens=t, repetition=two, presence=two, allowed=allowed).float()[0].tolist()
        assert out[0] != out[0] and out[1:] == [float("inf"), NEG, 0.5 - 2.0, NEG, NEG, NEG, 2.0]
        # a bias of -inf forbids a token, and a mask wins over one of +inf
        b = torch.tensor([[NEG, float("inf")]], device=DEV)
        bt = torch.tensor([[7, 4]], dtype=torch.int32, device=DEV)
        out = kda.logits_process(x.to(dtype), bias=b, bias_tokens=bt, allowed=allowed).float()[0].tolist()
        assert out[4] == NEG and out[7] == NEG


def test_long_histories():
    d = make(3, 2500, 20000, 0, torch.float32, seed=7)
    d["tokens"][1] = 17  # one token over and over
    d["lengths"] = torch.full((3,), 20000, dtype=torch.int32, device=DEV)
    d["frequency"] *= 0.01
    check(d, run(d), "long")


@pytest.mark.parametrize("L", [1, 4096, 4097, 8193, 16383, 16384])
@pytest.mark.parametrize("K", [0, 70, 8192])
def test_room_for_histories_and_biases(L, K):
    """Histories at the borders of the word sizes and of the room for them, in calls with many rows and with few:
    the same rows give the same results."""
    d = make(4, 5000, L, K, torch.float32, seed=L + K)
    d["lengths"] = torch.full((4,), L, dtype=torch.int32, device=DEV)
    d["tokens"][1] = torch.arange(L, device=DEV, dtype=torch.int32) % 5000  # most of them different
    d["frequency"] *= 0.01
    few = run(d)
    check(d, few, "%d %d" % (L, K))
    many = {n: x.repeat(150, *[1] * (x.dim() - 1)) for n, x in d.items()}
    assert torch.equal(run(many), few.repeat(150, 1))


@pytest.mark.parametrize("dtype", list(TYPES))
def test_strides_and_alignment(dtype):
    """Rows of a larger buffer at any element, input and output at different ones, lists with padding behind them;
    what lies between the rows stays."""
    d = make(5, 2100, 30, 4, TYPES[dtype], seed=8)
    want = run(d).clone()
    for off in (1, 2, 3, 5):
        buf = torch.randn(5, 2100 + 13, device=DEV).to(TYPES[dtype])
        big = torch.full((5, 2100 + 7), 9.0, device=DEV).to(TYPES[dtype])
        x, y = buf[:, off:off + 2100], big[:, off - 1:off - 1 + 2100]
        x.copy_(d["logits"])
        wide = {n: torch.cat([d[n], torch.zeros_like(d[n][:, :off])], 1)[:, :d[n].shape[1]]
                for n in ("tokens", "bias_tokens", "bias", "allowed")}
        out = run({**d, **wide, "logits": x}, out=y)
        assert out is y and torch.equal(y, want)
        edge = torch.ones(2107, dtype=torch.bool, device=DEV)
        edge[off - 1:off - 1 + 2100] = False
        assert (big[:, edge] == 9.0).all()
        keep = buf.clone()
        run({**d, "logits": x}, out=x)
        assert torch.equal(x, want) and torch.equal(buf[:, :off], keep[:, :off])
        assert torch.equal(buf[:, off + 2100:], keep[:, off + 2100:])


def test_beams_and_shared_lists():
    d = make(6, 700, 20, 3, torch.bfloat16, seed=9)
    want = run(d)
    three = {n: x.view(2, 3, *x.shape[1:]) for n, x in d.items()}
    out = run(three)
    assert out.shape == (2, 3, 700) and torch.equal(out.reshape(6, 700), want)
    # one list for all rows
    for n in ("tokens", "allowed"):
        one = {**d, n: d[n][2:3].expand_as(d[n])}
        assert torch.equal(run(one), run({**d, n: one[n].contiguous()}))
    one = {**d, "bias": d["bias"][:1].expand_as(d["bias"]), "bias_tokens": d["bias_tokens"][:1].expand_as(d["bias"])}
    assert torch.equal(run(one), run({n: x.contiguous() for n, x in one.items()}))


def test_nothing_to_do():
    x = torch.randn(3, 77, device=DEV)
    assert torch.equal(kda.logits_process(x), x)
    assert kda.logits_process(x, out=x) is x
    assert kda.logits_process(x[:0]).shape == (0, 77)
    none = torch.zeros(3, 0, dtype=torch.int32, device=DEV)
    assert torch.equal(kda.logits_process(x, tokens=none, presence=torch.ones(3, device=DEV)), x)
    assert torch.equal(kda.logits_process(x, bias_tokens=none, bias=none.float()), x)


def test_offsets_beyond_32_bits():
    R, V = 20000, 131072  # 5.2 GB of bf16: the last row is past 2^32 bytes and 2^31 elements
    x = torch.zeros(R, V, dtype=torch.bfloat16, device=DEV)
    x[-1] = torch.randn(V, device=DEV).bfloat16()
    t = torch.full((1, 1), V - 1, dtype=torch.int32, device=DEV).expand(R, 1)
    p = torch.zeros(R, device=DEV)
    p[-1] = 2.0
    last = kda.logits_process(x[-1:], tokens=t[:1], presence=p[-1:])
    assert last[0, -1] == (x[-1, -1].float() - 2.0).bfloat16()
    assert torch.equal(kda.logits_process(x, tokens=t, presence=p)[-1], last[0])
    kda.logits_process(x, tokens=t, presence=p, out=x)
    assert torch.equal(x[-1], last[0]) and not x[:-1].any()


def test_graph_and_streams():
    d = make(4, 5000, 60, 5, torch.bfloat16, seed=10)
    want = run(d)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = kda.logits_process(**d)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        out.zero_()
        assert torch.equal(run(d), want)
    other = make(4, 5000, 60, 5, torch.bfloat16, seed=11)
    want2 = run(other)
    for n in d:
        d[n].copy_(other[n])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want2)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = kda.logits_process(**other)
    side.synchronize()
    assert torch.equal(got, want2)


def test_a_run_of_beam_search():
    """Linear attention layers, logits, penalties and a mask, selection, states and histories that follow their
    parents: as the operators are used together, against plain torch in 64 bits."""
    D, H, B, W, V, steps = 128, 2, 2, 3, 300, 6
    gen = torch.Generator().manual_seed(12)
    emb = torch.randn(V, 3 * H * D, generator=gen).to(DEV)
    head = (torch.randn(H * D, V, generator=gen) / 8).to(DEV)
    g = torch.tensor([-0.3, -0.02], device=DEV)
    prompt = torch.randint(0, V, (B, 40), generator=gen).to(DEV)
    pres, freq, rep = (torch.full((B, W), x, device=DEV) for x in (0.5, 0.25, 1.25))
    allowed = torch.randint(-2**31, 2**31, (1, 1, -(-V // 32)), generator=gen).int().to(DEV).expand(B, W, -1)

    def qkv(tokens):
        return [x.bfloat16().contiguous().view(*tokens.shape, H, D) for x in emb[tokens].chunk(3, -1)]

    # the prompts' states, forked to their beams
    q, k, v = qkv(prompt)
    _, s = kda.linear_attention_prefill(q, k, v, g, output_final_state=True, scale=0.05)
    pool = torch.zeros(B * W + 2, H, D, D, device=DEV)
    pool[: B * W] = s.repeat_interleave(W, 0)
    slots = torch.arange(B * W, dtype=torch.int32, device=DEV).view(B, W)
    history = torch.full((B, W, 40 + steps), -1, dtype=torch.int32, device=DEV)
    history[:, :, :40] = prompt[:, None]
    scores = torch.tensor([0.0] + [NEG] * (W - 1), device=DEV).repeat(B, 1)
    prompts = torch.full((B, W), 40, dtype=torch.int32, device=DEV)
    # the same in 64 bits
    S = torch.zeros(B, H, D, D, dtype=torch.float64, device=DEV)
    qd, kd, vd = (x.double() for x in (q, k, v))
    for t in range(40):
        S = torch.exp(g.double())[:, None, None] * S + kd[:, t, :, :, None] * vd[:, t, :, None, :]
    assert ((s.double() - S).norm() <= 1e-5 * S.norm()).all()
    S = S.repeat_interleave(W, 0)
    last = prompt[:, -1:].repeat(1, W)
    for step in range(steps):
        n = torch.full((B, W), 40 + step, dtype=torch.int32, device=DEV)
        q, k, v = qkv(last.view(-1))
        o = kda.linear_attention_decode(q, k, v, g, pool, scale=0.05, slots=slots.view(-1))
        logits = (o.view(B * W, H * D).float() @ head).view(B, W, V)
        logits = kda.logits_process(logits, tokens=history, lengths=n, prompt_lengths=prompts, repetition=rep,
                                    frequency=freq, presence=pres, allowed=allowed)
        new, parents, tokens, _ = kda.beam_select(logits, scores)
        slots = kda.beam_reorder(pool, slots, parents)
        # 64 bits, on the same choices of the steps before
        qd, kd, vd = (x.double() for x in (q, k, v))
        S = torch.exp(g.double())[:, None, None] * S + kd[..., None] * vd[..., None, :]
        od = 0.05 * (S * qd[..., None]).sum(2)
        assert ((o.double() - od).norm() <= 2.0 ** -8 * od.norm()).all()
        x = (o.view(B * W, H * D).float() @ head).double()
        d = dict(logits=x.view(B * W, V).float(), tokens=history.view(B * W, -1), lengths=n.view(-1),
                 prompt_lengths=prompts.view(-1), repetition=rep.view(-1), frequency=freq.view(-1),
                 presence=pres.view(-1), allowed=allowed.reshape(B * W, -1))
        check(d, logits.view(B * W, V), "step %d" % step)
        total = torch.log_softmax(logits.double(), -1) + scores.double()[..., None]
        best = total.view(B, -1).sort(-1, descending=True).values[:, :W]
        assert (new.double() - best).abs().max() <= 1e-5 * (1 + best.abs().max())
        # what follows the parents
        at = parents.long()
        S = S.view(B, W, H, D, D).gather(1, at[:, :, None, None, None].expand(B, W, H, D, D)).view(B * W, H, D, D)
        history = history.gather(1, at[:, :, None].expand_as(history)).contiguous()
        history[:, :, 40 + step] = tokens
        last, scores = tokens.long(), new
        state = pool[slots.view(-1).long()]
        assert ((state.double() - S).norm() <= 1e-5 * S.norm()).all()


def test_refusals():
    d = make(4, 100, 10, 3, torch.float32, seed=13)
    x, t = d["logits"], d["tokens"]
    f = torch.ones(4, device=DEV)
    for bad in (dict(logits=x.double()), dict(logits=x[0]), dict(logits=x.t()), dict(logits=x.cpu()),
                dict(logits=x[:, ::2]), dict(out=x.half()), dict(out=x[:2]), dict(tokens=t.long(), presence=f),
                dict(tokens=t[:2], presence=f), dict(presence=f), dict(lengths=d["lengths"]),
                dict(tokens=t, presence=f.double()), dict(tokens=t, presence=f[:2]), dict(tokens=t, frequency=f[None]),
                dict(tokens=t.t().contiguous().t(), presence=f), dict(tokens=t.cpu(), presence=f),
                dict(bias=d["bias"]), dict(bias_tokens=d["bias_tokens"]),
                dict(bias=d["bias"][:, :2], bias_tokens=d["bias_tokens"]),
                dict(allowed=d["allowed"][:, :3]), dict(allowed=d["allowed"].long()), dict(logits=x[:, :0])):
        with pytest.raises(ValueError):
            kda.logits_process(**{"logits": x, **bad})
    with pytest.raises(kda.KDAError):  # shifted by a row
        kda.logits_process(x[1:], out=x[:3])
    buf = torch.zeros(4, 200, device=DEV)
    with pytest.raises(kda.KDAError):
        kda.logits_process(buf[:, :100], out=buf[:, 100:])  # between each other's rows
    with pytest.raises(kda.KDAError):
        kda.logits_process(x, allowed=x.view(torch.int32)[:, :4], out=x)


def test_a_history_without_penalties_changes_nothing():
    """Not even the bits of a NaN that is no quiet one."""
    x = torch.randn(3, 500, device=DEV).bfloat16()
    x.view(torch.int16)[:, 7] = 0x7f81
    t = torch.full((3, 4), 7, dtype=torch.int32, device=DEV)
    out = kda.logits_process(x, tokens=t)
    assert torch.equal(out.contiguous().view(torch.int16), x.view(torch.int16))
