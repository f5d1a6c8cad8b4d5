"""GPU tests of beam search's selection against plain 64-bit arithmetic on the
host. Parents and tokens are compared exactly: the candidates of one beam are
ordered by their logits, and those of two random beams are apart by far more
than the error of the log-sum-exp, or tie exactly. Scores are fp32 roundings of
64-bit values, 2^-24 relative. The log-sum-exp adds what its terms are off by,
relative to their sum: 2^-23 for exp2's last bit and 2^-24 for one fp32
addition, 1.8e-7 in all, and 2e-7 with the fp64 rest."""
import math

import pytest
import torch

import kda_chunked_delta_amd as kda
from kda_inputs import draw_decode

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
INF = float("inf")
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def say(*a):
    print(*a, flush=True)


def plain(logits, scores, n, finished=None, eos=None):
    x = torch.nan_to_num(logits.cpu().double(), nan=-INF, posinf=INF, neginf=-INF)
    s = torch.nan_to_num(scores.cpu().double(), nan=-INF, posinf=INF, neginf=-INF)
    B, W, V = x.shape
    top = x.amax(-1, keepdim=True)
    d = torch.where(x == top, torch.zeros_like(x), x - top)
    d = torch.where(top == -INF, torch.full_like(x, -INF), d - d.exp().sum(-1, keepdim=True).log())
    v = torch.where(x == -INF, torch.full_like(x, -INF), d + s[..., None])
    v = torch.nan_to_num(v, nan=-INF, posinf=INF, neginf=-INF)
    if finished is not None:
        only = torch.full_like(v, -INF)
        only[..., eos] = s
        v = torch.where(finished.cpu()[..., None], only, v)
    # by value, then by beam, then by logit (which resolves more than a value does), then by token
    inner = torch.where(v == -INF, v, x).sort(dim=-1, descending=True, stable=True).indices
    v = v.gather(2, inner).view(B, W * V)
    best, at = v.sort(dim=-1, descending=True, stable=True)
    best, at = best[:, :n], at[:, :n]
    at = at // V * V + inner.view(B, W * V).gather(1, at)
    parents, tokens = at // V, at % V
    done = None
    if eos is not None:
        done = tokens == eos
        if finished is not None:
            done |= finished.cpu().gather(1, parents)
    return best, parents.int(), tokens.int(), done


def check(logits, scores, n=None, **kw):
    got = kda.beam_select(logits, scores, n=n, **kw)
    want = plain(logits, scores, logits.shape[1] if n is None else n, **kw)
    assert torch.equal(got[1].cpu(), want[1]), (got[1].cpu() != want[1]).nonzero()[:4]
    assert torch.equal(got[2].cpu(), want[2]), (got[2].cpu() != want[2]).nonzero()[:4]
    assert (got[3] is None) == (want[3] is None) and (want[3] is None or torch.equal(got[3].cpu(), want[3]))
    g, w = got[0].cpu().double(), want[0]
    assert torch.equal(torch.isfinite(g), torch.isfinite(w)) and torch.equal(g[~torch.isfinite(g)], w[~torch.isfinite(w)])
    f = torch.isfinite(w)
    assert ((g - w).abs()[f] <= 2.0 ** -24 * w.abs()[f] + 2e-7).all(), (g - w).abs()[f].max()
    return got


def make(B, W, V, dtype, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed + B + W + V)
    x = (3 * torch.randn(B, W, V, generator=g, device=DEV)).to(dtype)
    s = -8 * torch.rand(B, W, generator=g, device=DEV)
    return x, s


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,W,V,n", [(1, 1, 1, 1), (1, 2, 1, 2), (2, 3, 5, 15), (3, 4, 1000, 4), (1, 4, 32000, 8),
                                     (5, 5, 2041, 5), (2, 3, 8185, 6), (2, 64, 777, 64), (7, 2, 50021, 33),
                                     (80, 8, 8193, 16), (1, 1, 200001, 64)])
def test_sizes_and_types(B, W, V, n, dtype):
    say("case", B, W, V, n, dtype)
    check(*make(B, W, V, dtype), n=n)


@pytest.mark.parametrize("dtype", TYPES)
def test_finished_beams_and_masks(dtype):
    say("case finished", dtype)
    x, s = make(9, 6, 4001, dtype)
    x[:, :, 3::4] = -INF
    x[1, 2] = -INF              # a row whose mask leaves nothing
    x[2] = -INF                 # a batch entry with nothing left
    x[3, :, 5:] = -INF          # fewer candidates than are asked for
    x[4, 0, 7] = float("nan")
    x[4, 1] = float("nan")
    x[5, 3, [17, 19]] = INF     # they share the row
    x[6] = torch.finfo(dtype).min
    s[7, 1:] = -INF             # the first step: one live beam
    s[8] = -INF
    fin = torch.zeros(9, 6, dtype=torch.bool, device=DEV)
    fin[0, 1] = fin[3, 2] = fin[8, 4] = True
    fin[5] = True
    for n in (6, 12, 64):
        check(x, s, n=n, finished=fin, eos=5)
        check(x, s, n=n, finished=fin, eos=0)
        check(x, s, n=n, eos=4000)
        check(x, s, n=n)


def test_scores_that_are_not_finite():
    x, s = make(4, 3, 100, torch.float32)
    s[0, 0], s[1, 1], s[2, 2] = INF, float("nan"), -INF
    x[0, 0, 4] = -INF
    x[3, 1, 9] = INF
    s[3, 1] = INF
    check(x, s, n=10)


@pytest.mark.parametrize("V", [3, 300, 9000])
def test_ties_go_to_the_lowest_index(V):
    x = torch.zeros(2, 4, V, device=DEV)
    x[1, :, ::2] = -0.0
    s = torch.zeros(2, 4, device=DEV)
    check(x, s, n=12)
    s[:, 2] = 1.0
    check(x, s, n=12)
    # equal beams
    y, _ = make(1, 1, V, torch.bfloat16)
    check(y.expand(3, 4, V).contiguous(), torch.full((3, 4), -2.0, device=DEV), n=12)


@pytest.mark.parametrize("W,V,n", [(8, 20000, 16), (4, 9000, 7), (3, 50000, 33)])
def test_more_ties_than_are_ranked_at_once(W, V, n):
    """Equal logits and scores: every candidate ties with every other."""
    say("case all tie", W, V, n)
    x = torch.full((2, W, V), 0.5, device=DEV)
    s = torch.full((2, W), -3.0, device=DEV)
    x[1, :, 100:] = -1.0  # a hundred per beam, in the first chunk
    check(x, s, n=n)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,shift", [(0, 1), (3, 0), (5, 3)])
def test_strided_rows(dtype, pad, shift):
    """A slice of a padded vocabulary, at any element alignment."""
    say("case strides", dtype, pad, shift)
    whole, s = make(3, 4, 3000 + pad + shift, dtype)
    x = whole[:, :, shift:3000 + shift]
    check(x, s, n=8)
    a, b = kda.beam_select(x, s, n=8), kda.beam_select(x.contiguous(), s, n=8)
    assert torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])


def test_large_logits():
    """A spread of logits at which exp under- and overflows without the maximum."""
    x, s = make(2, 3, 5000, torch.float32)
    check(x * 1e4, s * 100, n=8)
    check(x * 1e30, s, n=8)
    check(x * 1e-30, s, n=8)


def test_empty_batch_and_refusals():
    x, s = make(2, 3, 50, torch.float32)
    out = kda.beam_select(x[:0], s[:0], eos=1)
    assert [tuple(o.shape) for o in out] == [(0, 3)] * 4
    fin = torch.zeros(2, 3, dtype=torch.bool, device=DEV)
    for call in (lambda: kda.beam_select(x.double(), s), lambda: kda.beam_select(x, s.double()),
                 lambda: kda.beam_select(x, s[:1]), lambda: kda.beam_select(x[0], s), lambda: kda.beam_select(x, s, n=0),
                 lambda: kda.beam_select(x, s, n=65), lambda: kda.beam_select(x, s, finished=fin),
                 lambda: kda.beam_select(x, s, finished=fin, eos=50), lambda: kda.beam_select(x, s, eos=-1),
                 lambda: kda.beam_select(x, s, finished=fin.int(), eos=1), lambda: kda.beam_select(x[:, :, ::2], s),
                 lambda: kda.beam_select(x.transpose(0, 1), s.t().contiguous()), lambda: kda.beam_select(x.cpu(), s)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(kda.KDAError):
        kda.beam_select(x[:, :, :1], s, n=4)
    with pytest.raises(kda.KDAError):
        kda.beam_select(torch.zeros(1, 65, 4, device=DEV), torch.zeros(1, 65, device=DEV), n=4)


def test_two_streams_and_repetition():
    cases = [make(4, 4, 40000, torch.bfloat16, seed=i) for i in range(2)]
    want = [kda.beam_select(x, s, n=8) for x, s in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(4):
        for (x, s), st in zip(cases, streams):
            with torch.cuda.stream(st):
                got.append(kda.beam_select(x, s, n=8))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        for a, b in zip(g[:3], want[i % 2][:3]):
            assert torch.equal(a, b)


def test_beam_search_over_the_state_pool():
    """Beam search as it is used: decode over a pool, select, reorder, with
    every step in a graph, against the same search on the host in 64 bits with
    the states copied out for every beam."""
    B, W, H, V, steps, eos = 2, 3, 2, 37, 6, 5
    g = torch.Generator(device=DEV).manual_seed(7)
    emb = torch.randn(V, H, 128, generator=g, device=DEV)
    emb = (emb / emb.norm(dim=-1, keepdim=True)).bfloat16()
    val = torch.randn(V, H, 128, generator=g, device=DEV).bfloat16()
    gate = -torch.rand(V, H, generator=g, device=DEV)
    beta = torch.rand(V, H, generator=g, device=DEV)
    head = torch.randn(H * 128, V, generator=g, device=DEV)
    pool = 0.1 * torch.randn(B * W + 2, H, 128, 128, generator=g, device=DEV)
    slots = torch.tensor([[4, 1, 6], [0, 7, 3]], dtype=torch.int32, device=DEV)
    pool[slots.long()] = pool[slots[:, :1].long()].clone()  # one prompt per batch entry
    tokens = torch.full((B, W), 2, dtype=torch.int32, device=DEV)
    scores = torch.tensor([[0.0, -INF, -INF]] * B, device=DEV)
    fin = torch.zeros(B, W, dtype=torch.bool, device=DEV)
    states = pool[slots.long()].cpu().double()
    h = dict(tokens=tokens.cpu(), scores=scores.cpu().double(), fin=fin.cpu())

    def step():
        t = tokens.view(-1).long()
        o = kda.gated_delta_decode(emb[t], emb[t], val[t], gate[t], beta[t], pool, slots=slots.view(-1))
        logits = (o.float().view(B * W, H * 128) @ head).view(B, W, V)
        new_scores, parents, new_tokens, new_fin = kda.beam_select(logits, scores, finished=fin, eos=eos)
        slots.copy_(kda.beam_reorder(pool, slots, parents))
        scores.copy_(new_scores)
        tokens.copy_(new_tokens)
        fin.copy_(new_fin)
        return logits

    saved = [x.clone() for x in (pool, slots, scores, tokens, fin)]
    step()
    for x, y in zip((pool, slots, scores, tokens, fin), saved):
        x.copy_(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        logits = step()
    for x, y in zip((pool, slots, scores, tokens, fin), saved):
        x.copy_(y)
    f = lambda x: x.cpu().double()
    for it in range(steps):
        graph.replay()
        torch.cuda.synchronize()
        # the host's step, from the library's logits for the choice (they are bf16 outputs times a matrix)
        t = h["tokens"].view(-1).long()
        k, v, gm, b = f(emb)[t], f(val)[t], f(gate)[t].exp(), f(beta)[t]
        S = states.view(B * W, H, 128, 128) * gm[..., None, None]
        e = v - (S * k[..., None]).sum(-2)
        S = S + b[..., None, None] * k[..., None] * e[..., None, :]
        o = (S * k[..., None]).sum(-2)
        want = (o.reshape(B * W, H * 128) @ f(head)).view(B, W, V)
        # one bf16 rounding of o per term, and the fp32 product's sums
        bound = (o.abs().reshape(B * W, H * 128) @ f(head).abs()).view(B, W, V) * (2.0 ** -8 + 1e-4) + 1e-4
        assert ((f(logits) - want).abs() <= bound).all()
        best, parents, toks, done = plain(logits, h["scores"].float(), W, h["fin"], eos)
        assert torch.equal(tokens.cpu(), toks) and torch.equal(fin.cpu(), done)
        assert torch.allclose(f(scores), best, rtol=2.0 ** -22, atol=1e-6)
        states = S.view(B, W, H, 128, 128).gather(1, parents.long()[..., None, None, None].expand(-1, -1, H, 128, 128))
        h = dict(tokens=toks, scores=f(scores), fin=done)
        got = f(pool[slots.long()])
        live = torch.isfinite(best)
        assert (got - states)[live].norm() <= 1e-5 * states[live].norm()


def test_logits_beyond_2_31_elements():
    """The last batch entries of 4.4 GB of logits select what they select alone."""
    B, W, V = 33, 8, 8200000
    say("case logits beyond 2^31 elements")
    x = torch.empty(B, W, V, dtype=torch.bfloat16, device=DEV)
    x.normal_(generator=torch.Generator(device=DEV).manual_seed(3))
    x[:, :, 1234567] = torch.arange(20, 20 + W, device=DEV).to(torch.bfloat16)  # each beam's first, all apart
    s = torch.linspace(-1.0, 0.0, B * W, device=DEV).view(B, W)
    got = kda.beam_select(x, s, n=W)
    alone = kda.beam_select(x[-2:].contiguous(), s[-2:], n=W)
    for a, b in zip(got[1:3], alone[1:3]):
        assert torch.equal(a[-2:], b)
    # two log-sum-exps, each within 2e-7, and two roundings
    assert ((got[0][-2:] - alone[0]).abs() <= 4e-7 + 2.0 ** -23 * alone[0].abs()).all()
