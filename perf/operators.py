"""What the operators around the recurrent state cost: the gated delta rule (chunked prefill and
recurrent decode), beam search's selection with the reordering of states, and the page operations
of the state pool. `run` computes them in plain torch, or with `own` through the library."""
import math

import torch

own = False  # True: run() calls the library's operators

DEV = "cuda"
D = 128      # key and value channels of a state
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # a short prompt with one head: the smallest prefill, where latency counts
        dict(name="prefill_t64_h1", op="prefill", lengths="64", H=1, Hk=1, decay="strong", beta="fp32", state="none"),
        # a ragged batch with an empty and a one-token sequence, grouped value heads, bf16 beta and states
        dict(name="prefill_ragged_gva", op="prefill", lengths="0,1,33,700,129,64,1001,257", H=12, Hk=4, decay="gate",
             beta="bf16", state="bf16"),
        # the benchmark's packed batch: eight prompts of 512 to 4096 tokens, 32 heads, fp32 states continued
        dict(name="prefill_varlen8_h32", op="prefill", lengths="3779,1392,3289,3438,1776,2802,3054,617", H=32, Hk=32,
             decay="gate", beta="fp32", state="fp32"),
        # the benchmark's long prompt with few heads
        dict(name="prefill_long65536_h8", op="prefill", lengths="65536", H=8, Hk=8, decay="gate", beta="fp32",
             state="fp32"),
        # one sequence's next token
        dict(name="decode_n1_h32", op="decode", N=1, T=1, H=32, Hk=32, slots=False),
        # the benchmark's decode batch
        dict(name="decode_n256_h32", op="decode", N=256, T=1, H=32, Hk=32, slots=False),
        # four drafted tokens per sequence over a pool of states, grouped value heads, one padded entry
        dict(name="decode_n33_t4_gva", op="decode", N=33, T=4, H=12, Hk=4, slots=True),
        # beam search of one prompt, fp32 logits
        dict(name="beam_b1_w4_v32000", op="beam", B=1, W=4, V=32000, n=4, dtype="fp32", finished=False, masked=False),
        # a batch of prompts, twice as many candidates as beams, finished beams, masked tokens
        dict(name="beam_b32_w8_v131072", op="beam", B=32, W=8, V=131072, n=16, dtype="bf16", finished=True,
             masked=True),
        # the states of a beam batch follow their parents
        dict(name="reorder_b16_w4_h32", op="reorder", B=16, W=4, H=32),
        # one admission step: finished sequences freed, prefix snapshots forked, two states swapped
        dict(name="pages_p256_h32_f64", op="pages", P=256, H=32, F=64),
        # a half-empty pool is compacted
        dict(name="compact_p301_h12", op="compact", P=301, H=12),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "prefill", "decode", "decode", "beam", "beam", "reorder", "pages",
                     "compact"])
    if op == "prefill":
        Hk = rng.choice([1, 2, 4, 8, 12, 16])
        H = Hk * rng.choice([1, 1, 2, 3])
        room = 500_000 // H
        lengths = []
        for _ in range(_spread(rng, 1, 12)):
            n = min(_spread(rng, 1, 16000) if rng.random() > 0.05 else 0, room)
            lengths.append(n)
            room -= n
        if not sum(lengths):
            lengths[0] = 7
        return dict(op=op, lengths=",".join(map(str, lengths)), H=H, Hk=Hk, decay=rng.choice(["gate", "strong"]),
                    beta=rng.choice(["fp32", "bf16"]), state=rng.choice(["none", "fp32", "bf16"]))
    if op == "decode":
        Hk = rng.choice([1, 2, 3, 4, 8, 16, 32])
        H = Hk * rng.choice([1, 1, 2, 4]) if Hk < 16 else Hk
        return dict(op=op, N=_spread(rng, 1, 8192 // H if H > 31 else 256), T=rng.choice([1, 1, 1, 2, 3, 5, 8]), H=H,
                    Hk=Hk, slots=rng.random() < 0.5)
    if op == "beam":
        B, W = _spread(rng, 1, 32), rng.choice([1, 2, 3, 4, 5, 8])
        return dict(op=op, B=B, W=W, V=_spread(rng, 1000, 131072), n=W * rng.choice([1, 2]),
                    dtype=rng.choice(["bf16", "fp16", "fp32"]), finished=rng.random() < 0.5,
                    masked=rng.random() < 0.5)
    if op == "reorder":
        return dict(op=op, B=_spread(rng, 1, 32), W=rng.choice([2, 3, 4, 5, 8]), H=rng.choice([1, 4, 8, 12, 16]))
    if op == "pages":
        P = _spread(rng, 16, 512)
        return dict(op=op, P=P, H=rng.choice([1, 4, 8, 12, 16]), F=_spread(rng, 1, P // 4))
    return dict(op=op, P=_spread(rng, 8, 512), H=rng.choice([1, 4, 8, 12, 16]))


def _lengths(case):
    return [int(x) for x in case["lengths"].split(",")]


def _moves(case):
    """How many pages a pool case copies: fixed by the case, not by the seed."""
    if case["op"] == "reorder":
        return case["B"] * (case["W"] // 2)
    if case["op"] == "pages":
        return case["F"] + 2
    live = case["P"] - case["P"] // 2
    return min(live, case["P"] // 2) // 2


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _tokens(gen, rows, H, Hk, decay, beta):
    """q, k, v, g, beta of `rows` tokens: unit q and k, a log-decay per token and head (`gate`:
    -a * softplus(x + bias), slow and fast heads; `strong`: -softplus(x)) and beta = sigmoid(x)."""
    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    def unit(x):
        return x / x.norm(dim=-1, keepdim=True).clamp_min(1e-12)

    soft = torch.nn.functional.softplus
    d = dict(q=unit(normal(*rows, Hk, D)).bfloat16(), k=unit(normal(*rows, Hk, D)).bfloat16(),
             v=normal(*rows, H, D).bfloat16())
    x = normal(*rows, H)
    if decay == "strong":
        d["g"] = -soft(x)
    else:
        a = 16 * torch.rand(H, generator=gen, device=DEV) + 0.01
        dt = torch.exp(torch.rand(H, generator=gen, device=DEV) * math.log(100.0) + math.log(1e-3))
        d["g"] = -a * soft(x + torch.log(torch.expm1(dt)))
    d["beta"] = torch.sigmoid(normal(*rows, H)).to(TYPES[beta])
    return d


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    cpu = torch.Generator().manual_seed(int(seed))
    op = case["op"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    def ints(x):
        return torch.as_tensor(x, dtype=torch.int32).to(DEV)

    if op == "prefill":
        lengths, H = _lengths(case), case["H"]
        cu = [0]
        for n in lengths:
            cu.append(cu[-1] + n)
        s = _tokens(gen, (cu[-1],), H, case["Hk"], case["decay"], case["beta"])
        s.update(cu_host=cu, cu=ints(cu), s0=None, state_dtype=None)
        if case["state"] != "none":
            s["state_dtype"] = TYPES[case["state"]]
            s["s0"] = (0.1 * normal(len(lengths), H, D, D)).to(s["state_dtype"])
    elif op == "decode":
        N, H = case["N"], case["H"]
        s = _tokens(gen, (N, case["T"]), H, case["Hk"], "gate", "fp32")
        s.update(slots=None, state=None)
        if case["slots"]:  # the sequences' places in a larger pool; the last entry of a batch is padding
            slots = torch.randperm(N + 7, generator=cpu)[:N].int()
            if N > 1:
                slots[-1] = -1
            s["slots"] = slots.to(DEV)
        s["state"] = 0.1 * normal(N + 7 if case["slots"] else N, H, D, D)
    elif op == "beam":
        B, W, V = case["B"], case["W"], case["V"]
        x = 2.0 * normal(B, W, V)
        x.scatter_(2, torch.randint(0, V, (B, W, 8), generator=gen, device=DEV), 14.0 + normal(B, W, 8))
        if case["masked"]:  # a grammar's mask
            x[:, :, 1::7] = float("-inf")
        s = dict(logits=x.to(TYPES[case["dtype"]]), n=case["n"], eos=2 if case["finished"] else None, finished=None,
                 scores=(-10 * torch.rand(B, W, generator=gen, device=DEV)).sort(-1, descending=True).values)
        if case["finished"]:
            s["finished"] = torch.rand(B, W, generator=gen, device=DEV) < 0.2
    elif op == "reorder":
        B, W = case["B"], case["W"]
        # half of the beams of each batch entry lose their state to a copy of another's
        parents = torch.empty(B, W, dtype=torch.int32)
        for b in range(B):
            perm = torch.randperm(W, generator=cpu)
            keep = perm[: W - W // 2]
            kids = torch.cat([keep, keep[torch.randint(0, len(keep), (W // 2,), generator=cpu)]])
            parents[b] = kids[torch.randperm(W, generator=cpu)].int()
        s = dict(pool=normal(B * W + 3, case["H"], D, D), parents=parents.to(DEV),
                 slots=torch.randperm(B * W + 3, generator=cpu)[: B * W].view(B, W).int().to(DEV))
    elif op == "pages":
        P, F = case["P"], case["F"]
        perm = torch.randperm(P, generator=cpu)
        used = torch.ones(P, dtype=torch.bool)
        used[perm[: F // 2 + 1]] = False
        gone, live = perm[F // 2 + 1: 2 * F], perm[2 * F:]
        src = live[torch.randint(0, len(live), (F,), generator=cpu)].int()
        swap = live[torch.randperm(len(live), generator=cpu)[:2]].int()
        s = dict(pool=normal(P, case["H"], D, D), used=used.to(DEV), gone=gone.int().to(DEV),
                 src=torch.cat([src, torch.tensor([-1], dtype=torch.int32)]).to(DEV), swap=swap.to(DEV),
                 paws=swap.flip(0).to(DEV))
    else:
        P, m = case["P"], _moves(case)
        live = P - P // 2
        # `m` of the live pages lie behind the first `live` pages, in any order
        front, back = torch.randperm(live, generator=cpu), live + torch.randperm(P - live, generator=cpu)
        used = torch.zeros(P, dtype=torch.bool)
        used[front[m:]] = True
        used[back[:m]] = True
        table = torch.cat([used.nonzero()[:, 0], torch.tensor([-1])])
        table = table[torch.randperm(len(table), generator=cpu)].int()
        s = dict(pool=normal(P, case["H"], D, D), used=used.to(DEV), table=table.to(DEV))
    s["op"] = op
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    return _library(s) if own else PLAIN[s["op"]](s)


def _library(s):
    import kda_chunked_delta_amd as kda
    op = s["op"]
    if op == "prefill":
        return kda.gated_delta_prefill(s["q"], s["k"], s["v"], s["g"], s["beta"], cu_seqlens=s["cu"],
                                       cu_seqlens_host=s["cu_host"], initial_state=s["s0"],
                                       output_final_state=s["s0"] is not None)
    if op == "decode":
        o = kda.gated_delta_decode(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], slots=s["slots"])
        return o, s["state"]
    if op == "beam":
        return kda.beam_select(s["logits"], s["scores"], n=s["n"], finished=s["finished"], eos=s["eos"])
    if op == "reorder":
        return kda.beam_reorder(s["pool"], s["slots"], s["parents"]), s["pool"]
    if op == "pages":
        used = s["used"].clone()
        kda.pool_free(used, s["gone"])
        dst = kda.pool_fork(s["pool"], used, s["src"])
        kda.pool_copy(s["pool"], s["swap"], s["paws"])
        return dst, used, s["pool"]
    used, table = s["used"].clone(), s["table"].clone()
    newpos, live = kda.pool_compact(s["pool"], used, table)
    return newpos, live, used, table, s["pool"]


def _plain_prefill(s):
    """Chunks of 64 tokens of every sequence side by side, one product with the state at a time."""
    C = 64
    q, k, v, cu, s0 = s["q"], s["k"], s["v"], s["cu"].long(), s["s0"]
    H, rep = v.shape[1], v.shape[1] // k.shape[1]
    n = cu[1:] - cu[:-1]
    N, NC = len(n), -(-max(b - a for a, b in zip(s["cu_host"], s["cu_host"][1:])) // C)
    pos = torch.arange(NC * C, device=q.device)
    row = (cu[:-1, None] + pos).clamp(max=q.shape[0] - 1)
    inside = pos < n[:, None]

    def chunks(x, group=1):  # [Tt, h, ...] -> [N, h * group, NC, C, ...] in 32 bits, zero outside
        x = torch.where(inside.view(N, -1, *[1] * (x.dim() - 1)), x[row].float(), 0.0)
        x = x.view(N, NC, C, *x.shape[2:]).movedim(3, 1)
        return x.repeat_interleave(group, dim=1) if group > 1 else x

    Q, K, V, beta = chunks(q, rep), chunks(k, rep), chunks(v), chunks(s["beta"])
    G = chunks(s["g"]).double().cumsum(-1)  # differences of long sums: 64 bits
    decay = torch.exp((G[..., :, None] - G[..., None, :]).clamp(max=0.0)).float()
    gam, last = torch.exp(G).float(), torch.exp(G[..., -1:] - G).float()
    lower = torch.ones(C, C, device=q.device).tril()
    L = beta[..., None] * torch.matmul(K, K.transpose(-1, -2)) * decay * lower.tril(-1)
    A = torch.matmul(Q, K.transpose(-1, -2)) * decay * lower
    T = torch.eye(C, device=q.device).expand_as(L).contiguous()
    for r in range(1, C):  # (I + L)^-1 by rows
        T[..., r, :r] = -torch.matmul(L[..., r:r + 1, :r], T[..., :r, :r])[..., 0, :]
    T = T * beta[..., None, :]
    W, U0 = torch.matmul(T, gam[..., None] * K), torch.matmul(T, V)
    Qg, Kl = gam[..., None] * Q, (last[..., None] * K).transpose(-1, -2).contiguous()
    S = torch.zeros(N, H, D, D, device=q.device) if s0 is None else s0.float()
    O = torch.empty(N, H, NC, C, D, device=q.device)
    for c in range(NC):  # the recurrence goes from chunk to chunk
        U = U0[:, :, c] - torch.matmul(W[:, :, c], S)
        O[:, :, c] = torch.matmul(Qg[:, :, c], S) + torch.matmul(A[:, :, c], U)
        S = gam[:, :, c, -1, None, None] * S + torch.matmul(Kl[:, :, c], U)
    # back to packed rows: token t of the batch lies in its sequence's chunks
    t = torch.arange(q.shape[0], device=q.device)
    seq = (t[:, None] >= cu[None, 1:]).sum(1)
    out = O.movedim(1, 3).reshape(N, NC * C, H, D)[seq, t - cu[seq]].to(v.dtype)
    return out, (S.to(s["state_dtype"]) if s0 is not None else None)


def _plain_decode(s):
    q, k, v, state = s["q"], s["k"], s["v"], s["state"]
    rep = v.shape[2] // k.shape[2]
    Q, K, V = q.float().repeat_interleave(rep, 2), k.float().repeat_interleave(rep, 2), v.float()
    a = torch.exp(s["g"])
    slots = torch.arange(len(q), device=q.device) if s["slots"] is None else s["slots"].long()
    live = (slots >= 0) & (slots < len(state))
    at = torch.where(live, slots, 0)
    S = state[at]
    out = []
    for t in range(q.shape[1]):
        S = S * a[:, t, :, None, None]
        e = V[:, t] - (S * K[:, t, :, :, None]).sum(-2)
        S = S + (s["beta"][:, t, :, None] * K[:, t])[..., None] * e[..., None, :]
        out.append((S * Q[:, t, :, :, None]).sum(-2))
    out = torch.where(live[:, None, None, None], torch.stack(out, 1), 0.0).to(v.dtype)
    if s["slots"] is None:
        state.copy_(S)
    else:
        keep = live.nonzero()[:, 0]
        state[at[keep]] = S[keep]
    return out, state


def _plain_beam(s):
    """In 64 bits: candidates of two beams lie close together."""
    x, n = s["logits"].double(), s["n"]
    B, W, V = x.shape
    x = x - x.amax(-1, keepdim=True)
    x = x - torch.log(torch.exp(x).sum(-1, keepdim=True)) + s["scores"].double()[..., None]
    if s["finished"] is not None:
        only = torch.full_like(x, float("-inf"))
        only[..., s["eos"]] = s["scores"].double()
        x = torch.where(s["finished"][..., None], only, x)
    x = x.view(B, W * V)
    # the n best; of equal ones those with the lowest index
    edge = x.topk(n).values[:, -1:]
    ties = x == edge
    room = n - (x > edge).sum(-1, keepdim=True)
    keep = (x > edge) | (ties & (ties.cumsum(-1, dtype=torch.int32) <= room))
    index = torch.where(keep, torch.arange(W * V, 0, -1, device=x.device, dtype=torch.int32), 0)
    index = W * V - index.topk(n).values.long()
    best, order = x.gather(1, index).sort(dim=-1, descending=True, stable=True)
    index = index.gather(1, order)
    parents, tokens = (index // V).int(), (index % V).int()
    if s["finished"] is None:
        return best.float(), parents, tokens, None
    return best.float(), parents, tokens, s["finished"].gather(1, parents.long()) | (tokens == s["eos"])


def _plain_reorder(s):
    pool, slots, parents = s["pool"], s["slots"].long(), s["parents"].long()
    B, W = slots.shape
    same = parents[:, :, None] == parents[:, None, :]
    first = ~(same & torch.ones(W, W, device=slots.device, dtype=torch.bool).tril(-1)).any(-1)  # the parent's first child
    gone = ~(parents[:, None, :] == torch.arange(W, device=slots.device)[:, None]).any(-1)       # parents without a child
    free = torch.sort((~gone).int(), dim=-1, stable=True).indices                                # those, in order, come first
    rank = ((~first).cumsum(-1) - 1).clamp(min=0)
    src = slots.gather(1, parents)
    new = torch.where(first, src, slots.gather(1, free.gather(1, rank)))
    move = (new != src).view(-1).nonzero()[:, 0]
    pool[new.view(-1)[move]] = pool[src.view(-1)[move]]
    return new.int(), pool


def _plain_pages(s):
    pool, used = s["pool"], s["used"].clone()
    used[s["gone"].long()] = False
    # fork: the lowest free pages, in the order of the requests
    src = s["src"].long()
    good = (src >= 0) & (src < len(used)) & used[src.clamp(0, len(used) - 1)]
    rank = good.cumsum(0) - 1
    free = torch.sort(used.int(), stable=True).indices
    good = good & (rank < (~used).sum())
    dst = torch.where(good, free[rank.clamp(min=0)], -1)
    move = good.nonzero()[:, 0]
    used[dst[move]] = True
    pool[dst[move]] = pool[src[move]]
    # swap two pages
    pool[s["paws"].long()] = pool[s["swap"].long()]
    return dst.int(), used, pool


def _plain_compact(s):
    pool, used, table = s["pool"], s["used"], s["table"].long()
    P = len(used)
    page = torch.arange(P, device=used.device)
    live = used.sum()
    movers = (used & (page >= live)).nonzero()[:, 0]
    holes = (~used & (page < live)).nonzero()[:, 0]
    newpos = torch.where(used, page, -1)
    newpos[movers] = holes
    pool[holes] = pool[movers]
    fine = (table >= 0) & (table < P)
    table = torch.where(fine, newpos[table.clamp(0, P - 1)], -1)
    return newpos.int(), live.int().view(1), page < live, table.int(), pool


PLAIN = dict(prefill=_plain_prefill, decode=_plain_decode, beam=_plain_beam, reorder=_plain_reorder,
             pages=_plain_pages, compact=_plain_compact)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    page = case.get("H", 0) * D * D * 4
    if op == "prefill":
        lengths, H, Hk = _lengths(case), case["H"], case["Hk"]
        t = sum(lengths)
        n = t * (2 * Hk + 2 * H) * D * 2 + t * H * (4 + (2 if case["beta"] == "bf16" else 4))
        if case["state"] != "none":
            n += 2 * len(lengths) * H * D * D * (2 if case["state"] == "bf16" else 4)
        return dict(bytes=n, flops=t * H * 6 * D * D)
    if op == "decode":
        rows, H = case["N"] * case["T"], case["H"]
        live = case["N"] - (1 if case["slots"] and case["N"] > 1 else 0)
        return dict(bytes=2 * live * page + rows * (2 * case["Hk"] + 2 * H) * D * 2 + rows * H * 8,
                    flops=rows * H * 6 * D * D)
    if op == "beam":
        size = {"bf16": 2, "fp16": 2, "fp32": 4}[case["dtype"]]
        cells = case["B"] * case["W"] * case["V"]
        return dict(bytes=cells * size + case["B"] * (case["W"] * 5 + case["n"] * 13), flops=3 * cells)
    return dict(bytes=2 * _moves(case) * page, flops=0)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "prefill":  # token by token, all sequences and heads at once
        lengths = _lengths(case)
        if max(lengths) * 200e-6 + sum(lengths) * case["H"] * 2e-6 > 20:
            return None
        H, rep = case["H"], case["H"] // case["Hk"]
        N = len(lengths)
        order = sorted(range(N), key=lambda i: -lengths[i])  # the live sequences stay in front
        S = torch.zeros(N, H, D, D, dtype=torch.float64, device=DEV)
        if s["s0"] is not None:
            S = s["s0"].double()[order]
        start = torch.tensor([s["cu_host"][i] for i in order], device=DEV)
        out = torch.empty(s["v"].shape, dtype=torch.float64, device=DEV)
        for t in range(max(lengths)):
            m = sum(n > t for n in lengths)
            at = start[:m] + t
            q, k = (s[x][at].double().repeat_interleave(rep, 1) for x in "qk")
            Sm = S[:m]
            Sm *= torch.exp(s["g"][at].double())[..., None, None]
            e = s["v"][at].double() - torch.matmul(k[..., None, :], Sm)[..., 0, :]
            Sm += (s["beta"][at].double()[..., None] * k)[..., :, None] * e[..., None, :]
            out[at] = torch.matmul(q[..., None, :], Sm)[..., 0, :]
        if s["s0"] is None:
            return out, None
        back = torch.empty_like(S)
        back[order] = S
        return out, back
    if op == "decode":  # the matrix form, one (sequence, token) at a time over the heads
        H, rep = case["H"], case["H"] // case["Hk"]
        state = s["state"].double()
        out = torch.zeros(s["v"].shape, dtype=torch.float64, device=DEV)
        eye = torch.eye(D, dtype=torch.float64, device=DEV)
        for i in range(case["N"]):
            at = i if s["slots"] is None else int(s["slots"][i])
            if not 0 <= at < len(state):
                continue
            for t in range(case["T"]):
                q, k = (s[x][i, t].double().repeat_interleave(rep, 0) for x in "qk")
                b = s["beta"][i, t].double()[:, None, None]
                step = (eye - b * k[:, :, None] * k[:, None, :]) * torch.exp(s["g"][i, t].double())[:, None, None]
                S = torch.matmul(step, state[at]) + b * k[:, :, None] * s["v"][i, t].double()[:, None, :]
                state[at] = S
                out[i, t] = torch.matmul(q[:, None, :], S)[:, 0]
        return out, state
    if op == "beam":
        total = torch.empty(case["B"], case["n"], dtype=torch.float64, device=DEV)
        for b in range(case["B"]):
            p = torch.log_softmax(s["logits"][b].double(), -1) + s["scores"][b].double()[:, None]
            if s["finished"] is not None:
                for w in s["finished"][b].nonzero()[:, 0].tolist():
                    p[w] = float("-inf")
                    p[w, s["eos"]] = s["scores"][b, w].double()
            total[b] = p.view(-1).sort(descending=True).values[: case["n"]]
        return total, None, None, None
    return None  # pages are copied: equal to the plain form's, bit for bit
