"""What linear attention with a decay per head (chunked prefill, recurrent decode) and the processing of
logits in front of a selection (penalties, biases, masks) cost. `run` computes them in plain torch, or
with `own` through the library."""
import math

import torch

own = False  # True: run() calls the library's operators

DEV = "cuda"
D = 128      # key and value channels of a state
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
NEG = float("-inf")


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # a short prompt with one head: the smallest prefill, where latency counts
        dict(name="linear_t64_h1", op="prefill", lengths="64", H=1, Hk=1, decay="token", state="none"),
        # a ragged batch with an empty and a one-token sequence, grouped value heads, bf16 states
        dict(name="linear_ragged_gva", op="prefill", lengths="0,1,33,700,129,64,1001,257", H=12, Hk=4, decay="token",
             state="bf16"),
        # the benchmark's packed batch: eight prompts of 512 to 4096 tokens, 32 heads, fp32 states continued
        dict(name="linear_varlen8_h32", op="prefill", lengths="3779,1392,3289,3438,1776,2802,3054,617", H=32, Hk=32,
             decay="token", state="fp32"),
        # the benchmark's long prompt with few heads, one fixed decay per head
        dict(name="linear_long65536_h8", op="prefill", lengths="65536", H=8, Hk=8, decay="head", state="fp32"),
        # many equal prompts with many heads: throughput
        dict(name="linear_batch16x2048_h64", op="prefill", lengths=",".join(["2048"] * 16), H=64, Hk=64, decay="head",
             state="none"),
        # one sequence's next token
        dict(name="linear_decode_n1_h32", op="decode", N=1, T=1, H=32, Hk=32, decay="head", slots=False),
        # the benchmark's decode batch
        dict(name="linear_decode_n256_h32", op="decode", N=256, T=1, H=32, Hk=32, decay="token", slots=False),
        # four drafted tokens per sequence over a pool of states, grouped value heads, one padded entry
        dict(name="linear_decode_n33_t4_gva", op="decode", N=33, T=4, H=12, Hk=4, decay="token", slots=True),
        # the beams of one prompt after a hundred tokens, fp32 logits
        dict(name="logits_w4_v32000", op="logits", R=4, V=32000, L=100, K=0, dtype="fp32", repetition=True,
             frequency=False, mask=False, inplace=False),
        # a batch of beams with everything: long histories, requests' biases, a grammar's mask
        dict(name="logits_r256_v131072", op="logits", R=256, V=131072, L=4096, K=64, dtype="bf16", repetition=True,
             frequency=True, mask=True, inplace=False),
        # penalties alone, in place: few of the logits change
        dict(name="logits_inplace_r64_v131072", op="logits", R=64, V=131072, L=8192, K=0, dtype="fp32",
             repetition=False, frequency=True, mask=False, inplace=True),
        # a grammar's mask and biases alone, rows of an odd vocabulary in a padded buffer
        dict(name="logits_mask_r129_v100003", op="logits", R=129, V=100003, L=0, K=9, dtype="fp16", repetition=False,
             frequency=False, mask=True, inplace=False),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "decode", "logits"])
    if op == "prefill":
        Hk = rng.choice([1, 2, 4, 8, 12, 16, 32])
        H = Hk * rng.choice([1, 1, 2, 3])
        room = 1_000_000 // H
        lengths = []
        for _ in range(_spread(rng, 1, 12)):
            n = min(_spread(rng, 1, 40000) if rng.random() > 0.05 else 0, room)
            lengths.append(n)
            room -= n
        if not sum(lengths):
            lengths[0] = 7
        return dict(op=op, lengths=",".join(map(str, lengths)), H=H, Hk=Hk, decay=rng.choice(["token", "strong", "head"]),
                    state=rng.choice(["none", "fp32", "bf16"]))
    if op == "decode":
        Hk = rng.choice([1, 2, 3, 4, 8, 16, 32])
        H = Hk * rng.choice([1, 1, 2, 4]) if Hk < 16 else Hk
        return dict(op=op, N=_spread(rng, 1, 8192 // H if H > 31 else 256), T=rng.choice([1, 1, 1, 2, 3, 5, 8]), H=H,
                    Hk=Hk, decay=rng.choice(["token", "head"]), slots=rng.random() < 0.5)
    inplace = rng.random() < 0.3
    L = _spread(rng, 1, 8192) if inplace or rng.random() < 0.8 else 0
    K = _spread(rng, 1, 128) if not inplace and (not L or rng.random() < 0.5) else 0
    frequency = bool(L) and (inplace or rng.random() < 0.6)
    return dict(op=op, R=_spread(rng, 1, 256), V=_spread(rng, 1000, 131072), L=L, K=K,
                dtype=rng.choice(["bf16", "fp16", "fp32"]), repetition=bool(L) and not inplace and
                (not frequency or rng.random() < 0.5), frequency=frequency, mask=rng.random() < 0.5, inplace=inplace)


def _lengths(case):
    return [int(x) for x in case["lengths"].split(",")]


def _histories(case):
    """The rows' (tokens, distinct tokens, prompt tokens): fixed by the case, not by the seed."""
    rows, V, L = [], case["V"], case["L"]
    for r in range(case["R"]):
        n = L - r * 7919 % (L // 2 + 1)
        rows.append((n, min((n + 1) // 2, V // 2), n // 3))
    return rows


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _tokens(gen, rows, H, Hk, decay):
    """q, k, v, g of `rows` tokens: a log-decay per token and head (`token`: -a * softplus(x + bias), slow
    and fast heads; `strong`: -softplus(x)) or one per head (`head`: geometric slopes, the last head without)."""
    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEV, dtype=torch.bfloat16)

    soft = torch.nn.functional.softplus
    d = dict(q=normal(*rows, Hk, D), k=normal(*rows, Hk, D), v=normal(*rows, H, D), scale=D ** -0.5)
    if decay == "head":
        d["g"] = -torch.exp2(-8.0 * torch.arange(1, H + 1, device=DEV) / H)
        d["g"][H - 1] = 0.0
        return d
    x = torch.randn(*rows, H, generator=gen, device=DEV)
    if decay == "strong":
        d["g"] = -soft(x)
    else:
        a = 16 * torch.rand(H, generator=gen, device=DEV) + 0.01
        dt = torch.exp(torch.rand(H, generator=gen, device=DEV) * math.log(100.0) + math.log(1e-3))
        d["g"] = -a * soft(x + torch.log(torch.expm1(dt)))
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
        s = _tokens(gen, (cu[-1],), H, case["Hk"], case["decay"])
        s.update(cu_host=cu, cu=ints(cu), s0=None, state_dtype=None)
        if case["state"] != "none":
            s["state_dtype"] = TYPES[case["state"]]
            s["s0"] = normal(len(lengths), H, D, D).to(s["state_dtype"])
    elif op == "decode":
        N, H = case["N"], case["H"]
        s = _tokens(gen, (N, case["T"]), H, case["Hk"], case["decay"])
        s.update(slots=None, state=None)
        if case["slots"]:  # the sequences' places in a larger pool; the last entry of a batch is padding
            slots = torch.randperm(N + 7, generator=cpu)[:N].int()
            if N > 1:
                slots[-1] = -1
            s["slots"] = slots.to(DEV)
        s["state"] = normal(N + 7 if case["slots"] else N, H, D, D)
    else:
        R, V, L, K = case["R"], case["V"], case["L"], case["K"]
        dtype = TYPES[case["dtype"]]
        s = dict(V=V, inplace=case["inplace"], tokens=None, lengths=None, prompts=None, repetition=None, frequency=None,
                 presence=None, bias_tokens=None, bias=None, allowed=None)
        # rows of a padded buffer, as a product with a padded weight leaves them
        s["logits"] = (2.0 * normal(R, -(-V // 64) * 64)).to(dtype)[:, :V]
        if L:
            rows = _histories(case)
            length, distinct, prompt = (torch.tensor(x, device=DEV) for x in zip(*rows))
            most = max(m for _, m, _ in rows)
            base = torch.rand(R, V, generator=gen, device=DEV).topk(most).indices if most else None
            at = torch.arange(L, device=DEV)
            again = (torch.rand(R, L, generator=gen, device=DEV) ** 3 * distinct[:, None]).long()
            pick = torch.where(at < distinct[:, None], at, again).clamp(max=most - 1)  # each of them, then repeats
            s["tokens"] = torch.where(at < length[:, None], base.gather(1, pick), -1).int()
            s["lengths"], s["prompts"] = length.int(), prompt.int()
            if case["repetition"]:
                s["repetition"] = 1.0 + 0.5 * torch.rand(R, generator=gen, device=DEV)
            if case["frequency"]:
                s["frequency"] = 0.1 * torch.rand(R, generator=gen, device=DEV)
                s["presence"] = torch.rand(R, generator=gen, device=DEV)
        if K:
            s["bias_tokens"] = torch.randint(0, V, (R, K), generator=gen, device=DEV, dtype=torch.int32)
            s["bias"] = 5.0 * normal(R, K)
        if case["mask"]:  # every third row a grammar that leaves little, the others one that forbids little
            words = -(-V // 32)
            bits = torch.randint(-2**31, 2**31, (R, words, 4), generator=gen, device=DEV)
            few, many = bits[..., 0], bits[..., 1]
            for i in range(2, 4):
                few, many = few & bits[..., i], many | bits[..., i]
            few = torch.where(torch.rand(R, words, generator=gen, device=DEV) < 0.02, few, 0)
            s["allowed"] = torch.where(torch.arange(R, device=DEV)[:, None] % 3 == 0, few, many).int()
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
        return kda.linear_attention_prefill(s["q"], s["k"], s["v"], s["g"], cu_seqlens=s["cu"],
                                            cu_seqlens_host=s["cu_host"], initial_state=s["s0"],
                                            output_final_state=s["s0"] is not None, scale=s["scale"])
    if op == "decode":
        o = kda.linear_attention_decode(s["q"], s["k"], s["v"], s["g"], s["state"], scale=s["scale"], slots=s["slots"])
        return o, s["state"]
    return kda.logits_process(s["logits"], tokens=s["tokens"], lengths=s["lengths"], prompt_lengths=s["prompts"],
                              repetition=s["repetition"], frequency=s["frequency"], presence=s["presence"],
                              bias_tokens=s["bias_tokens"], bias=s["bias"], allowed=s["allowed"],
                              out=s["logits"] if s["inplace"] else None)


def _plain_prefill(s):
    """Chunks of 64 tokens of every sequence side by side; the states before the chunks are one product of the
    chunks' contributions with their decays to each other."""
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

    Q, K, V = chunks(q, rep), chunks(k, rep), chunks(v)
    G = chunks(s["g"] if s["g"].dim() == 2 else s["g"].expand(q.shape[0], H)).double().cumsum(-1)  # 64 bits: differences
    lower = torch.ones(C, C, device=q.device).tril()
    A = torch.matmul(Q, K.transpose(-1, -2).contiguous())
    A = A * torch.exp((G[..., :, None] - G[..., None, :]).clamp(max=0.0)).float() * lower
    O = torch.matmul(A, V)
    # each chunk's own contribution, and the running sum of the decay over whole chunks
    B = torch.matmul((torch.exp(G[..., -1:] - G).float()[..., None] * K).transpose(-1, -2).contiguous(), V)
    E = G[..., -1].cumsum(-1)
    first = torch.cat([torch.zeros_like(E[..., :1]), E], -1)  # the decay before chunk c, and of all
    to = first[..., :, None] - E[..., None, :]
    before = torch.arange(NC + 1, device=q.device)[:, None] > torch.arange(NC, device=q.device)
    W = torch.where(before, torch.exp(to.clamp(max=0.0)), 0.0).float()
    S = torch.matmul(W, B.view(N, H, NC, D * D)).view(N, H, NC + 1, D, D)
    if s0 is not None:
        S = S + torch.exp(first).float()[..., None, None] * s0.float()[:, :, None]
    O = O + torch.matmul(torch.exp(G).float()[..., None] * Q, S[:, :, :-1])
    # back to packed rows: token t of the batch lies in its sequence's chunks
    t = torch.arange(q.shape[0], device=q.device)
    seq = (t[:, None] >= cu[None, 1:]).sum(1)
    out = (s["scale"] * O.movedim(1, 3).reshape(N, NC * C, H, D)[seq, t - cu[seq]]).to(v.dtype)
    return out, (S[:, :, -1].to(s["state_dtype"]) if s0 is not None else None)


def _plain_decode(s):
    q, k, v, state = s["q"], s["k"], s["v"], s["state"]
    N, T, H = v.shape[:3]
    rep = H // k.shape[2]
    Q, K, V = q.float().repeat_interleave(rep, 2), k.float().repeat_interleave(rep, 2), v.float()
    G = (s["g"] if s["g"].dim() == 3 else s["g"].expand(N, T, H)).cumsum(1)
    slots = torch.arange(N, device=q.device) if s["slots"] is None else s["slots"].long()
    live = (slots >= 0) & (slots < len(state))
    at = torch.where(live, slots, 0)
    S = state[at]
    decay = torch.exp((G[:, :, None] - G[:, None, :]).clamp(max=0.0))  # [N, token, earlier token, H]
    lower = torch.ones(T, T, device=q.device).tril()[..., None]
    A = (Q[:, :, None] * K[:, None, :]).sum(-1) * decay * lower
    O = (A[..., None] * V[:, None, :]).sum(2)
    for t in range(T):  # the state as each token reads it, without what the tokens of this call add
        O[:, t] += torch.exp(G[:, t])[..., None] * (S * Q[:, t, :, :, None]).sum(-2)
    S = torch.exp(G[:, -1])[..., None, None] * S
    for t in range(T):
        S += (decay[:, -1, t, :, None] * K[:, t])[..., None] * V[:, t, :, None, :]
    out = torch.where(live[:, None, None, None], s["scale"] * O, 0.0).to(v.dtype)
    if s["slots"] is None:
        state.copy_(S)
    else:
        keep = live.nonzero()[:, 0]
        state[at[keep]] = S[keep]
    return out, state


def _plain_logits(s):
    V, logits = s["V"], s["logits"]
    x = logits.float()
    R = x.shape[0]
    if s["tokens"] is not None:
        t = s["tokens"].long()
        at = torch.arange(t.shape[1], device=x.device)
        past = (at < s["lengths"][:, None]) & (t >= 0) & (t < V)

        def count(which):  # how often each token stands in the chosen part of the history
            n = torch.zeros(R, V + 1, dtype=torch.int32, device=x.device)
            return n.scatter_add_(1, torch.where(which, t, V), which.int())[:, :V]

        if s["repetition"] is not None:
            r = s["repetition"][:, None]
            x = torch.where(count(past) > 0, torch.where(x > 0, x / r, x * r), x)
        if s["frequency"] is not None:
            n = count(past & (at >= s["prompts"][:, None]))
            x = torch.where(n > 0, x - (s["frequency"][:, None] * n + s["presence"][:, None]), x)
    if s["bias"] is not None:  # of a row's entries for one token the last counts
        t = s["bias_tokens"].long()
        last = torch.zeros(R, V, dtype=torch.int64, device=x.device)
        last.scatter_reduce_(1, t, torch.arange(1, t.shape[1] + 1, device=x.device).expand_as(t).contiguous(), "amax")
        x = torch.where(last > 0, x + s["bias"].gather(1, (last - 1).clamp(min=0)), x)
    if s["allowed"] is not None:
        v = torch.arange(V, device=x.device)
        x = torch.where((s["allowed"][:, v // 32] >> (v % 32)) & 1 == 1, x, NEG)
    return logits.copy_(x) if s["inplace"] else x.to(logits.dtype)


PLAIN = dict(prefill=_plain_prefill, decode=_plain_decode, logits=_plain_logits)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    page = case.get("H", 0) * D * D * 4
    if op == "prefill":
        lengths, H, Hk = _lengths(case), case["H"], case["Hk"]
        t = sum(lengths)
        n = t * (2 * Hk + 2 * H) * D * 2 + (H if case["decay"] == "head" else t * H) * 4
        if case["state"] != "none":
            n += 2 * len(lengths) * H * D * D * (2 if case["state"] == "bf16" else 4)
        return dict(bytes=n, flops=t * H * 4 * D * D)
    if op == "decode":
        rows, H = case["N"] * case["T"], case["H"]
        live = case["N"] - (1 if case["slots"] and case["N"] > 1 else 0)
        return dict(bytes=2 * live * page + rows * (2 * case["Hk"] + 2 * H) * D * 2 +
                    (H if case["decay"] == "head" else rows * H) * 4, flops=rows * H * 4 * D * D)
    size = {"bf16": 2, "fp16": 2, "fp32": 4}[case["dtype"]]
    R, V = case["R"], case["V"]
    rows = _histories(case) if case["L"] else []
    n = sum(4 * length for length, _, _ in rows) + R * case["K"] * 8 + R * 20
    if case["mask"]:
        n += R * -(-V // 32) * 4
    # in place, penalties touch the tokens of the history, and a mask writes what it forbids (1 in 8, 2 rows of 3)
    touched = sum(m for _, m, _ in rows)
    if not case["inplace"]:
        n += 2 * R * V * size
    else:
        n += 2 * touched * size + (sum(V if r % 3 == 0 else V // 8 for r in range(R)) * size if case["mask"] else 0)
    return dict(bytes=n, flops=2 * touched + (R * V if not case["inplace"] else 0))


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "prefill":  # every token's sum over the tokens before it, without chunks or states between
        H, rep, cu = case["H"], case["H"] // case["Hk"], s["cu_host"]
        pairs = sum(n * n for n in _lengths(case)) * H
        if pairs > 2e11:
            return None
        out = torch.empty(s["v"].shape, dtype=torch.float64, device=DEV)
        last = torch.zeros(len(cu) - 1, H, D, D, dtype=torch.float64, device=DEV)
        for i, (a, b) in enumerate(zip(cu, cu[1:])):
            if a == b:
                last[i] = s["s0"][i].double() if s["s0"] is not None else 0.0
                continue
            for h in range(H):
                q, k = s["q"][a:b, h // rep].double(), s["k"][a:b, h // rep].double()
                v = s["v"][a:b, h].double()
                g = s["g"][a:b, h].double() if s["g"].dim() == 2 else s["g"][h].double().expand(b - a)
                G = g.cumsum(0)
                kt = k.t().contiguous()
                for r in range(0, b - a, 4096):
                    e = min(r + 4096, b - a)
                    p = torch.matmul(q[r:e], kt[:, :e].contiguous())
                    p *= torch.exp(G[r:e, None] - G[None, :e]).tril(r)
                    o = torch.matmul(p, v[:e])
                    if s["s0"] is not None:
                        o += torch.matmul(q[r:e] * torch.exp(G[r:e])[:, None], s["s0"][i, h].double())
                    out[a + r:a + e, h] = s["scale"] * o
                if s["s0"] is not None:
                    last[i, h] = torch.exp(G[-1]) * s["s0"][i, h].double() + torch.matmul(
                        kt * torch.exp(G[-1] - G), v)
        return out, (last if s["s0"] is not None else None)
    if op == "decode":  # the recurrence as it is written
        N, T, H = s["v"].shape[:3]
        rep = H // case["Hk"]
        state = s["state"].double()
        out = torch.zeros(s["v"].shape, dtype=torch.float64, device=DEV)
        for i in range(N):
            at = i if s["slots"] is None else int(s["slots"][i])
            if not 0 <= at < len(state):
                continue
            for t in range(T):
                q, k = (s[x][i, t].double().repeat_interleave(rep, 0) for x in "qk")
                g = (s["g"][i, t] if s["g"].dim() == 3 else s["g"]).double()
                state[at] = torch.exp(g)[:, None, None] * state[at] + k[:, :, None] * s["v"][i, t].double()[:, None, :]
                out[i, t] = s["scale"] * torch.matmul(q[:, None, :], state[at])[:, 0]
        return out, state
    x = s["logits"].double()
    for r in range(case["R"]):  # row by row
        row = x[r]
        if case["L"]:
            n = int(s["lengths"][r])
            past = s["tokens"][r, :n].long()
            if s["repetition"] is not None:
                seen = past.unique()
                f = s["repetition"][r].double()
                row[seen] = torch.where(row[seen] > 0, row[seen] / f, row[seen] * f)
            if s["frequency"] is not None:
                seen, n = past[int(s["prompts"][r]):].unique(return_counts=True)
                row[seen] -= s["frequency"][r].double() * n + s["presence"][r].double()
        if case["K"]:
            for t, b in dict(zip(s["bias_tokens"][r].tolist(), s["bias"][r].tolist())).items():
                row[t] += b
        if s["allowed"] is not None:
            bits = (s["allowed"][r][:, None] >> torch.arange(32, device=DEV)) & 1
            row[bits.view(-1)[:case["V"]] == 0] = NEG
    return x
