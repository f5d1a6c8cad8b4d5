"""Host-side tests (no GPU) of linear attention's plans, and of the argument checks
and size limits of linear attention and of the processing of logits. No compute
entry point is called."""
import ctypes

import pytest

import kda_chunked_delta_amd as kda

OK, INVALID, UNSUPPORTED, ALIAS = 0, 1, 2, 3
A = 1 << 40  # addresses are compared only


def err(lib):
    return lib.kda_last_error().decode()


def cumulate(lengths):
    return [sum(lengths[:i]) for i in range(len(lengths) + 1)]


# ---------------------------------------------------------------------------
# plans
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("lengths,seg", [([700], 4), ([64], 1), ([65, 0, 1, 2000], 3), ([32] * 5, 1), ([31, 33], 1)])
def test_forced_segments_cover_every_chunk_once(kda_lib, lengths, seg):
    p = kda.plan_linear_attention_host(cumulate(lengths), 3, 256, True, seg)
    info, per = p.info(), {}
    for u in p.units():
        per.setdefault(u["seq"], []).append((u["chunk0"], u["n_chunks"], u["segment"], u["n_segments"]))
    slots = pre = 0
    for i, n_tok in enumerate(lengths):
        nch = -(-n_tok // 32)
        n = -(-nch // seg) if nch > seg else 1
        segs, at = sorted(per[i]), 0
        assert len(segs) == n and [s[2] for s in segs] == list(range(n)) and all(s[3] == n for s in segs)
        for c0, nc, _, _ in segs:
            assert c0 == at and (nc <= seg or n == 1)
            at += nc
        assert at == nch
        if n > 1:
            slots += n
            pre += n - 1
    assert info["n_carry_slots"] == slots and info["n_prescan"] == pre and info["uses_cp"] == (slots > 0)
    assert info["workspace_bytes"] == (slots * 3 * (65536 + 4) + 15) // 16 * 16
    assert info["total_chunks"] == sum(-(-n // 32) for n in lengths)


def test_modes(kda_lib):
    long, wide = [0, 65536], [0, 4096, 8192]
    assert kda.plan_linear_attention_host(long, 8, 256, False).info()["uses_cp"] == 0
    auto = kda.plan_linear_attention_host(long, 8, 256, "auto").info()
    assert auto["uses_cp"] == 1 and auto["est_cp_us"] < auto["est_serial_us"]
    assert kda.plan_linear_attention_host(wide, 128, 256, "auto").info()["uses_cp"] == 0
    assert kda.plan_linear_attention_host([0, 64], 1, 256, "auto").info()["workspace_bytes"] == 0
    # few compute units: nothing to gain from segments
    assert kda.plan_linear_attention_host(long, 8, 4, "auto").info()["uses_cp"] == 0


@pytest.mark.parametrize("cu,H,n_cus,seg", [([1, 5], 1, 256, 0), ([0, 5, 3], 1, 256, 0), ([0], 1, 256, 0),
                                            ([0, 5], 0, 256, 0), ([0, 5], 1 << 18, 256, 0), ([0, 5], 1, 0, 0),
                                            ([0, 5], 1, 256, -1)])
def test_plan_refusals(kda_lib, cu, H, n_cus, seg):
    with pytest.raises(kda.KDAError):
        kda.plan_linear_attention_host(cu, H, n_cus, "auto", seg)


def test_plan_refuses_other_head_dims_and_null(kda_lib):
    cu = (ctypes.c_int32 * 2)(0, 5)
    h = ctypes.c_void_p()
    f = kda_lib.kda_plan_linear_attention_host
    assert f(256, cu, 1, 1, 64, 128, 0, 0, ctypes.byref(h)) == UNSUPPORTED and not h
    assert f(256, cu, 1, 1, 128, 128, 9, 0, ctypes.byref(h)) == INVALID
    assert f(256, None, 1, 1, 128, 128, 0, 0, ctypes.byref(h)) == INVALID
    assert f(256, cu, 1, 1, 128, 128, 0, 0, None) == INVALID
    assert kda_lib.kda_plan_linear_attention(None, cu, 1, 1, 128, 128, 0, 0, ctypes.byref(h)) == INVALID


# threads of a workgroup: 512 per (unit, head), 16 x 256 per (segmented sequence, head)
@pytest.mark.parametrize("lengths,H,seg,fits", [
    ([1] * 65535, 128, 0, True), ([1] * 65536, 128, 0, False), ([1] * 63, 1 << 17, 0, True),
    ([1] * 64, 1 << 17, 0, False), ([32 * 63], 1 << 17, 1, True), ([32 * 64], 1 << 17, 1, False),
    ([64] * 7, 1 << 17, 1, True), ([64] * 8, 1 << 17, 1, False)])
def test_plan_units(kda_lib, lengths, H, seg, fits):
    make = lambda: kda.plan_linear_attention_host(cumulate_fast(lengths), H, 256, seg > 0, seg)
    if fits:
        assert make().info()["n_units"] >= len(lengths)
    else:
        with pytest.raises(kda.KDAError, match="work units") as e:
            make()
        assert e.value.status == INVALID


def cumulate_fast(lengths):
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    return cu


def test_a_prompt_of_nearly_2_31_tokens(kda_lib):
    info = kda.plan_linear_attention_host([0, (1 << 31) - 1], 1, 256, True, 1 << 20).info()
    assert info["total_chunks"] == 1 << 26 and info["n_units"] == 64 and info["max_unit_chunks"] == 1 << 20


# ---------------------------------------------------------------------------
# prefill and decode
# ---------------------------------------------------------------------------
NAMES = ("q", "k", "v", "g", "cu", "s0", "sT", "out", "ws")
AT = {n: A + (i << 32) for i, n in enumerate(NAMES)}


def prefill(lib, plan, opts=None, scale=1.0, ws_bytes=1 << 30, **kw):
    p = {**AT, **kw}
    return lib.kda_linear_attention_prefill_validate(plan.handle if plan else None, opts and ctypes.byref(opts), p["q"],
                                                     p["k"], p["v"], p["g"], p["cu"], scale, p["s0"], p["sT"], p["out"],
                                                     p["ws"], ws_bytes)


def test_prefill_validate(kda_lib):
    plan = kda.plan_linear_attention_host([0, 2000], 4, 256, True, 4)
    need = plan.info()["workspace_bytes"]
    assert need > 0
    for kw in ({}, dict(s0=None, sT=None), dict(sT=AT["s0"]), dict(opts=kda.LinearOpts(2, 1, 1)), dict(ws_bytes=need),
               dict(g=AT["g"] + 4), dict(opts=kda.LinearOpts(0, 1, 0), out=AT["g"] + 16)):
        assert prefill(kda_lib, plan, **kw) == OK, (kw, err(kda_lib))
    for kw in (dict(scale=float("nan")), dict(scale=float("inf")), dict(ws_bytes=need - 1), dict(ws=None), dict(q=None),
               dict(g=None), dict(out=None), dict(cu=None), dict(q=AT["q"] + 8), dict(out=AT["out"] + 2),
               dict(g=AT["g"] + 2), dict(s0=AT["s0"] + 4), dict(sT=AT["sT"] + 8), dict(ws=AT["ws"] + 8),
               dict(cu=AT["cu"] + 1), dict(opts=kda.LinearOpts(3, 0, 0)), dict(opts=kda.LinearOpts(-1, 0, 0))):
        assert prefill(kda_lib, plan, **kw) == INVALID, kw
    for kw in (dict(out=AT["v"]), dict(out=AT["q"] + 16), dict(out=AT["g"] + 16), dict(sT=AT["s0"] + 16),
               dict(sT=AT["out"]), dict(ws=AT["out"]), dict(ws=AT["k"]), dict(out=AT["s0"])):
        assert prefill(kda_lib, plan, **kw) == ALIAS, kw
    assert prefill(kda_lib, None) == INVALID


def test_plans_are_not_interchangeable(kda_lib):
    lin, gd = kda.plan_linear_attention_host([0, 5], 1, 256), kda.plan_gated_delta_host([0, 5], 1, 256)
    p = [A + (i << 24) for i in range(9)]
    assert kda_lib.kda_prefill_validate(lin.handle, p[0], p[1], p[2], p[3], p[4], p[5], 1.0, p[6], p[7], p[8]) == INVALID
    assert "linear attention" in err(kda_lib)
    st = kda_lib.kda_gated_delta_prefill_validate(lin.handle, None, p[0], p[1], p[2], p[3], p[4], p[5], 1.0, p[6],
                                                  p[7], p[8], None, 0)
    assert st == INVALID
    for other in (gd, kda.plan_host([0, 5], 1, 256)):
        assert prefill(kda_lib, other) == INVALID and "kda_plan_linear_attention" in err(kda_lib)


def decode(lib, n=3, T=2, H=4, Hk=2, dk=128, dv=128, fixed=0, scale=1.0, n_slots=3, slots=None, **kw):
    p = {n_: A + (i << 32) for i, n_ in enumerate(("q", "k", "v", "g", "state", "out"))}
    p.update(kw)
    return lib.kda_linear_attention_decode_validate(n, T, H, Hk, dk, dv, p["q"], p["k"], p["v"], p["g"], fixed, scale,
                                                    p["state"], n_slots, slots, p["out"])


def test_decode_validate(kda_lib):
    at = lambda i: A + (i << 32)
    for kw in ({}, dict(fixed=1), dict(n=0, n_slots=0), dict(T=0), dict(n_slots=9, slots=at(8)),
               dict(fixed=1, out=at(3) + 16), dict(n=(1 << 23) - 1, H=1, Hk=1, T=1, n_slots=9, slots=at(60),
                                                   **{n: at(100 * i) for i, n in enumerate(("q", "k", "v", "g", "state",
                                                                                            "out"))})):
        assert decode(kda_lib, **kw) == OK, (kw, err(kda_lib))
    for kw in (dict(n=-1), dict(T=-1), dict(H=0), dict(Hk=3), dict(Hk=0), dict(n_slots=-1), dict(n_slots=9),
               dict(scale=float("nan")), dict(q=None), dict(g=None), dict(out=None), dict(state=None),
               dict(k=at(1) + 8), dict(g=at(3) + 2), dict(state=at(4) + 4), dict(n_slots=9, slots=at(8) + 2),
               dict(n=1 << 24, H=1, Hk=1, n_slots=9, slots=at(60))):
        assert decode(kda_lib, **kw) == INVALID, kw
    assert decode(kda_lib, dk=64) == UNSUPPORTED and decode(kda_lib, dv=256) == UNSUPPORTED
    for kw in (dict(out=at(2)), dict(state=at(2)), dict(out=at(4) + 65536), dict(out=at(3) + 16),
               dict(n_slots=9, slots=at(4) + 64)):
        assert decode(kda_lib, **kw) == ALIAS, kw


# ---------------------------------------------------------------------------
# processing of logits
# ---------------------------------------------------------------------------
LISTS = ("tokens", "lengths", "prompt_lengths", "repetition", "frequency", "presence", "bias_tokens", "bias", "allowed")


def logits(lib, **kw):
    a = kda.Logits()
    a.rows, a.vocab, a.dtype, a.row_stride, a.out_stride = 6, 1000, 1, 1024, 1000
    a.logits, a.out = A, A + (1 << 32)
    for i, n in enumerate(LISTS):
        setattr(a, n, A + ((i + 2) << 32))
    a.token_stride = a.max_tokens = 50
    a.bias_stride = a.n_bias = 7
    a.allowed_stride = 32
    for n, x in kw.items():
        setattr(a, n, x)
    return lib.kda_logits_process_validate(ctypes.byref(a))


def test_logits_validate(kda_lib):
    at = lambda n: A + ((LISTS.index(n) + 2) << 32)
    none = dict.fromkeys(LISTS)
    for kw in ({}, {**none, "max_tokens": 0, "n_bias": 0}, dict(out=A, out_stride=1024), dict(rows=0, logits=None),
               dict(token_stride=0, bias_stride=0, allowed_stride=0), dict(max_tokens=0, tokens=None),
               dict(n_bias=0, bias=None, bias_tokens=None), dict(logits=A + 2), dict(dtype=0), dict(dtype=2),
               dict(rows=1, out=A, out_stride=1000), dict(n_bias=8192, bias_stride=8192), dict(lengths=None),
               dict(max_tokens=(1 << 30) - 1, token_stride=1 << 30, rows=1)):
        assert logits(kda_lib, **kw) == OK, (kw, err(kda_lib))
    for kw in (dict(rows=-1), dict(vocab=0), dict(dtype=3), dict(row_stride=999), dict(out_stride=999),
               dict(max_tokens=-1), dict(max_tokens=1 << 30, token_stride=1 << 30), dict(n_bias=-1),
               dict(n_bias=8193, bias_stride=8193), dict(token_stride=49), dict(token_stride=-50), dict(bias_stride=6),
               dict(allowed_stride=31), dict(tokens=None), dict(bias=None), dict(bias_tokens=None), dict(logits=None),
               dict(out=None), dict(logits=A + 1), dict(out=A + (1 << 32) + 1), dict(dtype=0, logits=A + 2),
               dict(tokens=at("tokens") + 2), dict(allowed=at("allowed") + 1), dict(presence=at("presence") + 3),
               dict(row_stride=(1 << 40) + 1)):
        assert logits(kda_lib, **kw) == INVALID, kw
    for kw in (dict(out=A + 2048), dict(out=A, out_stride=1000), dict(out=at("tokens")), dict(out=at("allowed") + 64),
               dict(out=at("lengths") + 8), dict(out=at("bias"))):
        assert logits(kda_lib, **kw) == ALIAS, kw
    assert kda_lib.kda_logits_process_validate(None) == INVALID


@pytest.mark.parametrize("rows,vocab,fits", [((1 << 23) - 1, 4096, True), (1 << 23, 4096, False),
                                             ((1 << 23) - 1, 4097, False), (1 << 22, 4097, False),
                                             ((1 << 22) - 1, 8192, True), (1, (1 << 31) - 1, True)])
def test_logits_launches(kda_lib, rows, vocab, fits):
    far = {n: (1 << 52) + (i << 46) for i, n in enumerate(LISTS)}
    st = logits(kda_lib, rows=rows, vocab=vocab, row_stride=vocab, out_stride=vocab, out=1 << 48,
                allowed_stride=1 << 27, **far)
    assert (st == OK) == fits, err(kda_lib)


def test_null_context(kda_lib):
    assert kda_lib.kda_logits_process(None, ctypes.byref(kda.Logits()), None) == INVALID
    plan = kda.plan_linear_attention_host([0, 5], 1, 256)
    a = [A + (i << 32) for i in range(9)]
    f = kda_lib.kda_linear_attention_prefill
    assert f(None, plan.handle, None, a[0], a[1], a[2], a[3], a[4], 1.0, a[5], a[6], a[7], None, 0, None) == INVALID
    assert kda_lib.kda_linear_attention_decode(None, 1, 1, 1, 1, 128, 128, a[0], a[1], a[2], a[3], 0, 1.0, a[4], 1, None,
                                               a[5], None) == INVALID
