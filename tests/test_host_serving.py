"""Host-side tests (no GPU) of the gated delta rule's plans and of the argument
checks of the gated delta rule, the state pool's pages and beam selection. No
compute entry point is called."""
import ctypes

import pytest

import kda_chunked_delta_amd as kda

OK, INVALID, UNSUPPORTED, ALIAS = 0, 1, 2, 3
A = 1 << 40  # addresses are compared only


def err(lib):
    return lib.kda_last_error().decode()


# ---------------------------------------------------------------------------
# plans
# ---------------------------------------------------------------------------
def segments(plan):
    per = {}
    for u in plan.units():
        per.setdefault(u["seq"], []).append((u["chunk0"], u["n_chunks"], u["segment"], u["n_segments"]))
    return {s: sorted(v) for s, v in per.items()}


@pytest.mark.parametrize("lengths,seg", [([700], 4), ([64], 1), ([65, 0, 1, 2000], 3), ([32] * 5, 1), ([31, 33], 1)])
def test_forced_segments_cover_every_chunk_once(kda_lib, lengths, seg):
    cu = [sum(lengths[:i]) for i in range(len(lengths) + 1)]
    p = kda.plan_gated_delta_host(cu, 3, 256, True, seg)
    info = p.info()
    carries = sums = 0
    for i, segs in segments(p).items():
        nch = -(-lengths[i] // 32)
        n = -(-nch // seg) if nch > seg else 1
        assert len(segs) == n and all(s[3] == n for s in segs) and [s[2] for s in segs] == list(range(n))
        at = 0
        for c0, nc, _, _ in segs:
            assert c0 == at and (nc <= seg or n == 1)
            at += nc
        assert at == nch
        if n > 1:
            carries += n
            sums += 2 * n - 3
    assert info["n_carry_slots"] == carries and info["n_prescan"] == sums
    assert info["workspace_bytes"] == (carries + sums) * 3 * 65536
    assert info["uses_cp"] == (carries > 0) and info["total_chunks"] == sum(-(-n // 32) for n in lengths)


def test_modes(kda_lib):
    long, wide = [0, 65536], [0, 4096, 8192]
    assert kda.plan_gated_delta_host(long, 8, 256, False).info()["uses_cp"] == 0
    auto = kda.plan_gated_delta_host(long, 8, 256, "auto").info()
    assert auto["uses_cp"] == 1 and auto["est_cp_us"] < auto["est_serial_us"]
    assert kda.plan_gated_delta_host(wide, 128, 256, "auto").info()["uses_cp"] == 0
    assert kda.plan_gated_delta_host([0, 64], 1, 256, "auto").info()["workspace_bytes"] == 0
    # few compute units: nothing to gain from segments
    assert kda.plan_gated_delta_host(long, 8, 4, "auto").info()["uses_cp"] == 0


@pytest.mark.parametrize("cu,H,n_cus,seg", [([1, 5], 1, 256, 0), ([0, 5, 3], 1, 256, 0), ([0], 1, 256, 0),
                                            ([0, 5], 0, 256, 0), ([0, 5], 1 << 18, 256, 0), ([0, 5], 1, 0, 0),
                                            ([0, 5], 1, 256, -1)])
def test_plan_refusals(kda_lib, cu, H, n_cus, seg):
    with pytest.raises(kda.KDAError):
        kda.plan_gated_delta_host(cu, H, n_cus, "auto", seg)


def test_plan_refuses_other_head_dims_and_null(kda_lib):
    cu = (ctypes.c_int32 * 2)(0, 5)
    h = ctypes.c_void_p()
    f = kda_lib.kda_plan_gated_delta_host
    assert f(256, cu, 1, 1, 64, 128, 0, 0, ctypes.byref(h)) == UNSUPPORTED and not h
    assert f(256, cu, 1, 1, 128, 128, 9, 0, ctypes.byref(h)) == INVALID
    assert f(256, None, 1, 1, 128, 128, 0, 0, ctypes.byref(h)) == INVALID
    assert f(256, cu, 1, 1, 128, 128, 0, 0, None) == INVALID
    assert kda_lib.kda_plan_gated_delta(None, cu, 1, 1, 128, 128, 0, 0, ctypes.byref(h)) == INVALID


def test_plans_are_not_interchangeable(kda_lib):
    gd, plain = kda.plan_gated_delta_host([0, 5], 1, 256), kda.plan_host([0, 5], 1, 256)
    p = [A + (i << 24) for i in range(9)]
    assert kda_lib.kda_prefill_validate(gd.handle, p[0], p[1], p[2], p[3], p[4], p[5], 1.0, p[6], p[7], p[8]) == INVALID
    assert "gated delta" in err(kda_lib)
    st = kda_lib.kda_gated_delta_prefill_validate(plain.handle, None, p[0], p[1], p[2], p[3], p[4], p[5], 1.0, p[6],
                                                  p[7], p[8], None, 0)
    assert st == INVALID and "KDA plan" in err(kda_lib)


# ---------------------------------------------------------------------------
# prefill
# ---------------------------------------------------------------------------
NAMES = ("q", "k", "v", "g", "beta", "cu", "s0", "sT", "out", "ws")


def prefill(lib, plan, opts=None, scale=1.0, ws_bytes=1 << 30, **kw):
    p = {n: A + (i << 32) for i, n in enumerate(NAMES)}
    p.update(kw)
    return lib.kda_gated_delta_prefill_validate(plan.handle if plan else None, opts and ctypes.byref(opts), p["q"],
                                                p["k"], p["v"], p["g"], p["beta"], p["cu"], scale, p["s0"], p["sT"],
                                                p["out"], p["ws"], ws_bytes)


def test_prefill_validate(kda_lib):
    at = lambda n: A + (NAMES.index(n) << 32)
    plan = kda.plan_gated_delta_host([0, 2000], 4, 256, True, 4)
    need = plan.info()["workspace_bytes"]
    assert need > 0
    assert prefill(kda_lib, plan) == OK
    assert prefill(kda_lib, plan, s0=None, sT=None) == OK
    assert prefill(kda_lib, plan, sT=at("s0")) == OK  # in place
    assert prefill(kda_lib, plan, kda.PrefillOpts(2, 1, 1)) == OK
    assert prefill(kda_lib, plan, ws_bytes=need) == OK
    assert prefill(kda_lib, plan, g=at("g") + 4, beta=at("beta") + 4) == OK
    for kw in (dict(scale=float("nan")), dict(scale=float("inf")), dict(ws_bytes=need - 1), dict(ws=None), dict(q=None),
               dict(g=None), dict(out=None), dict(cu=None), dict(q=at("q") + 8), dict(out=at("out") + 2),
               dict(g=at("g") + 2), dict(beta=at("beta") + 2), dict(s0=at("s0") + 4), dict(sT=at("sT") + 8),
               dict(ws=at("ws") + 8), dict(cu=at("cu") + 1), dict(opts=kda.PrefillOpts(3, 0, 0)),
               dict(opts=kda.PrefillOpts(-1, 0, 0))):
        assert prefill(kda_lib, plan, **kw) == INVALID, kw
        assert err(kda_lib)
    assert prefill(kda_lib, None) == INVALID
    for kw in (dict(out=at("v")), dict(out=at("q") + 1024), dict(sT=at("g")), dict(sT=at("s0") + 65536),
               dict(ws=at("s0")), dict(ws=at("out")), dict(ws=at("sT") + 1024), dict(sT=at("out")),
               dict(out=at("cu"))):
        assert prefill(kda_lib, plan, **kw) == ALIAS, kw
    empty = kda.plan_gated_delta_host([0, 0], 4, 256)
    assert prefill(kda_lib, empty, q=None, k=None, v=None, g=None, beta=None, out=None, ws=None, ws_bytes=0) == OK
    p = [A] * 11
    assert kda_lib.kda_gated_delta_prefill(None, plan.handle, None, *p[:6], 1.0, *p[:4], 0, None) == INVALID


# ---------------------------------------------------------------------------
# decode
# ---------------------------------------------------------------------------
def decode(lib, n=3, t=2, H=4, Hk=2, dk=128, dv=128, scale=1.0, n_slots=7, **kw):
    names = ("q", "k", "v", "g", "beta", "state", "slots", "out")
    p = {x: A + (i << 32) for i, x in enumerate(names)}
    p.update(kw)
    return lib.kda_gated_delta_decode_validate(n, t, H, Hk, dk, dv, p["q"], p["k"], p["v"], p["g"], p["beta"], scale,
                                               p["state"], n_slots, p["slots"], p["out"])


def test_decode_validate(kda_lib):
    assert decode(kda_lib) == OK
    assert decode(kda_lib, slots=None, n_slots=3) == OK
    assert decode(kda_lib, n=0, q=None) == OK and decode(kda_lib, t=0, q=None) == OK
    for kw in (dict(n=-1), dict(t=-1), dict(H=0), dict(Hk=0), dict(Hk=3), dict(n_slots=-1), dict(slots=None),
               dict(scale=float("nan")), dict(n=1 << 30, H=1 << 10, Hk=1), dict(q=None), dict(v=A + 8), dict(g=A + 2),
               dict(beta=None), dict(state=None), dict(state=A + 4), dict(slots=A + 2), dict(out=None),
               dict(out=A + 8)):
        assert decode(kda_lib, **kw) == INVALID, kw
    assert decode(kda_lib, dk=64) == UNSUPPORTED
    for kw in (dict(out=A), dict(state=A), dict(out=A + (5 << 32) + 1024), dict(out=A + (6 << 32))):
        assert decode(kda_lib, **kw) == ALIAS, kw
    p = [A] * 5
    assert kda_lib.kda_gated_delta_decode(None, 1, 1, 1, 1, 128, 128, *p, 1.0, A, 1, None, A, None) == INVALID


# ---------------------------------------------------------------------------
# pages
# ---------------------------------------------------------------------------
def pool(base=A, stride=0, page=65536, layers=1, pages=10):
    return kda.Pool(base, stride, page, layers, pages)


BAD_POOLS = [dict(base=None), dict(base=A + 8), dict(page=0), dict(page=24), dict(page=-16), dict(layers=0),
             dict(pages=-1), dict(layers=2, stride=9 * 65536), dict(layers=2, stride=655360 + 8),
             dict(layers=2, stride=-(1 << 30))]
T, U, V = A + (1 << 33), A + (2 << 33), A + (3 << 33)


@pytest.mark.parametrize("bad", BAD_POOLS)
def test_pool_layout_refusals(kda_lib, bad):
    p = ctypes.byref(pool(**bad))
    assert kda_lib.kda_pool_copy_validate(p, T, U, 2) == INVALID
    assert kda_lib.kda_pool_fork_validate(p, V, T, U, 2) == INVALID
    assert kda_lib.kda_pool_compact_validate(p, V, T, 2, U, U + 4096) == INVALID
    assert kda_lib.kda_beam_reorder_validate(p, T, U, V, 2, 2) == INVALID


def test_pool_calls_validate(kda_lib):
    p = ctypes.byref(pool())
    two = ctypes.byref(pool(layers=2, stride=655360))
    copy, fork = kda_lib.kda_pool_copy_validate, kda_lib.kda_pool_fork_validate
    for q in (p, two):
        assert copy(q, T, U, 1024) == OK and copy(q, None, None, 0) == OK
        assert fork(q, V, T, U, 8192) == OK
    assert copy(None, T, U, 1) == INVALID and copy(p, T, U, 1025) == INVALID and copy(p, T, U, -1) == INVALID
    assert copy(p, None, U, 1) == INVALID and copy(p, T, U + 2, 1) == INVALID
    assert copy(p, A + 64, U, 1) == ALIAS and copy(two, T, A + 655360 + 64, 1) == ALIAS
    assert fork(p, V, T, U, 8193) == INVALID and fork(p, None, T, U, 1) == INVALID
    for a, b, c in ((V, V, U), (V, T, V), (V, T, T), (A, T, U)):
        assert fork(p, a, b, c, 2) == ALIAS
    free = kda_lib.kda_pool_free_validate
    assert free(10, V, T, 3) == OK and free(10, V, None, 0) == OK and free(0, None, T, 3) == OK
    assert free(-1, V, T, 3) == INVALID and free(10, V, T, -1) == INVALID and free(10, V, T + 1, 1) == INVALID
    assert free(10, None, T, 3) == INVALID and free(10, V, V, 1) == ALIAS
    compact = kda_lib.kda_pool_compact_validate
    assert compact(p, V, T, 5, U, U + 4096) == OK and compact(p, V, None, 0, U, U + 4096) == OK
    assert compact(p, V, T, -1, U, U + 4096) == INVALID and compact(p, V, T, 5, None, U) == INVALID
    assert compact(p, V, T, 5, U, None) == INVALID and compact(p, V, None, 5, U, U + 4096) == INVALID
    assert compact(p, V, T, 5, T, U) == ALIAS and compact(p, V, T, 5, U, U) == ALIAS
    assert compact(p, V, T, 5, V, U) == ALIAS and compact(p, V, A, 5, U, U + 4096) == ALIAS
    reorder = kda_lib.kda_beam_reorder_validate
    assert reorder(p, T, U, V, 3, 64) == OK and reorder(p, None, None, None, 0, 4) == OK
    assert reorder(p, T, U, V, 3, 65) == INVALID and reorder(p, T, U, V, 3, 0) == INVALID
    assert reorder(p, T, U, V, -1, 2) == INVALID and reorder(p, T, None, V, 1, 2) == INVALID
    assert reorder(p, T, U, T, 1, 2) == ALIAS and reorder(p, T, U, U, 1, 2) == ALIAS and reorder(p, A, U, V, 1, 2) == ALIAS
    for f, args in ((kda_lib.kda_pool_copy, (p, T, U, 1, None)), (kda_lib.kda_pool_fork, (p, V, T, U, 1, None)),
                    (kda_lib.kda_pool_free, (10, V, T, 1, None)),
                    (kda_lib.kda_pool_compact, (p, V, T, 1, U, U + 4096, None)),
                    (kda_lib.kda_beam_reorder, (p, T, U, V, 1, 2, None))):
        assert f(None, *args) == INVALID


# ---------------------------------------------------------------------------
# beam selection
# ---------------------------------------------------------------------------
def select(lib, B=2, W=3, V=1000, n=6, dtype=0, stride=1000, eos=2, ws_bytes=None, **kw):
    names = ("logits", "scores", "fin", "o", "p", "t", "f", "ws")
    a = {x: A + (i << 32) for i, x in enumerate(names)}
    a.update(kw)
    if ws_bytes is None:
        ws_bytes = lib.kda_beam_select_workspace_bytes(B, W, V, n)
    return lib.kda_beam_select_validate(B, W, V, n, a["logits"], dtype, stride, a["scores"], a["fin"], eos, a["o"],
                                        a["p"], a["t"], a["f"], a["ws"], ws_bytes)


def test_beam_select_validate(kda_lib):
    assert select(kda_lib) == OK
    assert select(kda_lib, fin=None) == OK
    assert select(kda_lib, fin=None, eos=-1, f=None) == OK
    assert select(kda_lib, dtype=1, logits=A + 2) == OK and select(kda_lib, stride=1003) == OK
    assert select(kda_lib, B=0, logits=None, ws=None) == OK
    assert select(kda_lib, W=1, V=5, n=5, stride=5) == OK
    for kw in (dict(B=-1), dict(W=0), dict(W=65), dict(V=0), dict(n=0), dict(n=65), dict(W=1, V=5, n=6), dict(dtype=3),
               dict(stride=999), dict(eos=1000), dict(eos=-1), dict(eos=-1, f=None), dict(f=None), dict(logits=None),
               dict(logits=A + 2), dict(dtype=1, logits=A + 1), dict(scores=None), dict(scores=A + 2), dict(o=None),
               dict(p=A + 1), dict(ws=None), dict(ws=A + 8), dict(ws_bytes=8), dict(W=64, V=1 << 26, stride=1 << 26)):
        assert select(kda_lib, **kw) == INVALID, kw
    for kw in (dict(o=A), dict(ws=A), dict(t=A + (4 << 32)), dict(f=A + (2 << 32)), dict(ws=A + (1 << 32))):
        assert select(kda_lib, **kw) == ALIAS, kw
    size = kda_lib.kda_beam_select_workspace_bytes
    assert size(0, 1, 1, 1) == 0 and size(1, 4, 32000, 4) > 0
    p = [A] * 8
    assert kda_lib.kda_beam_select(None, 1, 1, 9, 1, A, 0, 9, A, None, -1, A, A, A, None, A, 99, None) == INVALID
