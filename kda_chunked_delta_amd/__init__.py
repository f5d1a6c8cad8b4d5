"""KDA forward prefill and decode on MI355X (gfx950): Python binding of libkda.so.

Argument marshalling only: every step runs in the library's HIP kernels,
reached through the C ABI of include/kda.h. PyTorch provides device memory and
the current HIP stream. There is no fallback: if the library is not built,
every entry point raises.

    import kda_chunked_delta_amd as kda
    o, s = kda.prefill(q, k, v, g, beta, cu_seqlens=cu, initial_state=s0,
                       output_final_state=True, use_intracard_cp="auto")
    o_t = kda.decode(q_t, k_t, v_t, g_t, beta_t, s)   # one token each, s in place
    o, s = kda.gated_delta_prefill(q, k, v, g1, beta, cu_seqlens=cu, output_final_state=True)
    o_t = kda.gated_delta_decode(q_t, k_t, v_t, g1_t, beta_t, s)   # g1: one decay per head
    o, s = kda.linear_attention_prefill(q, k, v, g1, cu_seqlens=cu, output_final_state=True)
    o_t = kda.linear_attention_decode(q_t, k_t, v_t, g1_t, s)

The interface follows the FLA-compatible prefill of "feat(kda/sm90): FlashKDA
prefill port + intracard-CP prefill" (cuLA pull request #103, description:
varlen packing, initial/final state, use_intracard_cp = "auto" | True | False,
default off) and the in-place state update exercised by "fix(cake_kda):
support non-aligned recurrent prefill head counts" (FlashInfer pull request
#4351, description).
"""
from __future__ import annotations

import atexit
import collections
import ctypes
import os
import threading

__all__ = ["prefill", "decode", "plan", "plan_host", "plan_segments", "Plan", "Context", "context",
           "gated_delta_prefill", "gated_delta_decode", "plan_gated_delta", "plan_gated_delta_host",
           "linear_attention_prefill", "linear_attention_decode", "plan_linear_attention",
           "plan_linear_attention_host", "logits_process", "beam_select", "beam_reorder", "pool_copy",
           "pool_fork", "pool_free", "pool_compact", "KDAError", "lib", "LIB_PATH", "CP_OFF", "CP_ON", "CP_AUTO"]

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkda.so")
D = 128
CP_OFF, CP_ON, CP_AUTO = 0, 1, 2


class KDAError(RuntimeError):
    """A libkda call returned an error status."""

    def __init__(self, status, message):
        super().__init__("%s (status %d)" % (message, status))
        self.status = status


class PlanInfo(ctypes.Structure):
    _fields_ = [("n_seqs", ctypes.c_int32), ("H", ctypes.c_int32), ("dk", ctypes.c_int32),
                ("dv", ctypes.c_int32), ("total_tokens", ctypes.c_int64),
                ("total_chunks", ctypes.c_int32), ("uses_cp", ctypes.c_int32),
                ("n_units", ctypes.c_int32), ("n_cp_seqs", ctypes.c_int32),
                ("n_prescan", ctypes.c_int32), ("n_carry_slots", ctypes.c_int32),
                ("max_unit_chunks", ctypes.c_int32), ("n_cus", ctypes.c_int32),
                ("workspace_bytes", ctypes.c_size_t), ("est_serial_us", ctypes.c_double),
                ("est_cp_us", ctypes.c_double), ("k1_materialized", ctypes.c_int32),
                ("n_split_seqs", ctypes.c_int32), ("split_warm_chunks", ctypes.c_int32),
                ("est_split_us", ctypes.c_double), ("warm_cp", ctypes.c_int32),
                ("warm_cp_seg_chunks", ctypes.c_int32), ("n_warm_segments", ctypes.c_int32),
                ("est_warm_cp_us", ctypes.c_double), ("speculation_off", ctypes.c_int32),
                ("split_warm_work", ctypes.c_int32)]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_}


class PrefillOpts(ctypes.Structure):
    _fields_ = [("qk_heads", ctypes.c_int32), ("beta_bf16", ctypes.c_int32), ("state_bf16", ctypes.c_int32)]


class LinearOpts(ctypes.Structure):
    _fields_ = [("qk_heads", ctypes.c_int32), ("g_fixed", ctypes.c_int32), ("state_bf16", ctypes.c_int32)]


class Logits(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("vocab", ctypes.c_int32), ("dtype", ctypes.c_int),
                ("logits", ctypes.c_void_p), ("row_stride", ctypes.c_int64), ("out", ctypes.c_void_p),
                ("out_stride", ctypes.c_int64), ("tokens", ctypes.c_void_p), ("token_stride", ctypes.c_int64),
                ("max_tokens", ctypes.c_int32), ("lengths", ctypes.c_void_p), ("prompt_lengths", ctypes.c_void_p),
                ("repetition", ctypes.c_void_p), ("frequency", ctypes.c_void_p), ("presence", ctypes.c_void_p),
                ("bias_tokens", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("bias_stride", ctypes.c_int64),
                ("n_bias", ctypes.c_int32), ("allowed", ctypes.c_void_p), ("allowed_stride", ctypes.c_int64)]


class Pool(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("layer_stride", ctypes.c_int64), ("page_bytes", ctypes.c_int64),
                ("n_layers", ctypes.c_int32), ("n_pages", ctypes.c_int32)]


class UnitInfo(ctypes.Structure):
    _fields_ = [("seq", ctypes.c_int32), ("chunk0", ctypes.c_int32), ("n_chunks", ctypes.c_int32),
                ("segment", ctypes.c_int32), ("n_segments", ctypes.c_int32),
                ("warm_chunks", ctypes.c_int32)]


_lib = None
_lib_lock = threading.Lock()


def lib():
    """The loaded libkda.so (raises if it has not been built)."""
    global _lib
    with _lib_lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise ImportError("libkda.so is not built (%s); run `python -m kda_chunked_delta_amd.build`"
                                  % LIB_PATH)
            L = ctypes.CDLL(LIB_PATH)
            P, I32, I64, F32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
            PP = ctypes.POINTER(ctypes.c_void_p)
            sig = {
                "kda_create": (ctypes.c_int, [ctypes.c_int, PP]),
                "kda_destroy": (None, [P]),
                "kda_last_error": (ctypes.c_char_p, []),
                "kda_version": (ctypes.c_char_p, []),
                "kda_plan_prefill": (ctypes.c_int, [P, P, I32, I32, I32, I32, ctypes.c_int, PP]),
                "kda_plan_prefill_host": (ctypes.c_int, [I32, P, I32, I32, I32, I32, ctypes.c_int, PP]),
                "kda_plan_prefill_segments": (ctypes.c_int, [P, P, I32, I32, I32, I32, I32, PP]),
                "kda_plan_prefill_split": (ctypes.c_int, [P, P, I32, I32, I32, I32, P, I32, PP]),
                "kda_plan_prefill_warm_cp": (ctypes.c_int, [P, P, I32, I32, I32, I32, I32, I32, PP]),
                "kda_plan_destroy": (None, [P]),
                "kda_plan_get_info": (ctypes.c_int, [P, ctypes.POINTER(PlanInfo)]),
                "kda_plan_workspace_bytes": (ctypes.c_size_t, [P]),
                "kda_plan_get_units": (ctypes.c_int, [P, ctypes.POINTER(UnitInfo), I32]),
                "kda_prefill_validate": (ctypes.c_int, [P, P, P, P, P, P, P, F32, P, P, P]),
                "kda_prefill": (ctypes.c_int, [P, P, P, P, P, P, P, P, F32, P, P, P, P]),
                "kda_debug_k1_records": (ctypes.c_int, [P, P, P, P, P, P, P, P, P, P]),
                "kda_prefill_ex": (ctypes.c_int, [P, P, ctypes.POINTER(PrefillOpts), P, P, P, P, P, P, F32, P, P,
                                                  P, P]),
                "kda_prefill_ex_validate": (ctypes.c_int, [P, ctypes.POINTER(PrefillOpts), P, P, P, P, P, P, F32,
                                                           P, P, P]),
                "kda_prefill_noalloc": (ctypes.c_int, [P, P, ctypes.POINTER(PrefillOpts), P, P, P, P, P, P, F32, P,
                                                       P, P, P]),
                "kda_noalloc_scratch_bytes": (ctypes.c_size_t, []),
                "kda_decode": (ctypes.c_int, [P, I32, I32, I32, I32, I32, P, P, P, P, P, F32, P, P, P]),
                "kda_decode_validate": (ctypes.c_int, [I32, I32, I32, I32, I32, P, P, P, P, P, F32, P, P]),
                "kda_decode_slots": (ctypes.c_int, [P, I32, I32, I32, I32, I32, P, P, P, P, P, F32, P, I32, P, P, P]),
                "kda_decode_slots_validate": (ctypes.c_int, [I32, I32, I32, I32, I32, P, P, P, P, P, F32, P, I32, P,
                                                             P]),
                "kda_plan_gated_delta": (ctypes.c_int, [P, P, I32, I32, I32, I32, ctypes.c_int, I32, PP]),
                "kda_plan_gated_delta_host": (ctypes.c_int, [I32, P, I32, I32, I32, I32, ctypes.c_int, I32, PP]),
                "kda_gated_delta_prefill": (ctypes.c_int, [P, P, ctypes.POINTER(PrefillOpts), P, P, P, P, P, P, F32,
                                                           P, P, P, P, ctypes.c_size_t, P]),
                "kda_gated_delta_prefill_validate": (ctypes.c_int, [P, ctypes.POINTER(PrefillOpts), P, P, P, P, P, P,
                                                                    F32, P, P, P, P, ctypes.c_size_t]),
                "kda_gated_delta_decode": (ctypes.c_int, [P, I32, I32, I32, I32, I32, I32, P, P, P, P, P, F32, P, I32,
                                                          P, P, P]),
                "kda_gated_delta_decode_validate": (ctypes.c_int, [I32, I32, I32, I32, I32, I32, P, P, P, P, P, F32,
                                                                   P, I32, P, P]),
                "kda_plan_linear_attention": (ctypes.c_int, [P, P, I32, I32, I32, I32, ctypes.c_int, I32, PP]),
                "kda_plan_linear_attention_host": (ctypes.c_int, [I32, P, I32, I32, I32, I32, ctypes.c_int, I32, PP]),
                "kda_linear_attention_prefill": (ctypes.c_int, [P, P, ctypes.POINTER(LinearOpts), P, P, P, P, P, F32, P,
                                                                P, P, P, ctypes.c_size_t, P]),
                "kda_linear_attention_prefill_validate": (ctypes.c_int, [P, ctypes.POINTER(LinearOpts), P, P, P, P, P,
                                                                         F32, P, P, P, P, ctypes.c_size_t]),
                "kda_linear_attention_decode": (ctypes.c_int, [P, I32, I32, I32, I32, I32, I32, P, P, P, P, I32, F32, P,
                                                               I32, P, P, P]),
                "kda_linear_attention_decode_validate": (ctypes.c_int, [I32, I32, I32, I32, I32, I32, P, P, P, P, I32,
                                                                        F32, P, I32, P, P]),
                "kda_logits_process": (ctypes.c_int, [P, ctypes.POINTER(Logits), P]),
                "kda_logits_process_validate": (ctypes.c_int, [ctypes.POINTER(Logits)]),
                "kda_pool_copy": (ctypes.c_int, [P, ctypes.POINTER(Pool), P, P, I32, P]),
                "kda_pool_copy_validate": (ctypes.c_int, [ctypes.POINTER(Pool), P, P, I32]),
                "kda_pool_fork": (ctypes.c_int, [P, ctypes.POINTER(Pool), P, P, P, I32, P]),
                "kda_pool_fork_validate": (ctypes.c_int, [ctypes.POINTER(Pool), P, P, P, I32]),
                "kda_pool_free": (ctypes.c_int, [P, I32, P, P, I32, P]),
                "kda_pool_free_validate": (ctypes.c_int, [I32, P, P, I32]),
                "kda_pool_compact": (ctypes.c_int, [P, ctypes.POINTER(Pool), P, P, I32, P, P, P]),
                "kda_pool_compact_validate": (ctypes.c_int, [ctypes.POINTER(Pool), P, P, I32, P, P]),
                "kda_beam_reorder": (ctypes.c_int, [P, ctypes.POINTER(Pool), P, P, P, I32, I32, P]),
                "kda_beam_reorder_validate": (ctypes.c_int, [ctypes.POINTER(Pool), P, P, P, I32, I32]),
                "kda_beam_select_workspace_bytes": (ctypes.c_size_t, [I32, I32, I32, I32]),
                "kda_beam_select": (ctypes.c_int, [P, I32, I32, I32, I32, P, ctypes.c_int, I64, P, P, I32, P, P, P, P,
                                                   P, ctypes.c_size_t, P]),
                "kda_beam_select_validate": (ctypes.c_int, [I32, I32, I32, I32, P, ctypes.c_int, I64, P, P, I32, P, P,
                                                            P, P, P, ctypes.c_size_t]),
                "kda_set_timing": (ctypes.c_int, [P, ctypes.c_int]),
                "kda_get_timing": (I32, [P, ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(ctypes.c_double),
                                         ctypes.POINTER(I32), I32]),
            }
            for name, (res, args) in sig.items():
                fn = getattr(L, name)
                fn.restype = res
                fn.argtypes = args
            _lib = L
        return _lib


def _check(status, what):
    if status != 0:
        raise KDAError(status, "%s: %s" % (what, lib().kda_last_error().decode()))


def _cp_mode(use_intracard_cp):
    if use_intracard_cp is False or use_intracard_cp is None or use_intracard_cp == CP_OFF:
        return CP_OFF
    if use_intracard_cp is True or use_intracard_cp == CP_ON:
        return CP_ON
    if use_intracard_cp == "auto" or use_intracard_cp == CP_AUTO:
        return CP_AUTO
    raise ValueError("use_intracard_cp must be 'auto', True or False (got %r)" % (use_intracard_cp,))


def _i32(name, x):
    """x as an int that the C ABI's 32 bits hold (ctypes would cut it to them)."""
    x = int(x)
    if not -2**31 <= x < 2**31:
        raise ValueError("%s must be below 2^31 (got %d)" % (name, x))
    return x


def _cu_array(cu):
    cu = [int(x) for x in cu]
    for x in (min(cu), max(cu)) if cu else ():
        _i32("cu_seqlens", x)
    return (ctypes.c_int32 * len(cu))(*cu), len(cu) - 1


class Context:
    """A libkda context on one device (device properties cached once)."""

    def __init__(self, device_index):
        self.device = int(device_index)
        h = ctypes.c_void_p()
        _check(lib().kda_create(self.device, ctypes.byref(h)), "kda_create")
        self.handle = h

    def close(self):
        if self.handle:
            lib().kda_destroy(self.handle)
            self.handle = None

    def set_timing(self, enable=True):
        _check(lib().kda_set_timing(self.handle, int(bool(enable))), "kda_set_timing")

    def timing(self):
        """{kernel name: (total ms, launches)} of the calls since the last read
        (waits for them; clears the log)."""
        most = 64  # the library has some thirty names
        names = (ctypes.c_char_p * most)()
        ms = (ctypes.c_double * most)()
        cnt = (ctypes.c_int32 * most)()
        n = lib().kda_get_timing(self.handle, names, ms, cnt, most)
        if n < 0:
            raise KDAError(5, "kda_get_timing: " + lib().kda_last_error().decode())
        return {names[i].decode(): (ms[i], cnt[i]) for i in range(n)}


_contexts = {}
_ctx_lock = threading.Lock()


def context(device=None):
    """The shared Context of a torch device (default: the current device)."""
    import torch
    idx = torch.cuda.current_device() if device is None else torch.device(device).index
    if idx is None:
        idx = torch.cuda.current_device()
    with _ctx_lock:
        ctx = _contexts.get(idx)
        if ctx is None:
            ctx = _contexts[idx] = Context(idx)
        return ctx


_shutting_down = False


@atexit.register
def _close_contexts():
    global _shutting_down
    _plan_cache.clear()
    _shutting_down = True
    for ctx in list(_contexts.values()):
        try:
            ctx.close()
        except Exception:
            pass
    _contexts.clear()


class Plan:
    """A libkda plan (chunk table, work units, CP segments)."""

    def __init__(self, handle, cu_host, device=None):
        self.handle = handle
        self.cu_host = [int(x) for x in cu_host]
        self.device = device
        self._cu_dev = None
        self._shape = None
        self._ws_bytes = None

    def __del__(self):
        try:
            if self.handle and _lib is not None and not _shutting_down:
                _lib.kda_plan_destroy(self.handle)
        except Exception:
            pass
        self.handle = None

    def info(self):
        pi = PlanInfo()
        _check(lib().kda_plan_get_info(self.handle, ctypes.byref(pi)), "kda_plan_get_info")
        return pi.as_dict()

    def shape(self):
        """(H, total tokens, sequences) the plan was built for (cached)."""
        if self._shape is None:
            i = self.info()
            self._shape = (i["H"], i["total_tokens"], i["n_seqs"])
        return self._shape

    def workspace_bytes(self):
        """Bytes of workspace a call with this plan uses (cached)."""
        if self._ws_bytes is None:
            self._ws_bytes = lib().kda_plan_workspace_bytes(self.handle)
        return self._ws_bytes

    def units(self):
        n = self.info()["n_units"]
        arr = (UnitInfo * max(n, 1))()
        _check(lib().kda_plan_get_units(self.handle, arr, n), "kda_plan_get_units")
        return [dict(seq=u.seq, chunk0=u.chunk0, n_chunks=u.n_chunks, segment=u.segment,
                     n_segments=u.n_segments, warm_chunks=u.warm_chunks) for u in arr[:n]]

    def cu_device(self):
        import torch
        if self._cu_dev is None:
            self._cu_dev = torch.tensor(self.cu_host, dtype=torch.int32, device="cuda:%d" % self.device)
        return self._cu_dev


def plan_host(cu_seqlens, H, n_cus, use_intracard_cp=False):
    """Host-only plan for an explicit CU count (inspection; no GPU needed)."""
    arr, n = _cu_array(cu_seqlens)
    h = ctypes.c_void_p()
    _check(lib().kda_plan_prefill_host(int(n_cus), arr, n, int(H), D, D, _cp_mode(use_intracard_cp),
                                       ctypes.byref(h)), "kda_plan_prefill_host")
    return Plan(h, cu_seqlens)


def plan(cu_seqlens, H, use_intracard_cp=False, device=None):
    """Executable plan on a device (tables uploaded to it)."""
    ctx = context(device)
    arr, n = _cu_array(cu_seqlens)
    h = ctypes.c_void_p()
    _check(lib().kda_plan_prefill(ctx.handle, arr, n, int(H), D, D, _cp_mode(use_intracard_cp),
                                  ctypes.byref(h)), "kda_plan_prefill")
    return Plan(h, cu_seqlens, ctx.device)


def plan_segments(cu_seqlens, H, seg_chunks, device=None):
    """Executable CP plan with a forced segment length (in 16-token chunks)."""
    ctx = context(device)
    arr, n = _cu_array(cu_seqlens)
    h = ctypes.c_void_p()
    _check(lib().kda_plan_prefill_segments(ctx.handle, arr, n, int(H), D, D, int(seg_chunks),
                                           ctypes.byref(h)), "kda_plan_prefill_segments")
    return Plan(h, cu_seqlens, ctx.device)


def plan_split(cu_seqlens, H, split_chunk, warm_chunks, device=None):
    """Executable plan with forced warm-start splits: sequence i is split at
    chunk split_chunk[i] (0: not split)."""
    ctx = context(device)
    arr, n = _cu_array(cu_seqlens)
    if len(split_chunk) != n:
        raise ValueError("split_chunk needs one entry per sequence (%d), got %d" % (n, len(split_chunk)))
    sp = (ctypes.c_int32 * max(n, 1))(*[int(x) for x in split_chunk])
    h = ctypes.c_void_p()
    _check(lib().kda_plan_prefill_split(ctx.handle, arr, n, int(H), D, D, sp, int(warm_chunks),
                                        ctypes.byref(h)), "kda_plan_prefill_split")
    return Plan(h, cu_seqlens, ctx.device)


def plan_warm_cp(cu_seqlens, H, seg_chunks, warm_chunks, device=None):
    """Executable warm-start CP plan with a forced segment length (chunks)."""
    ctx = context(device)
    arr, n = _cu_array(cu_seqlens)
    h = ctypes.c_void_p()
    _check(lib().kda_plan_prefill_warm_cp(ctx.handle, arr, n, int(H), D, D, int(seg_chunks), int(warm_chunks),
                                          ctypes.byref(h)), "kda_plan_prefill_warm_cp")
    return Plan(h, cu_seqlens, ctx.device)


_plan_cache = collections.OrderedDict()
_PLAN_CACHE_MAX = 64
# Plans used by a call captured into a graph: the graph holds their device
# tables, and may be replayed at any later time, so they are never released.
_captured_plans = []


def _cached_plan(cu_host, H, mode, device, make=plan):
    key = (device, tuple(cu_host), H, mode, make)
    p = _plan_cache.get(key)
    if p is None:
        p = make(cu_host, H, mode, device="cuda:%d" % device)
        _plan_cache[key] = p
        if len(_plan_cache) > _PLAN_CACHE_MAX:
            _plan_cache.popitem(last=False)
    else:
        _plan_cache.move_to_end(key)
    return p


def k1_records(q, k, v, g, beta, plan):
    """Run K1 alone and return its chunk records as a uint8 tensor
    [H, total_chunks, RECORD_BYTES] (layout documented in include/kda.h)."""
    import torch
    info = plan.info()
    rec = torch.empty(info["H"], info["total_chunks"], RECORD_BYTES, dtype=torch.uint8, device=q.device)
    ctx = context(q.device)
    stream = torch.cuda.current_stream(q.device).cuda_stream
    _check(lib().kda_debug_k1_records(ctx.handle, plan.handle, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                      _ptr(plan.cu_device()), _ptr(rec), ctypes.c_void_p(stream)),
           "kda_debug_k1_records")
    return rec


RECORD_BYTES = 14336


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def prefill(q, k, v, g, beta, cu_seqlens=None, initial_state=None, output_final_state=False,
            use_intracard_cp=False, scale=1.0, final_state=None, out=None, plan=None,
            cu_seqlens_host=None, state_dtype=None, no_alloc=False):
    """KDA forward prefill.

    q, k, v: bf16 [Tt, H, 128] packed, or [B, T, H, 128] (B equal-length
    sequences when cu_seqlens is None); g: fp32 log-decay, same shape;
    beta: fp32 or bf16 [Tt, H] (or [B, T, H]). q and k may have fewer heads
    Hk than v (grouped value heads, H a multiple of Hk: value head h reads
    q/k head h // (H // Hk)). cu_seqlens: int32 [N + 1] (device
    tensor, host list, or None). initial_state: [N, H, 128, 128] or None.
    final_state: a tensor to write the final state into (may be
    initial_state: in-place update); with output_final_state=True and no
    final_state, a new one is allocated. States are fp32, or all bf16
    (state_dtype, default: the dtype of the given state, else fp32).
    no_alloc=True runs kda_prefill_noalloc: the library then allocates
    nothing and uses its static per-device scratch (pass out, and
    final_state if wanted, so that this wrapper allocates nothing either).
    Returns (o, final_state or None).
    """
    import torch
    if q.dim() == 4:
        B, T = q.shape[0], q.shape[1]
        if cu_seqlens is None and cu_seqlens_host is None:
            cu_seqlens_host = [i * T for i in range(B + 1)]
        elif B != 1:
            raise ValueError("4-D inputs with cu_seqlens must have batch size 1")
        flat = lambda x: x.reshape(B * T, *x.shape[2:])
        o, s = prefill(flat(q), flat(k), flat(v), flat(g), flat(beta), cu_seqlens, initial_state,
                       output_final_state, use_intracard_cp, scale, final_state,
                       None if out is None else flat(out), plan, cu_seqlens_host, state_dtype)
        return o.view(v.shape), s
    if q.dim() != 3 or q.shape[-1] != D or v.dim() != 3:
        raise ValueError("q must be [Tt, H, 128] or [B, T, H, 128], got %s" % (tuple(q.shape),))
    Tt, Hk, H = q.shape[0], q.shape[1], v.shape[1]
    if H % Hk:
        raise ValueError("v has %d heads, not a multiple of the %d q/k heads" % (H, Hk))
    beta16 = beta.dtype == torch.bfloat16
    for name, t, dt, shape in (("q", q, torch.bfloat16, (Tt, Hk, D)), ("k", k, torch.bfloat16, (Tt, Hk, D)),
                               ("v", v, torch.bfloat16, (Tt, H, D)), ("g", g, torch.float32, (Tt, H, D)),
                               ("beta", beta, torch.bfloat16 if beta16 else torch.float32, (Tt, H))):
        if t.dtype != dt or tuple(t.shape) != shape or not t.is_contiguous() or not t.is_cuda:
            raise ValueError("%s must be a contiguous %s CUDA tensor of shape %s (got %s %s)"
                             % (name, dt, shape, t.dtype, tuple(t.shape)))
    dev = q.device.index
    if cu_seqlens_host is None:
        if cu_seqlens is None:
            cu_seqlens_host = [0, Tt]
        elif isinstance(cu_seqlens, (list, tuple)):
            cu_seqlens_host = list(cu_seqlens)
        else:
            cu_seqlens_host = cu_seqlens.tolist()  # host copy for the planner (synchronises)
    cu_seqlens_host = [int(x) for x in cu_seqlens_host]
    N = len(cu_seqlens_host) - 1
    # the library sizes every buffer from the plan, so the table must describe
    # exactly the packed tokens the tensors hold
    if (N < 1 or cu_seqlens_host[0] != 0 or cu_seqlens_host[-1] != Tt
            or any(b < a for a, b in zip(cu_seqlens_host, cu_seqlens_host[1:]))):
        raise ValueError("cu_seqlens must start at 0, never decrease and end at the %d packed tokens (got %d "
                         "entries from %s to %s)" % (Tt, N + 1, cu_seqlens_host[0] if N >= 0 else None,
                                                    cu_seqlens_host[-1] if N >= 0 else None))
    if plan is None:
        plan = _cached_plan(cu_seqlens_host, H, _cp_mode(use_intracard_cp), dev)
    else:
        if plan.device != dev:
            raise ValueError("the plan is for device %s, the tensors are on device %d" % (plan.device, dev))
        if plan.shape() != (H, Tt, N) or plan.cu_host != cu_seqlens_host:
            raise ValueError("the plan was built for H=%d, %d tokens, %d sequences (cu_seqlens %s...); the call "
                             "has H=%d, %d tokens, %d sequences" % (*plan.shape(), plan.cu_host[:4], H, Tt, N))
    if cu_seqlens is None or isinstance(cu_seqlens, (list, tuple)):
        cu_dev = plan.cu_device()
    else:
        cu_dev = cu_seqlens
        if cu_dev.dtype != torch.int32 or not cu_dev.is_cuda or cu_dev.numel() != N + 1:
            raise ValueError("cu_seqlens must be an int32 CUDA tensor of %d entries" % (N + 1))
    if state_dtype is None:
        given = initial_state if initial_state is not None else final_state
        state_dtype = given.dtype if given is not None else torch.float32
    if state_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("states must be fp32 or bf16, got %s" % (state_dtype,))
    for name, t in (("initial_state", initial_state), ("final_state", final_state)):
        if t is not None and (t.dtype != state_dtype or tuple(t.shape) != (N, H, D, D)
                              or not t.is_contiguous() or not t.is_cuda):
            raise ValueError("%s must be a contiguous %s CUDA tensor of shape %s"
                             % (name, state_dtype, (N, H, D, D)))
    if out is None:
        out = torch.empty_like(v)
    if final_state is None and output_final_state:
        final_state = torch.empty(N, H, D, D, dtype=state_dtype, device=q.device)
    ctx = context(q.device)
    stream = torch.cuda.current_stream(q.device).cuda_stream
    if torch.cuda.is_current_stream_capturing() and not any(p is plan for p in _captured_plans):
        _captured_plans.append(plan)
    opts = PrefillOpts(Hk, int(beta16), int(state_dtype == torch.bfloat16))
    entry = lib().kda_prefill_noalloc if no_alloc else lib().kda_prefill_ex
    _check(entry(ctx.handle, plan.handle, ctypes.byref(opts), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                 _ptr(cu_dev), float(scale), _ptr(initial_state), _ptr(final_state), _ptr(out),
                 ctypes.c_void_p(stream)), "kda_prefill_noalloc" if no_alloc else "kda_prefill")
    return out, final_state


def decode(q, k, v, g, beta, state, scale=1.0, out=None, slots=None):
    """KDA decode step: one new token per sequence, state advanced in place.

    q, k, v: bf16 [N, H, 128] (or [N, 1, H, 128]); g: fp32 log-decay, same
    shape as v; beta: fp32 [N, H] (or [N, 1, H]); state: fp32 [N, H, 128, 128],
    overwritten with the advanced state. q and k may have fewer heads than v
    (grouped value heads, as in prefill). With slots (int32 CUDA tensor [N]),
    state is a pool [n_slots, H, 128, 128] and sequence n uses slot slots[n];
    a slot outside the pool skips that sequence (zero output). Returns o,
    shaped like v.
    """
    import torch
    shape = v.shape
    if q.dim() == 4:
        if q.shape[1] != 1:
            raise ValueError("4-D decode inputs must have one token per sequence, got %s" % (tuple(q.shape),))
        sq = lambda x: x.reshape(x.shape[0], *x.shape[2:])
        q, k, v, g, beta = sq(q), sq(k), sq(v), sq(g), sq(beta)
        if out is not None:
            out = sq(out)
    if q.dim() != 3 or q.shape[-1] != D:
        raise ValueError("q must be [N, H, 128] or [N, 1, H, 128], got %s" % (tuple(shape),))
    N, Hk, H = q.shape[0], q.shape[1], v.shape[1]
    if H % Hk:
        raise ValueError("v has %d heads, not a multiple of the %d q/k heads" % (H, Hk))
    for name, t, dt, shp in (("q", q, torch.bfloat16, (N, Hk, D)), ("k", k, torch.bfloat16, (N, Hk, D)),
                             ("v", v, torch.bfloat16, (N, H, D)), ("g", g, torch.float32, (N, H, D)),
                             ("beta", beta, torch.float32, (N, H)),
                             ("state", state, torch.float32, (state.shape[0] if slots is not None else N, H, D, D))):
        if t.dtype != dt or tuple(t.shape) != shp or not t.is_contiguous() or not t.is_cuda:
            raise ValueError("%s must be a contiguous %s CUDA tensor of shape %s (got %s %s)"
                             % (name, dt, shp, t.dtype, tuple(t.shape)))
    if out is None:
        out = torch.empty_like(v)
    ctx = context(q.device)
    stream = torch.cuda.current_stream(q.device).cuda_stream
    if slots is not None:
        if slots.dtype != torch.int32 or tuple(slots.shape) != (N,) or not slots.is_contiguous() or not slots.is_cuda:
            raise ValueError("slots must be a contiguous int32 CUDA tensor of shape (%d,)" % N)
        _check(lib().kda_decode_slots(ctx.handle, N, H, Hk, D, D, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                      float(scale), _ptr(state), state.shape[0], _ptr(slots), _ptr(out),
                                      ctypes.c_void_p(stream)), "kda_decode_slots")
        return out.view(shape)
    _check(lib().kda_decode(ctx.handle, N, H, Hk, D, D, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                            float(scale), _ptr(state), _ptr(out), ctypes.c_void_p(stream)), "kda_decode")
    return out.view(shape)


# ---------------------------------------------------------------------------
# gated delta rule
# ---------------------------------------------------------------------------
def plan_gated_delta(cu_seqlens, H, use_intracard_cp="auto", seg_chunks=0, device=None):
    """Executable plan of a gated delta rule prefill. use_intracard_cp=True
    with seg_chunks cuts sequences into segments of at most that many chunks
    of 32 tokens (0: chosen)."""
    ctx = context(device)
    arr, n = _cu_array(cu_seqlens)
    h = ctypes.c_void_p()
    _check(lib().kda_plan_gated_delta(ctx.handle, arr, n, int(H), D, D, _cp_mode(use_intracard_cp), int(seg_chunks),
                                      ctypes.byref(h)), "kda_plan_gated_delta")
    return Plan(h, cu_seqlens, ctx.device)


def plan_gated_delta_host(cu_seqlens, H, n_cus, use_intracard_cp="auto", seg_chunks=0):
    """The same for an explicit CU count (inspection; no GPU needed)."""
    arr, n = _cu_array(cu_seqlens)
    h = ctypes.c_void_p()
    _check(lib().kda_plan_gated_delta_host(int(n_cus), arr, n, int(H), D, D, _cp_mode(use_intracard_cp),
                                           int(seg_chunks), ctypes.byref(h)), "kda_plan_gated_delta_host")
    return Plan(h, cu_seqlens)


def _need(name, t, dtype, shape, device):
    """Raise unless t is a contiguous tensor of this type and shape on CUDA device `device`."""
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != device or device < 0:
        raise ValueError("%s must be a contiguous %s tensor of shape %s on %s (got %s %s on %s, strides %s)"
                         % (name, dtype, tuple(shape), "cuda:%d" % device if device >= 0 else "a CUDA device", t.dtype,
                            tuple(t.shape), t.device, t.stride()))


def _addr(t):
    return t.data_ptr() if t is not None else None


def _on(device):
    """(library, context handle, current stream) of a CUDA device index."""
    import torch
    ctx = _contexts.get(device)
    if ctx is None:
        ctx = context("cuda:%d" % device)
    return _lib, ctx.handle, torch._C._cuda_getCurrentRawStream(device)


def _packed_plan(what, make, plan, cu_seqlens, cu_seqlens_host, Tt, H, dev, use_intracard_cp, capturing):
    """The plan of a packed call (given, cached or made), its cu_seqlens on the device, and the number of sequences."""
    import torch
    if cu_seqlens_host is None:
        if cu_seqlens is None:
            cu_seqlens_host = [0, Tt]
        elif isinstance(cu_seqlens, (list, tuple)):
            cu_seqlens_host = cu_seqlens
        elif capturing:
            raise ValueError("a graph capture needs cu_seqlens_host: device cu_seqlens cannot be read in it")
        else:
            cu_seqlens_host = cu_seqlens.tolist()  # host copy for the planner (synchronises)
    cu_seqlens_host = [int(x) for x in cu_seqlens_host]
    N = len(cu_seqlens_host) - 1
    # the library sizes every buffer from the plan, so the table must describe
    # exactly the packed tokens the tensors hold (one that has a plan never decreases)
    mode = _cp_mode(use_intracard_cp) if plan is None else None
    known = plan is not None or (dev, tuple(cu_seqlens_host), H, mode, make) in _plan_cache
    if (N < 1 or cu_seqlens_host[0] != 0 or cu_seqlens_host[-1] != Tt
            or not known and any(b < a for a, b in zip(cu_seqlens_host, cu_seqlens_host[1:]))):
        raise ValueError("cu_seqlens must start at 0, never decrease and end at the %d packed tokens (got %s)"
                         % (Tt, cu_seqlens_host[:8]))
    if plan is None:
        if capturing and not known:
            raise ValueError("a graph capture needs a plan made before it: pass plan=plan_%s(...), or call "
                             "once with these cu_seqlens" % what)
        plan = _cached_plan(cu_seqlens_host, H, mode, dev, make)
    elif plan.device != dev or plan.shape() != (H, Tt, N) or plan.cu_host != cu_seqlens_host:
        raise ValueError("the plan was built for device %s, H=%d, %d tokens, %d sequences (cu_seqlens %s...); the call "
                         "has device %s, H=%d, %d tokens, %d sequences"
                         % (plan.device, *plan.shape(), plan.cu_host[:4], dev, H, Tt, N))
    if cu_seqlens is None or isinstance(cu_seqlens, (list, tuple)):
        if capturing and plan._cu_dev is None:
            raise ValueError("a graph capture needs cu_seqlens on the device: pass them as a tensor, or call "
                             "plan.cu_device() before it")
        cu_dev = plan.cu_device()
    else:
        cu_dev = cu_seqlens
        _need("cu_seqlens", cu_dev, torch.int32, (N + 1,), dev)
    return plan, cu_dev, N


def gated_delta_prefill(q, k, v, g, beta, cu_seqlens=None, initial_state=None, output_final_state=False,
                        use_intracard_cp="auto", scale=1.0, final_state=None, out=None, plan=None,
                        cu_seqlens_host=None, state_dtype=None):
    """Gated delta rule forward prefill: one log-decay per token and head.

    q, k, v: bf16 [Tt, H, 128] packed, or [B, T, H, 128] (B equal-length
    sequences when cu_seqlens is None); g: fp32 log-decay [Tt, H] (or
    [B, T, H]); beta: fp32 or bf16, same shape. Grouped value heads,
    cu_seqlens, the states, scale, out and the returned (o, final_state or
    None) are as in prefill. use_intracard_cp: "auto" cuts long sequences with
    few heads into segments (equal within 1e-5 of a state's norm), False never
    does. Inputs have to be finite (but g may be -inf): the results of a head
    are not from the 32-token chunk of a value on that is not. plan: from plan_gated_delta; made on the first call with these
    cu_seqlens otherwise, which a graph capture cannot. The workspace of a
    segmented plan comes from torch's allocator, on the current stream.
    """
    import torch
    if q.dim() == 4:
        B, T = q.shape[0], q.shape[1]
        if cu_seqlens is None and cu_seqlens_host is None:
            cu_seqlens_host = [i * T for i in range(B + 1)]
        elif B != 1:
            raise ValueError("4-D inputs with cu_seqlens must have batch size 1")
        flat = lambda x: x.reshape(B * T, *x.shape[2:])
        if out is not None and not out.is_contiguous():
            raise ValueError("out must be contiguous")
        o, s = gated_delta_prefill(flat(q), flat(k), flat(v), flat(g), flat(beta), cu_seqlens, initial_state,
                                   output_final_state, use_intracard_cp, scale, final_state,
                                   None if out is None else flat(out), plan, cu_seqlens_host, state_dtype)
        return o.view(v.shape), s
    if q.dim() != 3 or q.shape[-1] != D or v.dim() != 3:
        raise ValueError("q must be [Tt, H, 128] or [B, T, H, 128], got %s" % (tuple(q.shape),))
    Tt, Hk, H, dev = q.shape[0], q.shape[1], v.shape[1], q.get_device()
    if Hk < 1 or H < 1 or H % Hk:
        raise ValueError("v has %d heads, not a multiple of the %d q/k heads" % (H, Hk))
    beta16 = beta.dtype == torch.bfloat16
    _need("q", q, torch.bfloat16, (Tt, Hk, D), dev)
    _need("k", k, torch.bfloat16, (Tt, Hk, D), dev)
    _need("v", v, torch.bfloat16, (Tt, H, D), dev)
    _need("g", g, torch.float32, (Tt, H), dev)
    _need("beta", beta, torch.bfloat16 if beta16 else torch.float32, (Tt, H), dev)
    capturing = torch.cuda.is_current_stream_capturing()
    plan, cu_dev, N = _packed_plan("gated_delta", plan_gated_delta, plan, cu_seqlens, cu_seqlens_host, Tt, H, dev,
                                   use_intracard_cp, capturing)
    if state_dtype is None:
        given = initial_state if initial_state is not None else final_state
        state_dtype = given.dtype if given is not None else torch.float32
    if state_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("states must be fp32 or bf16, got %s" % (state_dtype,))
    if initial_state is not None:
        _need("initial_state", initial_state, state_dtype, (N, H, D, D), dev)
    if final_state is not None:
        _need("final_state", final_state, state_dtype, (N, H, D, D), dev)
    elif output_final_state:
        final_state = torch.empty(N, H, D, D, dtype=state_dtype, device=q.device)
    if out is None:
        out = torch.empty_like(v)
    else:
        _need("out", out, torch.bfloat16, (Tt, H, D), dev)
    n_ws = plan.workspace_bytes()
    ws = torch.empty(n_ws, dtype=torch.uint8, device=q.device) if n_ws else None
    if capturing and not any(p is plan for p in _captured_plans):
        _captured_plans.append(plan)
    opts = PrefillOpts(Hk, int(beta16), int(state_dtype == torch.bfloat16))
    L, ctx, stream = _on(dev)
    _check(L.kda_gated_delta_prefill(ctx, plan.handle, ctypes.byref(opts), q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                     g.data_ptr(), beta.data_ptr(), cu_dev.data_ptr(), float(scale),
                                     _addr(initial_state), _addr(final_state), out.data_ptr(), _addr(ws), n_ws,
                                     stream),
           "kda_gated_delta_prefill")
    return out, final_state


def gated_delta_decode(q, k, v, g, beta, state, scale=1.0, out=None, slots=None):
    """Gated delta rule decode: new tokens per sequence, state advanced in place.

    q, k, v: bf16 [N, H, 128] (one token each) or [N, T, H, 128] (T tokens
    each, in order); g: fp32 log-decay [N, H] or [N, T, H]; beta: fp32, same
    shape; state: fp32 [N, H, 128, 128], overwritten. q and k may have fewer
    heads than v (grouped value heads, as in prefill). With slots (int32 CUDA
    tensor [N]), state is a pool [n_slots, H, 128, 128] and sequence n uses
    slot slots[n]; a slot outside the pool skips that sequence (zero output),
    and no two sequences may share one. Returns o, shaped like v.
    """
    import torch
    if q.dim() not in (3, 4) or v.dim() != q.dim() or q.shape[-1] != D:
        raise ValueError("q must be [N, H, 128] or [N, T, H, 128] (and v alike), got %s" % (tuple(q.shape),))
    rows, Hk, H, dev = q.shape[:-2], q.shape[-2], v.shape[-2], q.get_device()
    N = rows[0]
    if Hk < 1 or H < 1 or H % Hk:
        raise ValueError("v has %d heads, not a multiple of the %d q/k heads" % (H, Hk))
    _need("q", q, torch.bfloat16, (*rows, Hk, D), dev)
    _need("k", k, torch.bfloat16, (*rows, Hk, D), dev)
    _need("v", v, torch.bfloat16, (*rows, H, D), dev)
    _need("g", g, torch.float32, (*rows, H), dev)
    _need("beta", beta, torch.float32, (*rows, H), dev)
    n_slots = N
    if slots is not None:
        _need("slots", slots, torch.int32, (N,), dev)
        n_slots = state.shape[0]
    _need("state", state, torch.float32, (n_slots, H, D, D), dev)
    if out is None:
        out = torch.empty_like(v)
    else:
        _need("out", out, torch.bfloat16, v.shape, dev)
    L, ctx, stream = _on(dev)
    _check(L.kda_gated_delta_decode(ctx, N, rows[1] if len(rows) == 2 else 1, H, Hk, D, D, q.data_ptr(), k.data_ptr(),
                                    v.data_ptr(), g.data_ptr(), beta.data_ptr(), float(scale), state.data_ptr(),
                                    n_slots, _addr(slots), out.data_ptr(), stream), "kda_gated_delta_decode")
    return out


# ---------------------------------------------------------------------------
# linear attention
# ---------------------------------------------------------------------------
def plan_linear_attention(cu_seqlens, H, use_intracard_cp="auto", seg_chunks=0, device=None):
    """Executable plan of a linear attention prefill (arguments as in plan_gated_delta)."""
    ctx = context(device)
    arr, n = _cu_array(cu_seqlens)
    h = ctypes.c_void_p()
    _check(lib().kda_plan_linear_attention(ctx.handle, arr, n, _i32("H", H), D, D, _cp_mode(use_intracard_cp),
                                           _i32("seg_chunks", seg_chunks), ctypes.byref(h)),
           "kda_plan_linear_attention")
    return Plan(h, cu_seqlens, ctx.device)


def plan_linear_attention_host(cu_seqlens, H, n_cus, use_intracard_cp="auto", seg_chunks=0):
    """The same for an explicit CU count (inspection; no GPU needed)."""
    arr, n = _cu_array(cu_seqlens)
    h = ctypes.c_void_p()
    _check(lib().kda_plan_linear_attention_host(_i32("n_cus", n_cus), arr, n, _i32("H", H), D, D,
                                                _cp_mode(use_intracard_cp), _i32("seg_chunks", seg_chunks),
                                                ctypes.byref(h)), "kda_plan_linear_attention_host")
    return Plan(h, cu_seqlens)


def linear_attention_prefill(q, k, v, g, cu_seqlens=None, initial_state=None, output_final_state=False,
                             use_intracard_cp="auto", scale=1.0, final_state=None, out=None, plan=None,
                             cu_seqlens_host=None, state_dtype=None):
    """Linear attention forward prefill: S = exp(g) S + k v^T, o = scale S^T q.

    q, k, v: bf16 [Tt, H, 128] packed, or [B, T, H, 128] (B equal-length
    sequences when cu_seqlens is None); g: fp32 log-decay per token [Tt, H] (or
    [B, T, H]), or [H] for one decay per head. Grouped value heads, cu_seqlens,
    the states, scale, out, use_intracard_cp, plan (from plan_linear_attention),
    graph capture and the returned (o, final_state or None) are as in
    gated_delta_prefill. Inputs have to be finite (but g may be -inf).
    """
    import torch
    if q.dim() == 4:
        B, T = q.shape[0], q.shape[1]
        if cu_seqlens is None and cu_seqlens_host is None:
            cu_seqlens_host = [i * T for i in range(B + 1)]
        elif B != 1:
            raise ValueError("4-D inputs with cu_seqlens must have batch size 1")
        flat = lambda x: x.reshape(B * T, *x.shape[2:])
        if out is not None and not out.is_contiguous():
            raise ValueError("out must be contiguous")
        o, s = linear_attention_prefill(flat(q), flat(k), flat(v), g if g.dim() == 1 else flat(g), cu_seqlens,
                                        initial_state, output_final_state, use_intracard_cp, scale, final_state,
                                        None if out is None else flat(out), plan, cu_seqlens_host, state_dtype)
        return o.view(v.shape), s
    if q.dim() != 3 or q.shape[-1] != D or v.dim() != 3:
        raise ValueError("q must be [Tt, H, 128] or [B, T, H, 128], got %s" % (tuple(q.shape),))
    Tt, Hk, H, dev = q.shape[0], q.shape[1], v.shape[1], q.get_device()
    if Hk < 1 or H < 1 or H % Hk:
        raise ValueError("v has %d heads, not a multiple of the %d q/k heads" % (H, Hk))
    fixed = g.dim() == 1
    _need("q", q, torch.bfloat16, (Tt, Hk, D), dev)
    _need("k", k, torch.bfloat16, (Tt, Hk, D), dev)
    _need("v", v, torch.bfloat16, (Tt, H, D), dev)
    _need("g", g, torch.float32, (H,) if fixed else (Tt, H), dev)
    capturing = torch.cuda.is_current_stream_capturing()
    plan, cu_dev, N = _packed_plan("linear_attention", plan_linear_attention, plan, cu_seqlens, cu_seqlens_host, Tt, H,
                                   dev, use_intracard_cp, capturing)
    if state_dtype is None:
        given = initial_state if initial_state is not None else final_state
        state_dtype = given.dtype if given is not None else torch.float32
    if state_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("states must be fp32 or bf16, got %s" % (state_dtype,))
    if initial_state is not None:
        _need("initial_state", initial_state, state_dtype, (N, H, D, D), dev)
    if final_state is not None:
        _need("final_state", final_state, state_dtype, (N, H, D, D), dev)
    elif output_final_state:
        final_state = torch.empty(N, H, D, D, dtype=state_dtype, device=q.device)
    if out is None:
        out = torch.empty_like(v)
    else:
        _need("out", out, torch.bfloat16, (Tt, H, D), dev)
    n_ws = plan.workspace_bytes()
    ws = torch.empty(n_ws, dtype=torch.uint8, device=q.device) if n_ws else None
    if capturing and not any(p is plan for p in _captured_plans):
        _captured_plans.append(plan)
    opts = LinearOpts(Hk, int(fixed), int(state_dtype == torch.bfloat16))
    L, ctx, stream = _on(dev)
    _check(L.kda_linear_attention_prefill(ctx, plan.handle, ctypes.byref(opts), q.data_ptr(), k.data_ptr(),
                                          v.data_ptr(), g.data_ptr(), cu_dev.data_ptr(), float(scale),
                                          _addr(initial_state), _addr(final_state), out.data_ptr(), _addr(ws), n_ws,
                                          stream),
           "kda_linear_attention_prefill")
    return out, final_state


def linear_attention_decode(q, k, v, g, state, scale=1.0, out=None, slots=None):
    """Linear attention decode: new tokens per sequence, state advanced in place.

    q, k, v: bf16 [N, H, 128] (one token each) or [N, T, H, 128] (T tokens
    each, in order); g: fp32 log-decay [N, H] or [N, T, H], or [H] for one decay
    per head; state: fp32 [N, H, 128, 128], overwritten. Grouped value heads,
    slots and the returned o are as in gated_delta_decode.
    """
    import torch
    if q.dim() not in (3, 4) or v.dim() != q.dim() or q.shape[-1] != D:
        raise ValueError("q must be [N, H, 128] or [N, T, H, 128] (and v alike), got %s" % (tuple(q.shape),))
    rows, Hk, H, dev = q.shape[:-2], q.shape[-2], v.shape[-2], q.get_device()
    N = rows[0]
    if Hk < 1 or H < 1 or H % Hk:
        raise ValueError("v has %d heads, not a multiple of the %d q/k heads" % (H, Hk))
    fixed = g.dim() == 1
    _need("q", q, torch.bfloat16, (*rows, Hk, D), dev)
    _need("k", k, torch.bfloat16, (*rows, Hk, D), dev)
    _need("v", v, torch.bfloat16, (*rows, H, D), dev)
    _need("g", g, torch.float32, (H,) if fixed else (*rows, H), dev)
    n_slots = N
    if slots is not None:
        _need("slots", slots, torch.int32, (N,), dev)
        n_slots = state.shape[0]
    _need("state", state, torch.float32, (n_slots, H, D, D), dev)
    if out is None:
        out = torch.empty_like(v)
    else:
        _need("out", out, torch.bfloat16, v.shape, dev)
    L, ctx, stream = _on(dev)
    _check(L.kda_linear_attention_decode(ctx, N, rows[1] if len(rows) == 2 else 1, H, Hk, D, D, q.data_ptr(),
                                         k.data_ptr(), v.data_ptr(), g.data_ptr(), int(fixed), float(scale),
                                         state.data_ptr(), n_slots, _addr(slots), out.data_ptr(), stream),
           "kda_linear_attention_decode")
    return out


# ---------------------------------------------------------------------------
# pages of a state pool, and beam search over it
# ---------------------------------------------------------------------------
def _pool(pool, page_dim):
    """The library's view of a pool tensor with pages along page_dim (layers before it)."""
    if pool.dim() <= page_dim or page_dim not in (0, 1):
        raise ValueError("pool must be [pages, ...] (page_dim=0) or [layers, pages, ...] (page_dim=1), got %s"
                         % (tuple(pool.shape),))
    if pool.device.type != "cuda" or not pool.numel():
        raise ValueError("pool must be a non-empty CUDA tensor, got %s on %s" % (tuple(pool.shape), pool.device))
    page = pool[0] if page_dim == 0 else pool[0, 0]
    n_pages = pool.shape[page_dim]
    size = pool.element_size()
    n = page.numel()
    if not page.is_contiguous() or (n_pages > 1 and pool.stride(page_dim) != n):
        raise ValueError("the pages of a pool must be contiguous and back to back (strides %s)" % (pool.stride(),))
    layers = pool.shape[0] if page_dim else 1
    return Pool(pool.data_ptr(), pool.stride(0) * size if layers > 1 else 0, n * size, layers, n_pages)


def pool_copy(pool, src, dst, page_dim=0):
    """Copy page src[i] of a state pool to page dst[i], as if every source were
    read before any destination is written (swaps and rotations included).

    pool: [pages, ...], or [layers, pages, ...] with page_dim=1; any type, a
    page being a multiple of 16 bytes. src, dst: int32 CUDA tensors of up to
    1024 entries; pairs with an entry outside the pool (-1) are skipped, of
    pairs with one destination the last counts. In place, returns pool.
    """
    import torch
    view, dev = _pool(pool, page_dim), pool.get_device()
    n = src.numel()
    _need("src", src, torch.int32, (n,), dev)
    _need("dst", dst, torch.int32, (n,), dev)
    L, ctx, stream = _on(dev)
    _check(L.kda_pool_copy(ctx, ctypes.byref(view), src.data_ptr(), dst.data_ptr(), n, stream), "kda_pool_copy")
    return pool


def pool_fork(pool, used, src, page_dim=0):
    """Fork pages of a state pool: each source gets a copy in a free page.

    pool as in pool_copy; used: bool [pages], updated in place; src: int32
    CUDA tensor of up to 8192 entries (repeats allowed). The requests whose
    source is in use take the lowest free pages in order. Returns the new pages
    (int32, like src): -1 where the source is no used page or none was free.
    """
    import torch
    view, dev = _pool(pool, page_dim), pool.get_device()
    n = src.numel()
    _need("src", src, torch.int32, (n,), dev)
    _need("used", used, torch.bool, (view.n_pages,), dev)
    dst = torch.empty_like(src)
    L, ctx, stream = _on(dev)
    _check(L.kda_pool_fork(ctx, ctypes.byref(view), used.data_ptr(), src.data_ptr(), dst.data_ptr(), n, stream),
           "kda_pool_fork")
    return dst


def pool_free(used, pages):
    """Mark pages (int32 CUDA tensor) free in used (bool [n_pages], in place, returned).
    Entries outside the pool are skipped; free and repeated ones are harmless."""
    import torch
    n, dev = pages.numel(), used.get_device()
    _need("used", used, torch.bool, (used.numel(),), dev)
    _need("pages", pages, torch.int32, (n,), dev)
    L, ctx, stream = _on(dev)
    _check(L.kda_pool_free(ctx, used.numel(), used.data_ptr(), pages.data_ptr(), n, stream), "kda_pool_free")
    return used


def pool_compact(pool, used, table=None, page_dim=0):
    """Move the used pages of a state pool to its first pages.

    pool and used as in pool_fork, both updated in place; table: int32 CUDA
    tensor of pages (a slot table of any shape), whose entries are replaced in
    place by the new pages (-1 where they name no used page). Pages that lie in
    front already stay. Returns (new_pages, n_live): int32 [pages], each used
    page's new index or -1, and int32 [1], the number of used pages.
    """
    import torch
    view, dev = _pool(pool, page_dim), pool.get_device()
    _need("used", used, torch.bool, (view.n_pages,), dev)
    if table is not None:
        _need("table", table, torch.int32, table.shape, dev)
    new_pages = torch.empty(view.n_pages, dtype=torch.int32, device=pool.device)
    n_live = torch.empty(1, dtype=torch.int32, device=pool.device)
    L, ctx, stream = _on(dev)
    _check(L.kda_pool_compact(ctx, ctypes.byref(view), used.data_ptr(), _addr(table),
                              0 if table is None else table.numel(), new_pages.data_ptr(), n_live.data_ptr(), stream),
           "kda_pool_compact")
    return new_pages, n_live


def beam_reorder(pool, slots, parents, page_dim=0):
    """Let a beam batch's states follow their parents.

    pool as in pool_copy; slots: int32 [B, W], the (distinct) pages of the
    beams; parents: int32 [B, W], the beam of the same batch entry that each
    continues (the second result of beam_select). W <= 64. Returns the new
    slots: page new[b, w] holds what page slots[b, parents[b, w]] held. Only
    states that several beams continue are copied, into pages whose beam ends.
    """
    import torch
    view, dev = _pool(pool, page_dim), pool.get_device()
    if slots.dim() != 2:
        raise ValueError("slots must be [batch, beams], got %s" % (tuple(slots.shape),))
    _need("slots", slots, torch.int32, slots.shape, dev)
    _need("parents", parents, torch.int32, slots.shape, dev)
    new = torch.empty_like(slots)
    L, ctx, stream = _on(dev)
    _check(L.kda_beam_reorder(ctx, ctypes.byref(view), slots.data_ptr(), parents.data_ptr(), new.data_ptr(),
                              slots.shape[0], slots.shape[1], stream), "kda_beam_reorder")
    return new


def beam_select(logits, scores, n=None, finished=None, eos=None):
    """Beam search's selection: the n best of beams x vocabulary per batch entry.

    logits: [B, W, V] fp32, bf16 or fp16, rows of V contiguous elements at one
    even distance (a slice of a padded vocabulary is fine); scores: fp32
    [B, W] running log-probabilities. Candidate (w, t) has the value
    scores[w] + log_softmax(logits[w])[t]; the candidates of one beam go by
    logit, then by the lower t (by t alone where the score is -inf), equal
    values of two beams by the lower w.
    n: candidates per batch entry (default W; at most 64). finished: bool
    [B, W], needs eos: such a beam has the single candidate eos, at its own
    score. NaN counts as -inf. Returns (scores [B, n] fp32, parents [B, n]
    int32, tokens [B, n] int32, finished [B, n] bool, or None without eos).
    """
    import torch
    dev = logits.get_device()
    if logits.dim() != 3 or dev < 0:
        raise ValueError("logits must be a CUDA tensor [batch, beams, vocab], got %s on %s"
                         % (tuple(logits.shape), logits.device))
    B, W, V = logits.shape
    dtype = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}.get(logits.dtype)
    if dtype is None:
        raise ValueError("logits must be fp32, bf16 or fp16, got %s" % logits.dtype)
    per_entry, per_row, per_token = logits.stride()
    row = per_row if W > 1 else per_entry if B > 1 else V
    if (V > 1 and per_token != 1) or row < V or (B > 1 and per_entry != W * row):
        raise ValueError("the rows of logits must be contiguous and evenly spaced (strides %s)" % (logits.stride(),))
    _need("scores", scores, torch.float32, (B, W), dev)
    if finished is not None:
        if eos is None:
            raise ValueError("finished needs eos")
        _need("finished", finished, torch.bool, (B, W), dev)
    if eos is not None and not 0 <= eos < V:
        raise ValueError("eos must be a token of the vocabulary of %d, got %s" % (V, eos))
    n = W if n is None else int(n)
    if not 1 <= n <= 64:
        raise ValueError("n must be in [1, 64], got %d" % n)
    out_scores = torch.empty_like(scores) if n == W else torch.empty(B, n, dtype=torch.float32, device=logits.device)
    parents, tokens = torch.empty(2, B, n, dtype=torch.int32, device=logits.device).unbind(0)
    out_finished = None if eos is None else torch.empty(B, n, dtype=torch.bool, device=logits.device)
    L, ctx, stream = _on(dev)
    n_ws = L.kda_beam_select_workspace_bytes(B, W, V, n)
    ws = torch.empty(n_ws, dtype=torch.uint8, device=logits.device)
    _check(L.kda_beam_select(ctx, B, W, V, n, logits.data_ptr(), dtype, row, scores.data_ptr(), _addr(finished),
                             -1 if eos is None else int(eos), out_scores.data_ptr(), parents.data_ptr(),
                             tokens.data_ptr(), _addr(out_finished), ws.data_ptr(), n_ws, stream), "kda_beam_select")
    return out_scores, parents, tokens, out_finished


def _rows(name, t, dtype, lead, device):
    """(address, entries of a row, row stride) of a list per row: [*lead, n], rows at one even distance."""
    shape = t.shape
    if t.dtype != dtype or shape[:-1] != lead or t.get_device() != device:
        raise ValueError("%s must be a %s tensor [%s, n] on cuda:%d (got %s %s on %s)"
                         % (name, dtype, ", ".join(map(str, lead)), device, t.dtype, tuple(t.shape), t.device))
    n = shape[-1]
    if n >> 31:
        raise ValueError("the rows of %s must be below 2^31 (got %d)" % (name, n))
    if t.is_contiguous():
        return t.data_ptr(), n, n
    stride = t.stride()
    if lead.numel() <= 1:
        row = n
    else:
        row = stride[-2] if lead[-1] > 1 else stride[0]
    if (n > 1 and stride[-1] != 1) or (len(lead) == 2 and lead[0] > 1 and stride[0] != lead[1] * row):
        raise ValueError("the rows of %s must be contiguous and evenly spaced (strides %s)" % (name, stride))
    return t.data_ptr(), n, row


def logits_process(logits, tokens=None, lengths=None, prompt_lengths=None, repetition=None, frequency=None,
                   presence=None, bias_tokens=None, bias=None, allowed=None, out=None):
    """Penalties for repeated tokens, biases and a mask on logits, in front of a selection.

    logits: [R, V] or [B, W, V] fp32, bf16 or fp16, rows of V contiguous elements
    at one even distance. Per row, in this order and in fp32:
      repetition, fp32 [R]: x > 0 ? x / repetition : x * repetition for the
        tokens of the history;
      frequency, presence, fp32 [R]: x - (frequency m + presence) for the tokens
        that stand m > 0 times in the history past its prompt;
      bias, fp32 [R, K], of the tokens bias_tokens, int32 [R, K], K up to 8192:
        x + bias (of several for one token the last);
      allowed, int32 [R, ceil(V / 32)] or more: bit t & 31 of word t >> 5 is set
        where token t is allowed; the others become -inf.
    tokens: the histories, int32 [R, L], of which the first lengths [R] (int32;
    default L) count and the first prompt_lengths [R] (int32; default 0) are the
    prompt; entries outside the vocabulary (-1) are skipped. With [B, W, V]
    logits, [R] stands for [B, W]. Lists and masks may be expanded over all rows.
    out: a tensor like logits, or logits itself (in place: only what changes is
    touched); by default a new one, whose rows are padded to 128 bytes. Returns out.
    """
    import torch
    dev = logits.get_device()
    dtype = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}.get(logits.dtype)
    if logits.dim() not in (2, 3) or dev < 0 or dtype is None:
        raise ValueError("logits must be a CUDA tensor [rows, vocab] or [batch, beams, vocab] in fp32, bf16 or fp16, "
                         "got %s %s on %s" % (logits.dtype, tuple(logits.shape), logits.device))
    lead, V = logits.shape[:-1], logits.shape[-1]
    if V < 1:
        raise ValueError("logits have an empty vocabulary")
    a = Logits()
    a.rows, a.vocab, a.dtype = _i32("the rows of logits", lead.numel()), V, dtype
    a.logits, _, a.row_stride = _rows("logits", logits, logits.dtype, lead, dev)
    if out is None:
        step = 32 if dtype == 0 else 64  # rows of whole 128-byte lines
        a.out_stride = -(-V // step) * step
        out = torch.empty(*lead, a.out_stride, dtype=logits.dtype, device=logits.device)
        a.out = out.data_ptr()
        if a.out_stride != V:
            out = out[..., :V]
    elif out is logits:
        a.out, a.out_stride = a.logits, a.row_stride
    elif out.shape != logits.shape:
        raise ValueError("out must be like logits, %s (got %s)" % (tuple(logits.shape), tuple(out.shape)))
    else:
        a.out, _, a.out_stride = _rows("out", out, logits.dtype, lead, dev)
    if tokens is not None:
        a.tokens, a.max_tokens, a.token_stride = _rows("tokens", tokens, torch.int32, lead, dev)
        for name, t, dt in (("lengths", lengths, torch.int32), ("prompt_lengths", prompt_lengths, torch.int32),
                            ("repetition", repetition, torch.float32), ("frequency", frequency, torch.float32),
                            ("presence", presence, torch.float32)):
            if t is not None:
                _need(name, t, dt, lead, dev)
                setattr(a, name, t.data_ptr())
    elif not (lengths is prompt_lengths is repetition is frequency is presence is None):
        raise ValueError("lengths and penalties need tokens")
    if (bias is None) != (bias_tokens is None):
        raise ValueError("bias and bias_tokens go together")
    if bias is not None:
        a.bias_tokens, a.n_bias, a.bias_stride = _rows("bias_tokens", bias_tokens, torch.int32, lead, dev)
        a.bias, n, stride = _rows("bias", bias, torch.float32, lead, dev)
        if n != a.n_bias or (stride != a.bias_stride and a.rows > 1):
            raise ValueError("bias and bias_tokens must have the same shape and strides (got %s, %s)"
                             % (bias.stride(), bias_tokens.stride()))
    if allowed is not None:
        a.allowed, n, a.allowed_stride = _rows("allowed", allowed, torch.int32, lead, dev)
        if n < (V + 31) // 32:
            raise ValueError("allowed must have a bit for each of the %d tokens (got %d words)" % (V, n))
    L, ctx, stream = _on(dev)
    _check(L.kda_logits_process(ctx, ctypes.byref(a), stream), "kda_logits_process")
    return out
