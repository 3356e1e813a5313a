"""Thin ctypes binding of the QEvict C ABI (include/qevict.h).

Argument marshalling only: every step of the decode path runs in the CUDA library.  PyTorch
provides the device memory (the arena and the tensors) and the stream.  If the library is
missing this module raises; there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
# QEVICT_LIB=check loads the checked build (device bounds checks that report to the status word)
LIB_PATH = os.path.join(HERE, "libqevict_check.so" if os.environ.get("QEVICT_LIB") == "check" else "libqevict.so")

OK, EINVAL, EBUDGET, ENOMEM, ESCHEDULE, ECUDA, EDEVICE = range(7)
COUNTER_NAMES = ("promotions", "demotions", "first_quant", "reactivations", "evictions", "aged_full", "aged_quant")


class QEvictError(RuntimeError):
    word = 0   # of a status check that found bits set: those bits

    def __init__(self, status: int, where: str, msg: str):
        super().__init__(f"{where}: {msg} (status {status})")
        self.status = status


class Config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("batch", "n_layers", "h_q", "h_kv", "d_head", "n_sink", "n_recent",
                                             "window", "bits", "omega", "q_num", "q_den", "budget_num",
                                             "budget_den")] + \
               [("b_total", ctypes.c_int64), ("prompt_len", ctypes.c_int32), ("max_len", ctypes.c_int32),
                ("ranker", ctypes.c_int32), ("no_promotion", ctypes.c_int32), ("decay", ctypes.c_float),
                ("pnorm", ctypes.c_float), ("rope", ctypes.c_int32), ("reserved0", ctypes.c_int32)]


class BudgetInfo(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("full_bytes", "b_total", "b_sink", "b_local", "b_hist", "payload",
                                             "m_f", "m_q")] + \
               [(n, ctypes.c_int32) for n in ("k_f", "k_q", "n_windows", "ring_windows")]


_LAYOUT_REGIONS = ("sink", "ring", "fpool", "ledger", "score", "state", "fslot", "lslot", "ftab", "qtab", "meta")


class Layout(ctypes.Structure):
    _fields_ = [(f"{k}_{r}", ctypes.c_int64) for r in _LAYOUT_REGIONS for k in ("off", "stride")] + \
               [("qblock", ctypes.c_int64), ("arena_bytes", ctypes.c_int64), ("n_split", ctypes.c_int32),
                ("pad_", ctypes.c_int32), ("off_agg", ctypes.c_int64), ("stride_agg", ctypes.c_int64),
                ("off_rope", ctypes.c_int64)]


class Tuple(ctypes.Structure):
    """Device views of one (layer, sequence) cache tuple (qevict_tuple)."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("sink", "ring", "fpool", "ledger", "score", "state", "f_slot",
                                               "l_slot", "f_table", "q_table", "meta")]


class DiagConfig(ctypes.Structure):
    _fields_ = [("horizon", ctypes.c_int32), ("lir_m", ctypes.c_int32)]


class DiagReport(ctypes.Structure):
    _fields_ = [("events", ctypes.c_int64), ("fmm", ctypes.c_double), ("fmm_terms", ctypes.c_int64),
                ("churn", ctypes.c_double), ("churn_terms", ctypes.c_int64), ("qsa", ctypes.c_double),
                ("r_q", ctypes.c_double), ("qsa_terms", ctypes.c_int64), ("tier_mass", ctypes.c_double * 4),
                ("lir_eligible", ctypes.c_int64), ("lir_rescued", ctypes.c_int64),
                ("lir_fullkv_eligible", ctypes.c_int64), ("lir_fullkv_rescued", ctypes.c_int64),
                ("lag", ctypes.c_int64 * 32)]


class RopeConfig(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("scaling", ctypes.c_int32)] + \
               [(n, ctypes.c_double) for n in ("base", "factor", "orig_len", "low", "high")]


_Stride3 = ctypes.c_int64 * 3
_Stride2 = ctypes.c_int64 * 2
_Stride4 = ctypes.c_int64 * 4


class RopeDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("dtype", "batch", "seq", "h_q", "h_k", "d_head", "rot_dim", "interleaved",
                                             "inverse")] + \
               [("factor", ctypes.c_float), ("table_rows", ctypes.c_int64), ("pos0", ctypes.c_int64)] + \
               [(n, _Stride3) for n in ("q_in", "q_out", "k_in", "k_out")]


class AttnDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("dtype", "batch", "s_q", "s_kv", "h_q", "h_kv", "d_head", "causal")] + \
               [("scale", ctypes.c_float), ("softcap", ctypes.c_float)] + [(n, _Stride3) for n in ("q", "k", "v", "o")]


class AttnMask(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("slopes", "q_len", "kv_len", "prefix_len", "doc_ids")]


class PrefixAttnDesc(ctypes.Structure):
    _fields_ = [("attn", AttnDesc), ("s_prefix", ctypes.c_int32), ("k_prefix", _Stride2), ("v_prefix", _Stride2)]


class PagesDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("layers", "pages", "page", "h_kv", "d_head", "batch", "max_pages",
                                             "reserved0")] + [("k", _Stride4), ("v", _Stride4)]


class PagesLayout(ctypes.Structure):
    """Offsets of the bookkeeping's arrays, in int32 elements (qevict_pages_layout)."""
    _fields_ = [(n, ctypes.c_int64) for n in ("status", "n_free", "length", "held", "table", "refs", "free_bits", "ints")]


class PagesRows(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("layer", "layers", "n", "reserved0")] + [("k", _Stride4), ("v", _Stride4)]


class PagedAttnDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("dtype", "batch", "s_q", "h_q", "h_kv", "d_head")] + \
               [("scale", ctypes.c_float), ("softcap", ctypes.c_float)] + \
               [(n, ctypes.c_int32) for n in ("pages", "page", "max_pages", "reserved0")] + \
               [(n, _Stride3) for n in ("q", "o", "k", "v")]


class PagedAttnMask(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("slopes", "q_len", "parents")] + [("one_tree", ctypes.c_int32)]


_lib = None


def load() -> ctypes.CDLL:
    """Loads libqevict.so from the package directory; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with recoverable_quantized_kv_gb300.build.build()")
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    sig = {
        "qevict_budget": [ctypes.POINTER(Config), ctypes.POINTER(BudgetInfo)],
        "qevict_cache_bytes": [ctypes.POINTER(Config), ctypes.POINTER(ctypes.c_size_t)],
        "qevict_init_cache": [ctypes.POINTER(Config), P, ctypes.c_size_t, P, ctypes.POINTER(P)],
        "qevict_get_layout": [P, ctypes.POINTER(Layout)],
        "qevict_prefill_scores": [P, P, P, P, P],
        "qevict_prefill_route": [P, I32, P, P, P, P, P],
        "qevict_decode_step": [P, I32, P, P, P, P, P],
        "qevict_route": [P, P],
        "qevict_flush_scores": [P, P],
        "qevict_set_rope_table": [P, P, I64, P],
        "qevict_diag_bytes": [P, ctypes.POINTER(DiagConfig), ctypes.POINTER(ctypes.c_size_t)],
        "qevict_diag_init": [P, P, ctypes.POINTER(DiagConfig), P, ctypes.c_size_t, P, ctypes.POINTER(P)],
        "qevict_diag_route": [P, P],
        "qevict_diag_read": [P, ctypes.POINTER(DiagReport), P],
        "qevict_diag_destroy": [P],
        "qevict_get_tuple": [P, I32, I32, ctypes.POINTER(Tuple)],
        "qevict_export_bytes": [P, ctypes.POINTER(ctypes.c_size_t)],
        "qevict_export_state": [P, P, ctypes.c_size_t, P],
        "qevict_import_state": [P, P, ctypes.c_size_t, P],
        "qevict_read_counters": [P, ctypes.POINTER(I64), P],
        "qevict_check": [P, P],
        "qevict_selftest_wait": [P, P],
        "qevict_destroy": [P],
        "qevict_prefill_scores_noalloc": [I32, I32, I32, I32, I32, I32, P, P, P, P],
        "qevict_prefill_scores_noalloc_status": [P],
        "qevict_debug_cap_free_slots": [P, I32],
        "qevict_read_status": [P, ctypes.POINTER(I32), P],
        "qevict_rope_angles": [ctypes.POINTER(RopeConfig), ctypes.POINTER(ctypes.c_double)],
        "qevict_rope_table": [ctypes.POINTER(RopeConfig), I64, I64, P, P],
        "qevict_rope_apply": [ctypes.POINTER(RopeDesc), P, P, P, P, P, P, P, P],
        "qevict_attn_bytes": [ctypes.POINTER(AttnDesc), ctypes.POINTER(ctypes.c_size_t)],
        "qevict_attn": [ctypes.POINTER(AttnDesc), ctypes.POINTER(AttnMask), P, P, P, P, P, P, ctypes.c_size_t, P],
        "qevict_prefix_attn_bytes": [ctypes.POINTER(PrefixAttnDesc), ctypes.POINTER(ctypes.c_size_t)],
        "qevict_prefix_attn": [ctypes.POINTER(PrefixAttnDesc)] + [P] * 10 + [ctypes.c_size_t, P],
        "qevict_ops_status": [P, ctypes.POINTER(I32), P],
        "qevict_pages_get_layout": [ctypes.POINTER(PagesDesc), ctypes.POINTER(PagesLayout)],
        "qevict_pages_load": [ctypes.POINTER(PagesDesc), P, P, P, P],
        "qevict_pages_reserve": [ctypes.POINTER(PagesDesc), P, P, P, P, I32, P],
        "qevict_pages_append": [ctypes.POINTER(PagesDesc), ctypes.POINTER(PagesRows)] + [P] * 7,
        "qevict_pages_accept": [ctypes.POINTER(PagesDesc), P, P, P, P, P, I32, P],
        "qevict_pages_select": [ctypes.POINTER(PagesDesc), P, P, P],
        "qevict_pages_trim": [ctypes.POINTER(PagesDesc), P, P, P],
        "qevict_pages_compact": [ctypes.POINTER(PagesDesc), P, P, P, P],
        "qevict_paged_attn_bytes": [ctypes.POINTER(PagedAttnDesc), ctypes.POINTER(ctypes.c_size_t)],
        "qevict_paged_attn": [ctypes.POINTER(PagedAttnDesc), ctypes.POINTER(PagedAttnMask)] + [P] * 8 +
                             [ctypes.c_size_t, P],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    lib.qevict_status_string.argtypes = [ctypes.c_int]
    lib.qevict_status_string.restype = ctypes.c_char_p
    _lib = lib
    return lib


def exported_symbols():
    """Names of the C ABI entry points declared in include/qevict.h."""
    return ["qevict_budget", "qevict_cache_bytes", "qevict_init_cache", "qevict_get_layout",
            "qevict_prefill_scores", "qevict_prefill_route", "qevict_decode_step", "qevict_route",
            "qevict_read_counters", "qevict_check", "qevict_destroy", "qevict_status_string",
            "qevict_prefill_scores_noalloc", "qevict_flush_scores", "qevict_get_tuple", "qevict_export_bytes",
            "qevict_export_state", "qevict_import_state", "qevict_set_rope_table", "qevict_diag_bytes",
            "qevict_diag_init", "qevict_diag_route", "qevict_diag_read", "qevict_diag_destroy",
            "qevict_selftest_wait", "qevict_prefill_scores_noalloc_status", "qevict_debug_cap_free_slots",
            "qevict_read_status", "qevict_rope_angles", "qevict_rope_table", "qevict_rope_apply", "qevict_attn_bytes",
            "qevict_attn", "qevict_prefix_attn_bytes", "qevict_prefix_attn", "qevict_ops_status",
            "qevict_pages_get_layout", "qevict_pages_load", "qevict_pages_reserve", "qevict_pages_append",
            "qevict_pages_accept", "qevict_pages_select", "qevict_pages_trim", "qevict_pages_compact",
            "qevict_paged_attn_bytes", "qevict_paged_attn"]


def _check(status: int, where: str):
    if status != OK:
        raise QEvictError(status, where, load().qevict_status_string(status).decode())


def make_config(wl, **over) -> Config:
    """C config from any object with the workload's field names (e.g. synth.Workload)."""
    c = Config()
    for name, _ in Config._fields_:
        if name == "b_total":
            c.b_total = int(over.get("b_total", getattr(wl, "b_total", 0) or 0))
        elif name == "max_len":
            c.max_len = int(over.get("max_len", wl.prompt_len + wl.steps))
        elif name in ("decay", "pnorm"):
            setattr(c, name, float(over.get(name, getattr(wl, name, 0.0))))
        elif name in ("ranker", "no_promotion"):
            setattr(c, name, int(over.get(name, getattr(wl, name, 0))))
        elif name == "rope":   # keys carry RoPE and are quantised before it when the workload has a base
            c.rope = int(over.get("rope", 1 if float(getattr(wl, "rope_base", 0.0) or 0.0) > 0 else 0))
        elif name == "reserved0":
            c.reserved0 = 0
        else:
            setattr(c, name, int(over.get(name, getattr(wl, name))))
    return c


def budget(cfg: Config) -> BudgetInfo:
    b = BudgetInfo()
    _check(load().qevict_budget(ctypes.byref(cfg), ctypes.byref(b)), "qevict_budget")
    return b


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream=None) -> int:
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def prefill_scores_noalloc(batch, prompt_len, h_q, h_kv, n_sink, window, q_prompt, k_prompt, s0_out, stream=None):
    """Prefill scores through the allocation-free entry point (scratch inside the library image)."""
    _check(load().qevict_prefill_scores_noalloc(batch, prompt_len, h_q, h_kv, n_sink, window, _ptr(q_prompt),
                                                _ptr(k_prompt), _ptr(s0_out), _stream(stream)),
           "qevict_prefill_scores_noalloc")


def prefill_scores_noalloc_status(stream=None):
    """Reads and clears the allocation-free entry point's device status word (raises EDEVICE if set)."""
    _check(load().qevict_prefill_scores_noalloc_status(_stream(stream)), "qevict_prefill_scores_noalloc_status")


class Cache:
    """A QEvict cache over a torch-allocated arena (uint8 CUDA tensor)."""

    def __init__(self, cfg: Config, device="cuda", stream=None, arena=None):
        import torch
        lib = load()
        self.cfg = cfg
        self.bud = budget(cfg)
        nbytes = ctypes.c_size_t()
        _check(lib.qevict_cache_bytes(ctypes.byref(cfg), ctypes.byref(nbytes)), "qevict_cache_bytes")
        self.arena = arena if arena is not None else torch.empty(nbytes.value, dtype=torch.uint8, device=device)
        if self.arena.data_ptr() % 256:
            raise QEvictError(EINVAL, "Cache", "arena must be 256-byte aligned")
        h = ctypes.c_void_p()
        _check(lib.qevict_init_cache(ctypes.byref(cfg), self.arena.data_ptr(), self.arena.numel(), _stream(stream),
                                     ctypes.byref(h)), "qevict_init_cache")
        self.handle = h
        self.layout = Layout()
        _check(lib.qevict_get_layout(h, ctypes.byref(self.layout)), "qevict_get_layout")

    def close(self):
        if self.handle:
            load().qevict_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # ---- the C ABI calls
    def prefill_scores(self, q_prompt, k_prompt, s0_out, stream=None):
        _check(load().qevict_prefill_scores(self.handle, _ptr(q_prompt), _ptr(k_prompt), _ptr(s0_out),
                                            _stream(stream)), "qevict_prefill_scores")

    def set_rope_table(self, table, stream=None):
        """table: fp32 CUDA tensor [rows][64][2] of (cos, sin) per position and channel pair."""
        import torch
        if table.dtype != torch.float32 or not table.is_cuda or not table.is_contiguous():
            raise QEvictError(EINVAL, "set_rope_table", "table must be a contiguous float32 CUDA tensor")
        _check(load().qevict_set_rope_table(self.handle, _ptr(table), int(table.shape[0]), _stream(stream)),
               "qevict_set_rope_table")

    def prefill_route(self, layer: int, k_prompt, v_prompt, s0=None, q_prompt=None, stream=None):
        _check(load().qevict_prefill_route(self.handle, layer, _ptr(k_prompt), _ptr(v_prompt), _ptr(s0),
                                           _ptr(q_prompt), _stream(stream)), "qevict_prefill_route")

    def decode_step(self, layer: int, q, k_new, v_new, out, stream=None):
        _check(load().qevict_decode_step(self.handle, layer, _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(out),
                                         _stream(stream)), "qevict_decode_step")

    def route(self, stream=None):
        _check(load().qevict_route(self.handle, _stream(stream)), "qevict_route")

    def flush_scores(self, stream=None):
        _check(load().qevict_flush_scores(self.handle, _stream(stream)), "qevict_flush_scores")

    def tuple(self, layer: int, seq: int) -> Tuple:
        t = Tuple()
        _check(load().qevict_get_tuple(self.handle, layer, seq, ctypes.byref(t)), "qevict_get_tuple")
        return t

    def export_state(self, stream=None):
        """Checkpoint of the whole cache as a host uint8 numpy array (synchronises the stream)."""
        import numpy as np
        n = ctypes.c_size_t()
        _check(load().qevict_export_bytes(self.handle, ctypes.byref(n)), "qevict_export_bytes")
        buf = np.empty(n.value, dtype=np.uint8)
        _check(load().qevict_export_state(self.handle, buf.ctypes.data, buf.nbytes, _stream(stream)),
               "qevict_export_state")
        return buf

    def import_state(self, buf, stream=None):
        """Loads a checkpoint made by export_state of a cache with the same configuration."""
        import numpy as np
        buf = np.ascontiguousarray(buf, dtype=np.uint8)
        _check(load().qevict_import_state(self.handle, buf.ctypes.data, buf.nbytes, _stream(stream)),
               "qevict_import_state")

    def counters(self, stream=None) -> dict:
        buf = (ctypes.c_int64 * 7)()
        _check(load().qevict_read_counters(self.handle, buf, _stream(stream)), "qevict_read_counters")
        return dict(zip(COUNTER_NAMES, list(buf)))

    def check(self, stream=None):
        _check(load().qevict_check(self.handle, _stream(stream)), "qevict_check")

    def selftest_wait(self, stream=None):
        """Enqueue the bounded-wait self-test: a wait that runs out and records a timeout."""
        _check(load().qevict_selftest_wait(self.handle, _stream(stream)), "qevict_selftest_wait")

    def status_word(self, stream=None) -> int:
        """The device status word (bit 1 timeout, 2 slot exhaustion, 4 inconsistent state, 8 bounds)."""
        w = ctypes.c_int32()
        _check(load().qevict_read_status(self.handle, ctypes.byref(w), _stream(stream)), "qevict_read_status")
        return w.value

    def debug_cap_free_slots(self, cap: int):
        """Routing events see at most `cap` free F / ledger slots (-1: no cap); a test hook."""
        _check(load().qevict_debug_cap_free_slots(self.handle, cap), "qevict_debug_cap_free_slots")

    # ---- tensor views of the cache tuple inside the arena (read-only use in tests)
    def region(self, name: str, unit: int, nbytes: int):
        off = getattr(self.layout, f"off_{name}") + unit * getattr(self.layout, f"stride_{name}")
        return self.arena[off:off + nbytes]

    def unit(self, layer: int, seq: int) -> int:
        return layer * self.cfg.batch + seq


class Diagnostics:
    """Routing diagnostics of a policy cache against a FullKV cache fed the same inputs (QEvict App. I).
    Create after both caches are prefilled; call route() in place of both caches' route()."""

    def __init__(self, policy: "Cache", fullkv: "Cache", horizon: int = 0, lir_m: int = 0, stream=None):
        import torch
        lib = load()
        self.policy, self.fullkv = policy, fullkv
        self.dc = DiagConfig(horizon, lir_m)
        n = ctypes.c_size_t()
        _check(lib.qevict_diag_bytes(policy.handle, ctypes.byref(self.dc), ctypes.byref(n)), "qevict_diag_bytes")
        self.buf = torch.empty(n.value, dtype=torch.uint8, device=policy.arena.device)
        h = ctypes.c_void_p()
        _check(lib.qevict_diag_init(policy.handle, fullkv.handle, ctypes.byref(self.dc), self.buf.data_ptr(),
                                    self.buf.numel(), _stream(stream), ctypes.byref(h)), "qevict_diag_init")
        self.handle = h

    def route(self, stream=None):
        _check(load().qevict_diag_route(self.handle, _stream(stream)), "qevict_diag_route")

    def report(self, stream=None) -> dict:
        r = DiagReport()
        _check(load().qevict_diag_read(self.handle, ctypes.byref(r), _stream(stream)), "qevict_diag_read")
        import numpy as np
        return {"events": r.events, "fmm": r.fmm, "fmm_terms": r.fmm_terms, "churn": r.churn,
                "churn_terms": r.churn_terms, "qsa": r.qsa, "r_q": r.r_q, "qsa_terms": r.qsa_terms,
                "tier_mass": np.array(list(r.tier_mass)), "lir_eligible": r.lir_eligible,
                "lir_rescued": r.lir_rescued, "lir_fullkv_eligible": r.lir_fullkv_eligible,
                "lir_fullkv_rescued": r.lir_fullkv_rescued, "lag": np.array(list(r.lag)).reshape(8, 2, 2)}

    def close(self):
        if self.handle:
            load().qevict_diag_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---------------------------------------------------------------------------------------------- operators
# Rotary positions, attention over dense tensors and over a cache in pages (no cache handle).  Tensors keep their strides; a call
# runs on the device of its first tensor, on `stream` or that device's current stream.

_ROPE_SCALING = {"none": 0, "linear": 1, "ntk": 2, "parts": 3}


def _dtype_code(dtype, where, allowed):
    import torch
    code = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}.get(dtype)
    if code is None or code not in allowed:
        raise QEvictError(EINVAL, where, f"unsupported dtype {dtype}")
    return code


def _need(ok, where, what):
    if not ok:
        raise QEvictError(EINVAL, where, what)


def _tensor(t, where, name, shape, dtype, device, dense=False):
    """Checks one tensor argument: CUDA, on the call's device, of this shape and dtype, channels contiguous."""
    _need(t.is_cuda and t.device == device, where, f"{name} must be a CUDA tensor on {device}")
    _need(tuple(t.shape) == tuple(shape), where, f"{name} must have shape {tuple(shape)}, has {tuple(t.shape)}")
    _need(t.dtype == dtype, where, f"{name} must be {dtype}, is {t.dtype}")
    if dense:
        _need(t.is_contiguous(), where, f"{name} must be contiguous")
    else:
        _need(t.shape[-1] == 1 or t.stride(-1) == 1, where, f"{name}'s channels must be contiguous")


def _enter(device_index, stream, tensors, home=None, own=()):
    """The raw stream of a call on a device, and the device to make current for it (None: it is).  Tensors used on
    another stream than the device's current one are made known to the allocator (so they are checked before), and so are
    the operator's `own`, which its caller does not see, on any stream but the one they were made on, `home`."""
    torch = _torch_module or _torch()
    other = None if torch._C._cuda_getDevice() == device_index else torch.device("cuda", device_index)
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(device_index)
        if own and raw != home:
            for t in own:
                t.record_stream(torch.cuda.current_stream(device_index))
        return raw, other
    _need(stream.device.index == device_index, "stream", f"{stream} is not on the tensors' device cuda:{device_index}")
    if stream != torch.cuda.current_stream(device_index):
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
    if stream.cuda_stream != home:
        for t in own:
            t.record_stream(stream)
    return stream.cuda_stream, other


def _home(index):
    """The raw stream that new tensors of a device belong to."""
    return _torch()._C._cuda_getCurrentRawStream(index)


def _call(name, other, args, turns=None):
    """One C call, with the call's device current.  ctypes lets other threads run meanwhile; of a plan or cache, whose calls
    enqueue kernels that belong together, they take turns by its lock."""
    fn = getattr(_lib or load(), name)
    if turns is not None:
        turns.acquire()
    try:
        if other is None:
            st = fn(*args)
        else:
            with _torch().cuda.device(other):
                st = fn(*args)
    finally:
        if turns is not None:
            turns.release()
    if st != OK:
        _check(st, name)


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _array(where, name, t, shape, dtype, index):
    """Address of a dense device array of this shape and dtype; None stays None."""
    if t is None:
        return None
    if not (t.dtype is dtype and t.get_device() == index and t.shape == shape and t.is_contiguous()):
        _tensor(t, where, name, shape, dtype, _torch().device("cuda", index), dense=True)
    return t.data_ptr()


def _no_graph(where, tensors):
    """Refuses inputs that ask for a gradient: no graph is recorded, and the outputs would silently have none."""
    for t in tensors:
        if t is not None and t.requires_grad and _torch().is_grad_enabled():
            raise QEvictError(EINVAL, where, "no gradient is recorded: call under torch.no_grad(), or with detached tensors")


def _fits(t, shape, dtype, index):
    """Fast form of _tensor's checks but for the strides (a descriptor made for them has passed): true when all hold."""
    return t.shape == shape and t.dtype is dtype and t.get_device() == index


def _settled(t):
    """Waits until what the current stream has written to a new tensor is there, so that any stream may use it (in a
    capture the writes are the graph's)."""
    torch = _torch()
    if t.is_cuda:
        with torch.cuda.device(t.device):
            if not torch.cuda.is_current_stream_capturing():
                torch.cuda.current_stream().synchronize()


_TIMEOUT = 1   # bit of a status word: a wait ran out


def _ops_status(word, stream):
    """Synchronises the stream and raises if the status word was set (cleared then); the error has it as `word`."""
    s, other = _enter(word.get_device(), stream, (word,))
    bits = ctypes.c_int32()
    try:
        _call("qevict_ops_status", other, (word.data_ptr(), ctypes.byref(bits), s))
    except QEvictError as e:
        e.word = bits.value
        raise


def _rope_config(rot_dim, base, scaling, factor, orig_len, low, high):
    _need(scaling in _ROPE_SCALING, "rope", f"scaling must be one of {sorted(_ROPE_SCALING)}, is {scaling!r}")
    return RopeConfig(int(rot_dim), _ROPE_SCALING[scaling], float(base), float(factor), float(orig_len), float(low),
                      float(high))


def rope_angles(rot_dim=128, base=10000.0, scaling="none", factor=1.0, orig_len=0, low=1.0, high=32.0):
    """Angle per position of every rotated pair, as a list of floats (host fp64)."""
    cfg = _rope_config(rot_dim, base, scaling, factor, orig_len, low, high)
    out = (ctypes.c_double * max(1, int(rot_dim) // 2))()
    _check(load().qevict_rope_angles(ctypes.byref(cfg), out), "qevict_rope_angles")
    return list(out)


def rope_table(rows, rot_dim=128, base=10000.0, scaling="none", factor=1.0, orig_len=0, low=1.0, high=32.0, first=0,
               out=None, device="cuda", stream=None):
    """fp32 [rows][rot_dim / 2][2] table of (cos, sin) of the positions from `first` on, for Rope and (rot_dim 128,
    first 0) Cache.set_rope_table.  scaling: "none", "linear", "ntk" or "parts"; see qevict_rope_config."""
    import torch
    cfg = _rope_config(rot_dim, base, scaling, factor, orig_len, low, high)
    rows = int(rows)
    _need(rows >= 1 and cfg.rot_dim >= 2 and cfg.rot_dim % 2 == 0, "rope_table", "rows and an even rot_dim of at least 2")
    shape = (rows, cfg.rot_dim // 2, 2)
    if out is None:
        rope_angles(rot_dim, base, scaling, factor, orig_len, low, high)   # refuses before anything is allocated
        with torch.cuda.device(device), torch.cuda.stream(stream):
            out = torch.empty(shape, dtype=torch.float32, device=device)
    if not (out.is_cuda and out.dtype is torch.float32 and out.shape == shape and out.is_contiguous()):
        _tensor(out, "rope_table", "out", shape, torch.float32, out.device, dense=True)
    s, other = _enter(out.get_device(), stream, (out,))
    _call("qevict_rope_table", other, (ctypes.byref(cfg), int(first), rows, out.data_ptr(), s))
    return out


class Rope:
    """Rotations with one (cos, sin) table (fp32 [rows][rot_dim / 2][2], e.g. from rope_table)."""

    def __init__(self, table):
        import torch
        load()
        _need(table.dim() == 3 and table.shape[2] == 2, "Rope", "table must have shape [rows][rot_dim / 2][2]")
        _tensor(table, "Rope", "table", table.shape, torch.float32, table.device, dense=True)
        self.table = table
        self.index = table.get_device()
        self.status = torch.zeros(1, dtype=torch.int32, device=table.device)
        _settled(self.status)
        self._home, self._own = _home(self.index), (table, self.status)
        table.record_stream(torch.cuda.current_stream(self.index))   # it may have been made on another
        self._table_ptr, self._status_ptr, self._descs = table.data_ptr(), self.status.data_ptr(), {}

    def apply(self, q, k=None, positions=None, pos0=0, interleaved=False, inverse=False, factor=1.0, q_out=None,
              k_out=None, stream=None):
        """Rotates q [batch][seq][heads][d] and, if given, k; returns (q_out, k_out), new tensors unless given
        (q_out=q rotates in place).  positions: int32 [batch][seq], default pos0 + t.  inverse=True rotates back
        and, with the same factor, is the gradient of the forward call.  Tokens whose position is outside the
        table are not written; check() reports them.  Nothing is recorded for autograd: q and k that require a gradient
        are refused unless gradients are off."""
        index = self.index
        _no_graph("Rope.apply", (q, k))
        if k is None:
            _need(k_out is None, "Rope.apply", "k_out without k")
        if q_out is None or (k_out is None and k is not None):
            q_out, k_out = self._outputs(q, k, q_out, k_out, stream)
        dt, shape = q.dtype, q.shape
        key = (dt, shape, q.stride(), q_out.stride(), interleaved, inverse, factor, pos0)
        if k is not None:
            key += (k.shape, k.stride(), k_out.stride())
        desc = self._descs.get(key)
        if desc is None:
            desc = self._desc(key, q, k, q_out, k_out, interleaved, inverse, factor, pos0)
        if not (q.get_device() == index and _fits(q_out, shape, dt, index)):
            _tensor(q, "Rope.apply", "q", shape, dt, self.table.device)
            _tensor(q_out, "Rope.apply", "q_out", shape, dt, self.table.device)
        if k is not None and not (k.dtype is dt and k.get_device() == index and _fits(k_out, k.shape, dt, index)):
            _tensor(k, "Rope.apply", "k", k.shape, dt, self.table.device)
            _tensor(k_out, "Rope.apply", "k_out", k.shape, dt, self.table.device)
        if positions is not None:
            _array("Rope.apply", "positions", positions, shape[:2], _torch().int32, index)
        st, other = _enter(index, stream, (q, k, q_out, k_out, positions), self._home, self._own)
        _call("qevict_rope_apply", other,
              (desc, self._table_ptr, None if positions is None else positions.data_ptr(), q.data_ptr(), q_out.data_ptr(),
               None if k is None else k.data_ptr(), None if k is None else k_out.data_ptr(), self._status_ptr, st))
        return q_out, k_out

    def _outputs(self, q, k, q_out, k_out, stream):
        import torch
        with torch.cuda.device(self.table.device), torch.cuda.stream(stream):
            if q_out is None:
                q_out = torch.empty(q.shape, dtype=q.dtype, device=self.table.device)
            if k is not None and k_out is None:
                k_out = torch.empty(k.shape, dtype=k.dtype, device=self.table.device)
        return q_out, k_out

    def _desc(self, key, q, k, q_out, k_out, interleaved, inverse, factor, pos0):
        """Descriptor of calls with these shapes and strides, kept for the next one."""
        where, dev = "Rope.apply", self.table.device
        _need(q.dim() == 4 and (k is None or k.dim() == 4), where, "q and k must be [batch][seq][heads][d]")
        b, s, hq, d = q.shape
        _tensor(q, where, "q", q.shape, q.dtype, dev)
        _tensor(q_out, where, "q_out", q.shape, q.dtype, dev)
        desc = RopeDesc(_dtype_code(q.dtype, where, (0, 1, 2)), b, s, hq, 0 if k is None else k.shape[2], d,
                        2 * self.table.shape[1], int(bool(interleaved)), int(bool(inverse)), float(factor),
                        self.table.shape[0], int(pos0), _Stride3(*q.stride()[:3]), _Stride3(*q_out.stride()[:3]))
        if k is not None:
            _tensor(k, where, "k", (b, s, k.shape[2], d), q.dtype, dev)
            _tensor(k_out, where, "k_out", k.shape, q.dtype, dev)
            desc.k_in, desc.k_out = _Stride3(*k.stride()[:3]), _Stride3(*k_out.stride()[:3])
        if len(self._descs) > 64:
            self._descs.clear()
        ref = self._descs[key] = ctypes.byref(desc)
        return ref

    def check(self, stream=None):
        """Raises EDEVICE if a call since the last check met a position outside the table.  Synchronises `stream` (the
        current one unless given): the one that the calls ran on."""
        _ops_status(self.status, stream)


class _AttnPlan:
    """Sizes, options and the workspace of an attention operator.  A plan serves one call at a time: calls that can
    overlap on the GPU (two streams, two replayed graphs) need plans of their own.  Host threads may share a plan on one
    stream."""

    def _setup(self, where, batch, s_q, s_kv, h_q, h_kv, dtype, causal, softcap, scale, device):
        import torch
        self.desc = AttnDesc(_dtype_code(dtype, where, (0, 1)), int(batch), int(s_q), int(s_kv), int(h_q), int(h_kv), 128,
                             int(bool(causal)), float(scale), float(softcap))
        self.dtype = dtype
        self.device = torch.device(device)
        if self.device.type == "cuda" and self.device.index is None and torch.cuda.is_available():
            self.device = torch.device("cuda", torch.cuda.current_device())
        d = self.desc
        dense = lambda s, h: _Stride3(s * h * 128, h * 128, 128)   # noqa: E731
        d.q = d.o = dense(max(1, d.s_q), max(1, d.h_q))
        d.k = d.v = dense(max(1, d.s_kv), max(1, d.h_kv))

    def _workspace(self, nbytes):
        import torch
        self.work = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        self.work[:256].zero_()
        _settled(self.work)
        d = self.desc
        self.index, self._descs = self.work.get_device(), {}
        self._home, self._own, self._turns = _home(self.index), (self.work,), threading.RLock()
        self._work = (self.work.data_ptr(), nbytes)
        self.q_shape, self.kv_shape = (d.batch, d.s_q, d.h_q, 128), (d.batch, d.s_kv, d.h_kv, 128)

    def _tensors(self, where, q, k, v, out, lse, stream, strides=()):
        """Checks a call's tensors, makes the outputs that were not given; the descriptor with the call's strides (kept for
        the next call of the same strides)."""
        dt, i = self.dtype, self.index
        if out is None or lse is None:
            import torch
            with torch.cuda.device(self.device), torch.cuda.stream(stream):
                if out is None:
                    out = torch.empty(self.q_shape, dtype=dt, device=self.device)
                if lse is None:
                    lse = torch.empty(self.q_shape[:3], dtype=torch.float32, device=self.device)
        qs, ks = self.q_shape, self.kv_shape
        if not (q.dtype is dt and k.dtype is dt and v.dtype is dt and out.dtype is dt and q.shape == qs and out.shape == qs and
                k.shape == ks and v.shape == ks and
                q.get_device() == k.get_device() == v.get_device() == out.get_device() == i):
            for name, t, shape in (("q", q, self.q_shape), ("k", k, self.kv_shape), ("v", v, self.kv_shape),
                                   ("out", out, self.q_shape)):
                _tensor(t, where, name, shape, dt, self.device)
        _array(where, "lse", lse, qs[:3], _torch().float32, i)
        key = (q.stride(), k.stride(), v.stride(), out.stride()) + strides
        desc = self._descs.get(key)
        if desc is None:
            _need(all(st[-1] == 1 for st in key), where, "the channels of every tensor must be contiguous")
            if len(self._descs) > 64:
                self._descs.clear()
            desc = self._descs[key] = ctypes.byref(self._with_strides(key))
        return desc, out, lse

    def _with_strides(self, key):
        desc = AttnDesc.from_buffer_copy(self.desc)
        desc.q, desc.k, desc.v, desc.o = (_Stride3(*st[:3]) for st in key[:4])
        return desc

    def check(self, stream=None):
        """Raises EDEVICE if a call since the last check recorded a fault: a length outside its range (clamped), or
        a wait that ran out.  Synchronises `stream` (the current one unless given): the one that the calls ran on."""
        try:
            _ops_status(self.work, stream)
        except QEvictError as e:
            if e.word & _TIMEOUT:   # which leaves the count of units undone; no call is under way now
                with _torch().cuda.stream(stream):
                    self.work[:256].zero_()
                    _settled(self.work)
            raise


class Attention(_AttnPlan):
    """Attention of the last q_len[b] positions of every sequence over a dense KV cache: prompts (s_q = s_kv), a
    prompt's last chunk, single tokens (s_q = 1).  See qevict_attn for the masks and the definition."""

    def __init__(self, batch, s_q, s_kv, h_q, h_kv, dtype=None, causal=True, softcap=0.0, scale=0.0, device="cuda"):
        import torch
        self._setup("Attention", batch, s_q, s_kv, h_q, h_kv, dtype or torch.bfloat16, causal, softcap, scale, device)
        n = ctypes.c_size_t()
        with torch.cuda.device(self.device):
            _check(load().qevict_attn_bytes(ctypes.byref(self.desc), ctypes.byref(n)), "qevict_attn_bytes")
        self._workspace(n.value)

    def run(self, q, k, v, out=None, lse=None, slopes=None, q_len=None, kv_len=None, prefix_len=None, doc_ids=None,
            stream=None):
        """q [batch][s_q][h_q][128], k, v [batch][s_kv][h_kv][128], any strides that are multiples of 8 elements;
        returns (out, lse), new tensors unless given.  Rows behind q_len[b] are not written.  There is no backward pass:
        inputs that require a gradient are refused unless gradients are off."""
        _no_graph("Attention.run", (q, k, v, slopes))
        desc, out, lse = self._tensors("Attention.run", q, k, v, out, lse, stream)
        d, i, mask = self.desc, self.index, None
        if not (slopes is None and q_len is None and kv_len is None and prefix_len is None and doc_ids is None):
            f32, i32, where = _torch().float32, _torch().int32, "Attention.run"
            batch = self.q_shape[:1]
            mask = ctypes.byref(AttnMask(_array(where, "slopes", slopes, (d.h_q,), f32, i),
                                         _array(where, "q_len", q_len, batch, i32, i),
                                         _array(where, "kv_len", kv_len, batch, i32, i),
                                         _array(where, "prefix_len", prefix_len, batch, i32, i),
                                         _array(where, "doc_ids", doc_ids, (d.batch, d.s_kv), i32, i)))
        s, other = _enter(i, stream, (q, k, v, out, lse, slopes, q_len, kv_len, prefix_len, doc_ids), self._home, self._own)
        _call("qevict_attn", other, (desc, mask, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                                     *self._work, s), self._turns)
        return out, lse


class PrefixAttention(_AttnPlan):
    """Causal attention of s_q new tokens of every sequence over a prefix that all sequences share (read once) and
    each sequence's own keys behind it.  s_kv: room for own keys.  See qevict_prefix_attn."""

    def __init__(self, batch, s_q, s_prefix, s_kv, h_q, h_kv, dtype=None, softcap=0.0, scale=0.0, device="cuda"):
        import torch
        self._setup("PrefixAttention", batch, s_q, s_kv, h_q, h_kv, dtype or torch.bfloat16, True, softcap, scale, device)
        self.s_prefix, self.prefix_shape = int(s_prefix), (int(s_prefix), int(h_kv), 128)
        n = ctypes.c_size_t()
        st = _Stride2(self.desc.h_kv * 128, 128)
        pd = PrefixAttnDesc(self.desc, self.s_prefix, st, st)
        with torch.cuda.device(self.device):
            _check(load().qevict_prefix_attn_bytes(ctypes.byref(pd), ctypes.byref(n)), "qevict_prefix_attn_bytes")
        self._workspace(n.value)

    def run(self, q, k_prefix, v_prefix, k, v, out=None, lse=None, slopes=None, kv_len=None, stream=None):
        """q [batch][s_q][h_q][128], k_prefix, v_prefix [s_prefix][h_kv][128], k, v [batch][s_kv][h_kv][128];
        returns (out, lse), new tensors unless given.  Inputs that require a gradient are refused unless gradients are
        off."""
        where, d, i = "PrefixAttention.run", self.desc, self.index
        _no_graph(where, (q, k_prefix, v_prefix, k, v, slopes))
        desc, out, lse = self._tensors(where, q, k, v, out, lse, stream, (k_prefix.stride(), v_prefix.stride()))
        if not (_fits(k_prefix, self.prefix_shape, self.dtype, i) and _fits(v_prefix, self.prefix_shape, self.dtype, i)):
            for name, t in (("k_prefix", k_prefix), ("v_prefix", v_prefix)):
                _tensor(t, where, name, self.prefix_shape, self.dtype, self.device)
        args = (desc, _array(where, "slopes", slopes, (d.h_q,), _torch().float32, i),
                _array(where, "kv_len", kv_len, self.q_shape[:1], _torch().int32, i), q.data_ptr(), k_prefix.data_ptr(),
                v_prefix.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), *self._work)
        s, other = _enter(i, stream, (q, k_prefix, v_prefix, k, v, out, lse, slopes, kv_len), self._home, self._own)
        _call("qevict_prefix_attn", other, (*args, s), self._turns)
        return out, lse

    def _with_strides(self, key):
        return PrefixAttnDesc(super()._with_strides(key), self.s_prefix, _Stride2(*key[4][:2]), _Stride2(*key[5][:2]))


def _sizes(where, **sizes):
    """Sizes as ints of the C interface; one that is larger, or no whole number, would be another there."""
    res = []
    for name, n in sizes.items():
        try:
            whole = int(n)
        except (TypeError, ValueError, OverflowError):
            whole = None
        _need(whole is not None and whole == n, where, f"{name} is no whole number: {n!r}")
        _need(-2 ** 31 <= whole < 2 ** 31, where, f"{name} is out of range: {n}")
        res.append(whole)
    return tuple(res)


class PagedCache:
    """A KV cache in pages: the pool k, v [layers][pages][page][h_kv][128], and which pages hold the tokens of each of
    `batch` sequences (at most max_pages each).  A step: reserve() room, append() each layer's new rows, attend
    (PagedAttention), accept() what counts.  select() forks, reorders and frees; trim() shortens; compact() gathers the pages in
    use at the pool's beginning.  See qevict_pages_* for what each does.

    length, held [batch], table [batch][max_pages], refs [pages] and n_free are views of `state`, one int32 tensor: with copies
    of it and the pool a cache is saved and restored.  Calls of a cache run in order: one stream (host threads may share it), or
    ordered by the caller."""

    def __init__(self, layers, pages, page, h_kv, batch, max_pages, dtype=None, device="cuda", k=None, v=None):
        import torch
        where = "PagedCache"
        self.dtype = dtype or torch.bfloat16
        _dtype_code(self.dtype, where, (0, 1))
        _need((k is None) == (v is None), where, "k and v are given together")
        self.device = torch.device(device) if k is None else k.device
        _need(self.device.type == "cuda", where, "the pool must be on a CUDA device")
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        layers, pages, page, h_kv, batch, max_pages = _sizes(where, layers=layers, pages=pages, page=page, h_kv=h_kv, batch=batch,
                                                            max_pages=max_pages)
        shape = (layers, pages, page, h_kv, 128)
        step = [shape[1] * shape[2] * shape[3] * 128, shape[2] * shape[3] * 128, shape[3] * 128, 128]
        if k is not None:
            for name, t in (("k", k), ("v", v)):
                _tensor(t, where, name, shape, self.dtype, self.device)
            _no_graph(where, (k, v))
        desc = PagesDesc(*shape, batch, max_pages, 0,
                         _Stride4(*(step if k is None else k.stride()[:4])),
                         _Stride4(*(step if v is None else v.stride()[:4])))
        self.layout = PagesLayout()
        _check(load().qevict_pages_get_layout(ctypes.byref(desc), ctypes.byref(self.layout)), "qevict_pages_get_layout")
        if k is None:
            k = torch.empty(shape, dtype=self.dtype, device=self.device)
            v = torch.empty(shape, dtype=self.dtype, device=self.device)
        self.k, self.v, self.shape, self.batch = k, v, shape, batch
        self.state = torch.empty(self.layout.ints, dtype=torch.int32, device=self.device)
        part = lambda off, n: self.state[off:off + n]   # noqa: E731
        lay = self.layout
        self.n_free = part(lay.n_free, 1)
        self.length, self.held, self.refs = part(lay.length, desc.batch), part(lay.held, desc.batch), part(lay.refs, desc.pages)
        self.table = part(lay.table, desc.batch * desc.max_pages).view(desc.batch, desc.max_pages)
        self.index, self._i32 = self.state.get_device(), torch.int32
        self._seqs, self._home, self._own = self.length.shape, _home(self.index), (self.state, k, v)
        self._turns = threading.RLock()
        self._desc, self._state, self._pool, self._rows = ctypes.byref(desc), self.state.data_ptr(), \
            (k.data_ptr(), v.data_ptr()), {}
        self.load()
        _settled(self.state)

    def _ints(self, where, name, t, shape):
        """Address of an int32 array of this shape."""
        if t is not None and t.dtype is self._i32 and t.shape == shape and t.get_device() == self.index and t.is_contiguous():
            return t.data_ptr()
        return _array(where, name, t, shape, self._i32, self.index)

    def _run(self, name, stream, tensors, *args):
        s, other = _enter(self.index, stream, tensors, self._home, self._own)
        _call(name, other, (self._desc, *args, s), self._turns)

    def load(self, table=None, length=None, stream=None):
        """Starts the bookkeeping from a table int32 [batch][max_pages] (-1: no page) and lengths int32 [batch], or empty."""
        where = "PagedCache.load"
        _need((table is None) == (length is None), where, "table and length are given together")
        self._run("qevict_pages_load", stream, (table, length), self._state,
                  self._ints(where, "table", table, self.table.shape), self._ints(where, "length", length, self._seqs))

    def reserve(self, new, stream=None):
        """Makes `new` rows behind every sequence writable: an int, or an int32 tensor [batch]."""
        where = "PagedCache.reserve"
        if hasattr(new, "data_ptr"):
            self._run("qevict_pages_reserve", stream, (new,), *self._pool, self._state,
                      self._ints(where, "new", new, self._seqs), 0)
        else:
            self._run("qevict_pages_reserve", stream, (), *self._pool, self._state, None, *_sizes(where, new=new))

    def append(self, k, v, layer=None, n=None, stream=None):
        """Writes rows behind every sequence's length: k, v [batch][n][h_kv][128] of one layer, or [layers][batch][n][h_kv][128]
        of all.  n: int32 [batch], the rows of each sequence (default all).  Inputs that require a gradient are refused
        unless gradients are off."""
        where = "PagedCache.append"
        _no_graph(where, (k, v))
        key = (k.shape, k.stride(), v.shape, v.stride(), layer)
        rows = self._rows.get(key)
        if rows is None:
            rows = self._rows_of(where, key, k, v, layer)
        i, dt = self.index, self.dtype
        if not (k.dtype is dt and v.dtype is dt and k.get_device() == i and v.get_device() == i):
            for name, t in (("k", k), ("v", v)):
                _tensor(t, where, name, t.shape, dt, self.device)
        self._run("qevict_pages_append", stream, (k, v, n), rows, *self._pool, self._state, k.data_ptr(), v.data_ptr(),
                  self._ints(where, "n", n, self._seqs))

    def _rows_of(self, where, key, k, v, layer):
        """Descriptor of rows with these shapes and strides, kept for the next call."""
        layers, _, _, h_kv, d = self.shape
        _need(k.dim() == (5 if layer is None else 4), where, "k and v must be [layers][batch][n][h_kv][128], or without layers")
        lead = (layers, self.batch) if layer is None else (self.batch,)
        shape = lead + (k.shape[-3], h_kv, d)
        for name, t in (("k", k), ("v", v)):
            _tensor(t, where, name, shape, self.dtype, self.device)
        st = [(0,) * (4 - len(shape) + 1) + tuple(t.stride()[:-1]) for t in (k, v)]
        first = 0
        if layer is not None:
            first, = _sizes(where, layer=layer)
            _need(0 <= first < layers, where, f"layer must be in [0, {layers}), is {layer}")
        rows = ctypes.byref(PagesRows(first, layers if layer is None else 1, shape[-3], 0,
                                      _Stride4(*st[0]), _Stride4(*st[1])))
        if len(self._rows) > 256:   # (another thread may clear them too)
            self._rows.clear()
        self._rows[key] = rows
        return rows

    def accept(self, count, path=None, stream=None):
        """The first count[b] rows behind each length count from now on; with path int32 [batch][max_path], max_path 1 to 256,
        rows path[b][j] (strictly ascending) move there first."""
        where, most = "PagedCache.accept", 0
        if path is not None:
            _need(path.dim() == 2 and 1 <= path.shape[1] <= 256, where,   # (one of no columns has no address: it would be none)
                  f"path must be [batch][1 to 256], has shape {tuple(path.shape)}")
            most = path.shape[1]
            path_at = self._ints(where, "path", path, (self.batch, most))
        self._run("qevict_pages_accept", stream, (count, path), *self._pool, self._state,
                  self._ints(where, "count", count, self._seqs), None if path is None else path_at, most)

    def select(self, src, stream=None):
        """Sequence b becomes a copy of what sequence src[b] (int32 [batch]) was, or ends (-1); pages are shared, no rows copied."""
        self._run("qevict_pages_select", stream, (src,), self._state,
                  self._ints("PagedCache.select", "src", src, self._seqs))

    def trim(self, length, stream=None):
        """Cuts sequences to their first length[b] tokens (int32 [batch]; negative: as it is) and gives pages behind back."""
        self._run("qevict_pages_trim", stream, (length,), self._state,
                  self._ints("PagedCache.trim", "length", length, self._seqs))

    def compact(self, stream=None):
        """Moves the pages in use to the beginning of the pool."""
        self._run("qevict_pages_compact", stream, (), *self._pool, self._state)

    def check(self, stream=None):
        """Raises EDEVICE if a call since the last check recorded a fault: too few free pages, an argument or index out of
        range, a table that cannot be.  Synchronises `stream` (the current one unless given): the one that the calls ran on."""
        _ops_status(self.state, stream)


class PagedAttention(_AttnPlan):
    """Attention of the newest tokens of every sequence over a cache in pages: single tokens (s_q = 1), chunks of a prompt,
    trees of drafts.  See qevict_paged_attn."""

    def __init__(self, batch, s_q, pages, page, max_pages, h_q, h_kv, dtype=None, softcap=0.0, scale=0.0, device="cuda"):
        import torch
        batch, s_q, pages, page, max_pages, h_q, h_kv = _sizes("PagedAttention", batch=batch, s_q=s_q, pages=pages, page=page,
                                                              max_pages=max_pages, h_q=h_q, h_kv=h_kv)
        self._setup("PagedAttention", batch, s_q, 1, h_q, h_kv, dtype or torch.bfloat16, True, softcap, scale, device)
        self.pool_shape, self.table_shape = (pages, page, h_kv, 128), (batch, max_pages)
        n, d = ctypes.c_size_t(), self.desc
        pool, q = (page * h_kv * 128, h_kv * 128, 128), tuple(d.q)
        with torch.cuda.device(self.device):
            _check(load().qevict_paged_attn_bytes(ctypes.byref(self._with_strides((q, pool, pool, q))), ctypes.byref(n)),
                   "qevict_paged_attn_bytes")
        self._workspace(n.value)
        self.kv_shape, self._i32 = self.pool_shape, torch.int32
        self._heads, self._seqs, self._tree, self._trees = (d.h_q,), (d.batch,), (d.s_q,), (d.batch, d.s_q)

    def run(self, q, k, v, table, length, out=None, lse=None, parents=None, q_len=None, slopes=None, stream=None):
        """q [batch][s_q][h_q][128], k, v [pages][page][h_kv][128] (one layer's pool), table int32 [batch][max_pages], length
        int32 [batch]: the tokens before the queries, whose own keys and values stand behind them.  parents: int32
        [batch][s_q], or [s_q] for all.  Returns (out, lse), new tensors unless given; rows behind q_len[b] are not
        written.  Inputs that require a gradient are refused unless gradients are off."""
        where, i, i32, mask = "PagedAttention.run", self.index, self._i32, None
        if q.requires_grad or k.requires_grad or v.requires_grad or slopes is not None:
            _no_graph(where, (q, k, v, slopes))
        desc, out, lse = self._tensors(where, q, k, v, out, lse, stream)
        _need(table is not None and length is not None, where, "table and length are needed")
        if not (slopes is None and q_len is None and parents is None):
            one = parents is not None and parents.dim() == 1
            mask = ctypes.byref(PagedAttnMask(_array(where, "slopes", slopes, self._heads, _torch().float32, i),
                                              _array(where, "q_len", q_len, self._seqs, i32, i),
                                              _array(where, "parents", parents, self._tree if one else self._trees, i32, i),
                                              one))
        args = (desc, mask, q.data_ptr(), k.data_ptr(), v.data_ptr(), _array(where, "table", table, self.table_shape, i32, i),
                _array(where, "length", length, self._seqs, i32, i), out.data_ptr(), lse.data_ptr(), *self._work)
        s, other = _enter(i, stream, (q, k, v, table, length, out, lse, parents, q_len, slopes), self._home, self._own)
        _call("qevict_paged_attn", other, (*args, s), self._turns)
        return out, lse

    def _with_strides(self, key):
        d, (pages, page, h_kv, _) = self.desc, self.pool_shape
        return PagedAttnDesc(d.dtype, d.batch, d.s_q, d.h_q, h_kv, 128, d.scale, d.softcap, pages, page, self.table_shape[1], 0,
                             *(_Stride3(*key[n][:3]) for n in (0, 3, 1, 2)))
