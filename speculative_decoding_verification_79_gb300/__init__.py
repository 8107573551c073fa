"""Python binding of libspecverify (GB300 / sm_103a).

Argument marshalling only: every step of the schedule and of verification runs in the
CUDA kernels of libspecverify.so, called through its C-ABI (include/specverify.h).
PyTorch provides device memory and streams. There is no CPU fallback: without the
built library, or without a CUDA device, calls raise.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import _build

_lib = None

SV_OK, SV_ERR_ARG, SV_ERR_SHAPE, SV_ERR_DTYPE = 0, -1, -2, -3
SV_ERR_CUDA, SV_ERR_DEVICE_INPUT, SV_ERR_TIMEOUT, SV_ERR_WORKSPACE = -4, -5, -6, -7
SV_ERR_NO_PAGES = -8
SV_F32, SV_BF16, SV_F16 = 0, 1, 2
SV_MAX_B, SV_MAX_K = 4096, 32


class _CacheStruct(ctypes.Structure):
    """sv_kv_cache of specverify.h."""

    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale", "table",
                                               "n_pages", "len", "refs")] + \
               [(n, ctypes.c_int) for n in ("layers", "pages", "page", "heads", "dim", "batch",
                                            "max_pages")]


class _RopeStruct(ctypes.Structure):
    """sv_rope_spec of specverify.h."""

    _fields_ = [("freq", ctypes.c_void_p), ("rot", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("gain", ctypes.c_float)]


class SpecVerifyError(RuntimeError):
    def __init__(self, fn, code):
        self.code = code
        super().__init__(f"{fn} failed: {status_string(code)} ({code})")


def library_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = True):
    """Open libspecverify.so (building it first when it is missing or stale)."""
    global _lib
    if _lib is not None:
        return _lib
    if build_if_missing and not _build.up_to_date():
        _build.build()
    if not os.path.exists(_build.LIB):
        raise RuntimeError("libspecverify.so is not built; run __graft_entry__.build()")
    lib = ctypes.CDLL(_build.LIB)
    vp, i32, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.sv_workspace_bytes.argtypes = [i32, i32, i32]
    lib.sv_workspace_bytes.restype = sz
    lib.sv_workspace_init.argtypes = [vp, sz, vp]
    lib.sv_workspace_init.restype = i32
    lib.sv_schedule.argtypes = [vp, i32, i32, f32, i32, vp, vp, sz, vp]
    lib.sv_schedule.restype = i32
    lib.sv_schedule_cal.argtypes = [vp, vp, vp, f32, f32, f32, i32, i32, i32, vp, vp, vp, vp, sz,
                                    vp]
    lib.sv_schedule_cal.restype = i32
    lib.sv_schedule_curve.argtypes = [vp, vp, vp, f32, f32, f32, vp, i32, i32, i32, i32, vp, vp,
                                      vp, vp, vp, vp, sz, vp]
    lib.sv_schedule_curve.restype = i32
    lib.sv_calib_stats_len.argtypes = [i32]
    lib.sv_calib_stats_len.restype = sz
    lib.sv_calib_observe.argtypes = [vp, vp, vp, i32, i32, vp, vp]
    lib.sv_calib_observe.restype = i32
    lib.sv_calib_update.argtypes = [vp, vp, i32, f32, f32, vp, vp]
    lib.sv_calib_update.restype = i32
    lib.sv_markov_keys_len.argtypes = [i32, i32]
    lib.sv_markov_keys_len.restype = sz
    lib.sv_markov_draft.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, sz, vp]
    lib.sv_markov_draft.restype = i32
    lib.sv_verify.argtypes = [vp, vp, i32, vp, vp, vp, i32, i32, i32, f32, vp, vp, vp, sz, vp]
    lib.sv_verify.restype = i32
    lib.sv_verify_diag.argtypes = [vp, vp, i32, vp, vp, vp, i32, i32, i32, f32, vp, vp, vp, vp,
                                   vp, vp, vp, vp, sz, vp]
    lib.sv_set_wait_limit.argtypes = [ctypes.c_longlong]
    lib.sv_set_wait_limit.restype = ctypes.c_longlong
    lib.sv_verify_diag.restype = i32
    lib.sv_verify_tree.argtypes = [vp, vp, i32, vp, vp, vp, vp, i32, i32, i32, f32, vp, vp, vp,
                                   vp, sz, vp]
    lib.sv_verify_tree.restype = i32
    i64, cp = ctypes.c_int64, ctypes.POINTER(_CacheStruct)
    lib.sv_kv_workspace_bytes.argtypes = [cp]
    lib.sv_kv_workspace_bytes.restype = sz
    lib.sv_kv_reserve.argtypes = [cp, vp, vp, vp, sz, vp]
    lib.sv_kv_reserve.restype = i32
    lib.sv_kv_append.argtypes = [cp, i32, vp, vp, i32, i64, i64, i64, i64, i32, vp, vp, sz, vp]
    lib.sv_kv_append.restype = i32
    lib.sv_kv_read.argtypes = [cp, i32, i32, vp, vp, i32, vp, vp, i32, vp, sz, vp]
    lib.sv_kv_read.restype = i32
    lib.sv_kv_attend.argtypes = [cp, i32, vp, i32, i64, i64, i32, i32, vp, vp, f32, i32, i32, vp,
                                 vp, vp, sz, vp]
    lib.sv_kv_attend.restype = i32
    lib.sv_set_share_always.argtypes = [i32]
    lib.sv_set_share_always.restype = i32
    lib.sv_kv_share_bytes.argtypes = [cp, i32, i32]
    lib.sv_kv_share_bytes.restype = sz
    lib.sv_kv_share.argtypes = [cp, vp, vp, sz, vp, sz, vp]
    lib.sv_kv_share.restype = i32
    lib.sv_kv_attend_shared.argtypes = [cp, i32, vp, i32, i64, i64, i32, i32, vp, vp, f32, i32, i32,
                                        vp, vp, vp, sz, vp, sz, vp]
    lib.sv_kv_attend_shared.restype = i32
    lib.sv_kv_commit.argtypes = [cp, vp, vp, i32, vp, sz, vp]
    lib.sv_kv_commit.restype = i32
    lib.sv_kv_fork.argtypes = [cp, vp, vp, vp, sz, vp]
    lib.sv_kv_fork.restype = i32
    f64, rp = ctypes.c_double, ctypes.POINTER(_RopeStruct)
    lib.sv_rope_fixed.argtypes = [vp, i32, vp]
    lib.sv_rope_fixed.restype = i32
    lib.sv_rope_freqs.argtypes = [i32, f64, i32, f64, f64, f64, f64, vp]
    lib.sv_rope_freqs.restype = i32
    lib.sv_rope.argtypes = [rp, vp, i32, i64, i64, i32, i32, i32, i32, vp, vp, vp, vp, i32, vp, i64,
                            i64, vp, sz, vp]
    lib.sv_rope.restype = i32
    lib.sv_kv_append_rope.argtypes = [cp, i32, vp, vp, i32, i64, i64, i64, i64, i32, vp, vp, rp, vp,
                                      i64, i64, i32, vp, i64, i64, vp, sz, vp]
    lib.sv_kv_append_rope.restype = i32
    lib.sv_get_status.argtypes = [vp, vp, i32, ctypes.POINTER(ctypes.c_int32)]
    lib.sv_get_status.restype = i32
    lib.sv_status_string.argtypes = [i32]
    lib.sv_status_string.restype = ctypes.c_char_p
    lib.sv_version.argtypes = []
    lib.sv_version.restype = i32
    _lib = lib
    return lib


load_lib = load  # the library loader, for functions whose arguments shadow `load`


def status_string(code: int) -> str:
    return load().sv_status_string(int(code)).decode()


def _check(fn, code):
    if code != SV_OK:
        raise SpecVerifyError(fn, code)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dev(t, name, dtype=None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t


class Workspace:
    """Device workspace for shapes up to (B, K, V); zeroed once at creation (the
    constructor waits for the zeroing, so the workspace can be used on any stream)."""

    def __init__(self, B, K, V, device=None, stream=None):
        self.nbytes = int(load().sv_workspace_bytes(int(B), int(K), int(V)))
        if self.nbytes == 0:
            raise ValueError(f"unsupported workspace shape B={B} K={K} V={V}")
        self.buf = torch.empty(self.nbytes + 256, dtype=torch.uint8, device=device or "cuda")
        off = (-self.buf.data_ptr()) % 256
        self.t = self.buf[off: off + self.nbytes]
        _check("sv_workspace_init",
               load().sv_workspace_init(_ptr(self.t), self.nbytes, _stream(stream)))
        # The zeroing must be complete before a call on any other stream uses it.
        torch.cuda.synchronize(self.t.device)

    def status(self, stream=None, clear=False) -> int:
        out = ctypes.c_int32(0)
        _check("sv_get_status", load().sv_get_status(_ptr(self.t), _stream(stream), int(clear),
                                                     ctypes.byref(out)))
        return int(out.value)


def sv_schedule(conf, tau, token_budget, ws: Workspace, out_len=None, stream=None):
    """Verify lengths [B] int32 from confidences [B,K] float32 (see specverify.h)."""
    conf = _dev(conf, "conf", torch.float32)
    B, K = conf.shape
    if out_len is None:
        out_len = torch.empty(B, dtype=torch.int32, device=conf.device)
    _dev(out_len, "out_len", torch.int32)
    _check("sv_schedule", load().sv_schedule(_ptr(conf), B, K, float(tau), int(token_budget),
                                             _ptr(out_len), _ptr(ws.t), ws.nbytes,
                                             _stream(stream)))
    return out_len


def sv_schedule_cal(conf, temps, load, tau, tau_min, tau_max, token_budget, ws: Workspace,
                    out_len=None, conf_cal=None, tau_out=None, stream=None):
    """sv_schedule on calibrated confidences, optionally with the load-aware threshold
    (see specverify.h). temps [K] float32 or None; load [4] float32 or None. Returns
    (out_len, conf_cal, tau_out); conf_cal [B,K] float32 and tau_out [1] float64 are
    allocated when not given."""
    conf = _dev(conf, "conf", torch.float32)
    B, K = conf.shape
    if temps is not None:
        _dev(temps, "temps", torch.float32)
    if load is not None:
        _dev(load, "load", torch.float32)
    if out_len is None:
        out_len = torch.empty(B, dtype=torch.int32, device=conf.device)
    if conf_cal is None:
        conf_cal = torch.empty(B, K, dtype=torch.float32, device=conf.device)
    if tau_out is None:
        tau_out = torch.empty(1, dtype=torch.float64, device=conf.device)
    _dev(out_len, "out_len", torch.int32)
    _dev(conf_cal, "conf_cal", torch.float32)
    _dev(tau_out, "tau_out", torch.float64)
    _check("sv_schedule_cal", load_lib().sv_schedule_cal(
        _ptr(conf), _ptr(temps), _ptr(load), float(tau), float(tau_min), float(tau_max), B, K,
        int(token_budget), _ptr(out_len), _ptr(conf_cal), _ptr(tau_out), _ptr(ws.t), ws.nbytes,
        _stream(stream)))
    return out_len, conf_cal, tau_out


def sv_schedule_curve(conf, temps, load, tau, tau_min, tau_max, curve, token_budget,
                      ws: Workspace, out_len=None, stream=None):
    """Schedule whose budget is chosen from a throughput curve (see specverify.h).
    curve: [2, n_pts] float32 (tokens, tokens/s). Returns (out_len, n [1] int32,
    goodput [1] float64)."""
    conf = _dev(conf, "conf", torch.float32)
    B, K = conf.shape
    curve = _dev(curve, "curve", torch.float32)
    if curve.dim() != 2 or curve.shape[0] != 2:
        raise ValueError("curve must be [2, n_pts]")
    if temps is not None:
        _dev(temps, "temps", torch.float32)
    if load is not None:
        _dev(load, "load", torch.float32)
    dev = conf.device
    if out_len is None:
        out_len = torch.empty(B, dtype=torch.int32, device=dev)
    n_out = torch.empty(1, dtype=torch.int32, device=dev)
    g_out = torch.empty(1, dtype=torch.float64, device=dev)
    _check("sv_schedule_curve", load_lib().sv_schedule_curve(
        _ptr(conf), _ptr(temps), _ptr(load), float(tau), float(tau_min), float(tau_max),
        _ptr(curve), curve.shape[1], B, K, int(token_budget), _ptr(out_len), None, None,
        _ptr(n_out), _ptr(g_out), _ptr(ws.t), ws.nbytes, _stream(stream)))
    return out_len, n_out, g_out


def sv_calib_stats_len(K: int) -> int:
    """Length (float64) of the calibration window buffer for K positions."""
    return int(load_lib().sv_calib_stats_len(int(K)))


def sv_calib_observe(conf_cal, verify_len, accepted, stats, stream=None):
    """Add one verification round to the window stats (float64, in place)."""
    conf_cal = _dev(conf_cal, "conf_cal", torch.float32)
    B, K = conf_cal.shape
    _dev(verify_len, "verify_len", torch.int32)
    _dev(accepted, "accepted", torch.int32)
    _dev(stats, "stats", torch.float64)
    if stats.numel() != sv_calib_stats_len(K):
        raise ValueError("stats has the wrong length")
    _check("sv_calib_observe", load_lib().sv_calib_observe(
        _ptr(conf_cal), _ptr(verify_len), _ptr(accepted), B, K, _ptr(stats), _stream(stream)))


def sv_calib_update(stats, temps, lr, temp_floor, ece=None, stream=None):
    """Close the window: update temps [K] float32 in place, write the ECE into ece [1]
    float64 (allocated when not given) and zero stats. Returns ece."""
    _dev(stats, "stats", torch.float64)
    _dev(temps, "temps", torch.float32)
    K = temps.numel()
    if stats.numel() != sv_calib_stats_len(K):
        raise ValueError("stats has the wrong length")
    if ece is None:
        ece = torch.empty(1, dtype=torch.float64, device=temps.device)
    _dev(ece, "ece", torch.float64)
    _check("sv_calib_update", load_lib().sv_calib_update(
        _ptr(stats), _ptr(temps), K, float(lr), float(temp_floor), _ptr(ece), _stream(stream)))
    return ece


def sv_markov_draft(logits, U, Vm, prev_tok, ws: Workspace, corrected=None, draft_tok=None,
                    keys=None, stream=None):
    """Markov logit-bias head + greedy drafting loop (see specverify.h). logits [B,K,V]
    bf16, U and Vm [V,r] bf16, prev_tok [B] int32. Returns (corrected [B,K,V] bf16,
    draft_tok [B,K] int32)."""
    logits = _dev(logits, "logits", torch.bfloat16)
    U = _dev(U, "U", torch.bfloat16)
    Vm = _dev(Vm, "Vm", torch.bfloat16)
    prev_tok = _dev(prev_tok, "prev_tok", torch.int32)
    B, K, V = logits.shape
    r = U.shape[1]
    if tuple(U.shape) != (V, r) or tuple(Vm.shape) != (V, r):
        raise ValueError("U and Vm must be [V, r]")
    dev = logits.device
    if corrected is None:
        corrected = torch.empty_like(logits)
    if draft_tok is None:
        draft_tok = torch.empty((B, K), dtype=torch.int32, device=dev)
    if keys is None:
        keys = torch.empty(max(1, B * K), dtype=torch.int64, device=dev)
    _dev(corrected, "corrected", torch.bfloat16)
    _dev(draft_tok, "draft_tok", torch.int32)
    _dev(keys, "keys", torch.int64)
    _check("sv_markov_draft", load_lib().sv_markov_draft(
        _ptr(logits), _ptr(U), _ptr(Vm), _ptr(prev_tok), B, K, V, r, _ptr(corrected),
        _ptr(draft_tok), _ptr(keys), _ptr(ws.t), ws.nbytes, _stream(stream)))
    return corrected, draft_tok


def _dtype_code(t):
    if t.dtype == torch.bfloat16:
        return SV_BF16
    if t.dtype == torch.float32:
        return SV_F32
    raise ValueError(f"logits must be bfloat16 or float32, got {t.dtype}")


def sv_verify(target, draft, draft_tok, verify_len, uniforms, temperature, ws: Workspace,
              out_tok=None, out_accepted=None, diag=False, accept_count=None,
              tested_count=None, stream=None):
    """Rejection-sampling verification (see specverify.h).

    target [B,K+1,V], draft [B,K,V] (bf16 or fp32; draft/uniforms may be None at T=0),
    draft_tok [B,K] int32, verify_len [B] int32, uniforms [B,K+1] float32.
    Returns (out_tok [B,K+1], out_accepted [B]) and, with diag=True, also (p, q) [B,K]
    and the near-tie flags [B] int32.
    """
    target = _dev(target, "target")
    B, K1, V = target.shape
    K = K1 - 1
    draft = _dev(draft, "draft", target.dtype)
    draft_tok = _dev(draft_tok, "draft_tok", torch.int32)
    verify_len = _dev(verify_len, "verify_len", torch.int32)
    uniforms = _dev(uniforms, "uniforms", torch.float32)
    dev = target.device
    if out_tok is None:
        out_tok = torch.empty((B, K + 1), dtype=torch.int32, device=dev)
    if out_accepted is None:
        out_accepted = torch.empty(B, dtype=torch.int32, device=dev)
    lib = load()
    if diag or accept_count is not None or tested_count is not None:
        p = torch.empty((B, K), dtype=torch.float32, device=dev) if diag else None
        q = torch.empty((B, K), dtype=torch.float32, device=dev) if diag else None
        flags = torch.empty(B, dtype=torch.int32, device=dev) if diag else None
        rc = lib.sv_verify_diag(_ptr(target), _ptr(draft), _dtype_code(target), _ptr(draft_tok),
                                _ptr(verify_len), _ptr(uniforms), B, K, V, float(temperature),
                                _ptr(out_tok), _ptr(out_accepted), _ptr(p), _ptr(q),
                                _ptr(accept_count), _ptr(tested_count), _ptr(flags), _ptr(ws.t),
                                ws.nbytes, _stream(stream))
        _check("sv_verify_diag", rc)
        return (out_tok, out_accepted, p, q, flags) if diag else (out_tok, out_accepted)
    rc = lib.sv_verify(_ptr(target), _ptr(draft), _dtype_code(target), _ptr(draft_tok),
                       _ptr(verify_len), _ptr(uniforms), B, K, V, float(temperature),
                       _ptr(out_tok), _ptr(out_accepted), _ptr(ws.t), ws.nbytes, _stream(stream))
    _check("sv_verify", rc)
    return out_tok, out_accepted


def set_wait_limit(cycles: int) -> int:
    """Bound (GPU clock cycles) on a verify or cache attention call's waits for other warps;
    cycles <= 0 restores the default. Returns the previous bound (a testing aid)."""
    return int(load().sv_set_wait_limit(int(cycles)))


def set_share_always(on: bool) -> bool:
    """Have sv_kv_attend_shared read every group's common tokens once, whether that is faster or
    not (a testing aid). Returns what was set before."""
    return bool(load().sv_set_share_always(int(bool(on))))


def sv_verify_tree(target, draft, parent, draft_tok, n_nodes, uniforms, temperature,
                   ws: Workspace, out_tok=None, out_accepted=None, out_path=None,
                   want_path=True, stream=None):
    """Tree (multi-candidate) verification (see specverify.h).

    target, draft [B,N,V] (bf16 or fp32; draft/uniforms may be None at T=0), parent and
    draft_tok [B,N] int32, n_nodes [B] int32, uniforms [B,N] float32. Any workspace works
    (only its status word is used). Returns (out_tok [B,N], out_accepted [B], out_path
    [B,N] or None).
    """
    target = _dev(target, "target")
    B, N, V = target.shape
    draft = _dev(draft, "draft", target.dtype)
    parent = _dev(parent, "parent", torch.int32)
    draft_tok = _dev(draft_tok, "draft_tok", torch.int32)
    n_nodes = _dev(n_nodes, "n_nodes", torch.int32)
    uniforms = _dev(uniforms, "uniforms", torch.float32)
    dev = target.device
    if out_tok is None:
        out_tok = torch.empty((B, N), dtype=torch.int32, device=dev)
    if out_accepted is None:
        out_accepted = torch.empty(B, dtype=torch.int32, device=dev)
    if out_path is None and want_path:
        out_path = torch.empty((B, N), dtype=torch.int32, device=dev)
    rc = load().sv_verify_tree(_ptr(target), _ptr(draft), _dtype_code(target), _ptr(parent),
                               _ptr(draft_tok), _ptr(n_nodes), _ptr(uniforms), B, N, V,
                               float(temperature), _ptr(out_tok), _ptr(out_accepted),
                               _ptr(out_path), _ptr(ws.t), ws.nbytes, _stream(stream))
    _check("sv_verify_tree", rc)
    return out_tok, out_accepted, out_path


class KVCache:
    """A paged 8-bit key/value cache (see specverify.h): k, v [layers, pages, heads, page,
    dim] float8_e4m3fn with k_scale, v_scale [layers, pages, heads] float32; table [batch,
    max_pages], n_pages, len [batch] and refs [pages] int32. Starts empty; the pools are
    not initialised. Holds the workspace of its calls."""

    def __init__(self, layers, pages, page, heads, dim, batch, max_pages, device=None,
                 stream=None):
        sizes = dict(layers=int(layers), pages=int(pages), page=int(page), heads=int(heads),
                     dim=int(dim), batch=int(batch), max_pages=int(max_pages))
        c = _CacheStruct(**sizes)
        self.nbytes = int(load().sv_kv_workspace_bytes(ctypes.byref(c)))
        if self.nbytes == 0 or any(x != _int32(x) for x in sizes.values()):
            raise ValueError("unsupported cache sizes " + ", ".join(
                f"{k}={v}" for k, v in sizes.items()))
        dev = torch.device(device or "cuda")
        i32 = dict(dtype=torch.int32, device=dev)
        pool = (c.layers, c.pages, c.heads, c.page, c.dim)
        self.k = torch.empty(pool, dtype=torch.float8_e4m3fn, device=dev)
        self.v = torch.empty(pool, dtype=torch.float8_e4m3fn, device=dev)
        self.k_scale = torch.ones(pool[:3], dtype=torch.float32, device=dev)
        self.v_scale = torch.ones(pool[:3], dtype=torch.float32, device=dev)
        self.table = torch.full((c.batch, c.max_pages), -1, **i32)
        self.n_pages = torch.zeros(c.batch, **i32)
        self.len = torch.zeros(c.batch, **i32)
        self.refs = torch.zeros(c.pages, **i32)
        for n in ("k", "v", "k_scale", "v_scale", "table", "n_pages", "len", "refs"):
            setattr(c, n, getattr(self, n).data_ptr())
        self.c, self.ref = c, ctypes.byref(c)
        self.buf = torch.empty(self.nbytes + 256, dtype=torch.uint8, device=dev)
        off = (-self.buf.data_ptr()) % 256
        self.t = self.buf[off: off + self.nbytes]
        self.index = self.t.get_device()
        with torch.cuda.device(self.index):
            _check("sv_workspace_init",
                   load().sv_workspace_init(_ptr(self.t), self.nbytes, _kv_stream(stream, self)))
        # Everything above must be complete before a call on any other stream uses it.
        torch.cuda.synchronize(self.t.device)

        self.ws = self.t.data_ptr()
        self.__dict__.update(sizes)  # layers, pages, page, heads, dim, batch, max_pages
        self.rows = (c.batch,)

    def status(self, stream=None, clear=False) -> int:
        _kv_stream(stream, self)
        return Workspace.status(self, stream, clear)


# The cache's calls are made for every layer of every step, so their marshalling is kept
# short: plain integers for pointers, the current stream without a Python object for it.
def _addr(t):
    return None if t is None else t.data_ptr()


def _int32(x):
    """An int argument of the C calls, where a larger one would wrap: the nearest that fits. (A
    window or a number of sinks that large takes in every position; a layer, length or size
    that large, and a negative one, is refused.)"""
    x = int(x)
    return x if -2147483648 <= x <= 2147483647 else (2147483647 if x > 0 else -2147483648)


# (torch's own shortcuts to the current stream's handle and device, 2 and 0.1 us faster than the
# public ways, which serve where they are missing.)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _kv_stream(stream, cache):
    """Handle of a call's stream. A call runs on the current device: that must be the cache's (or
    the rotary table's)."""
    if _current_device() != cache.index:
        raise ValueError(f"the {getattr(cache, 'what', 'cache')} is on {cache.t.device}, which is not the current device")
    if stream is None:
        return _raw_stream(cache.index)
    if stream.device.index != cache.index:
        raise ValueError(f"the {getattr(cache, 'what', 'cache')} is on {cache.t.device}, the stream on {stream.device}")
    return stream.cuda_stream


def _kv_made(stream, cache, *made):
    """Results that the binding allocated, on the current stream, and a call on another one
    writes: their memory is not handed out again before that stream is through with them."""
    if stream.cuda_stream != _raw_stream(cache.index):
        for t in made:
            if t is not None:
                t.record_stream(stream)


def _kv_on(t, name, cache, dtype):
    """A dense tensor of the type on the cache's device."""
    if t.get_device() != cache.index:
        raise ValueError(f"{name} must be on {cache.t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t


def _kv_src(t, name, cache, heads):
    """A [batch, T, heads, dim] tensor whose last two dimensions are dense: its shape, and
    the element strides of rows and tokens."""
    if t.get_device() != cache.index:
        raise ValueError(f"{name} must be on {cache.t.device}")
    shape, stride = t.shape, t.stride()
    if len(shape) != 4 or shape[0] != cache.batch or shape[3] != cache.dim or \
            (heads is not None and shape[2] != heads):
        raise ValueError(f"{name} must be [{cache.batch}, T, {heads or 'q_heads'}, {cache.dim}], "
                         f"got {list(shape)}")
    if stride[3] != 1 or (shape[2] > 1 and stride[2] != shape[3]):
        raise ValueError(f"{name}: heads and dim must be contiguous")
    # Strides of dimensions of one element are free in torch: use the dense ones.
    tok = stride[1] if shape[1] > 1 else shape[2] * shape[3]
    row = stride[0] if shape[0] > 1 else shape[1] * tok
    return shape, row, tok


def _kv_counts(t, name, cache):
    if t is not None:
        _kv_on(t, name, cache, torch.int32)
        if t.shape != cache.rows:
            raise ValueError(f"{name} must be [{cache.batch}]")
    return t


_KV_DTYPES = {torch.float32: SV_F32, torch.bfloat16: SV_BF16, torch.float16: SV_F16}


def _kv_dtype(t, name):
    code = _KV_DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be bfloat16, float16 or float32, got {t.dtype}")
    return code


def sv_kv_reserve(cache: KVCache, n_new, ok=None, stream=None):
    """Pages for n_new [batch] int32 more tokens per row (see specverify.h). ok [batch]
    int32, when given, receives 1 per row served. Returns ok."""
    _kv_counts(n_new, "n_new", cache)
    _kv_counts(ok, "ok", cache)
    _check("sv_kv_reserve", load().sv_kv_reserve(cache.ref, _addr(n_new), _addr(ok),
                                                 cache.ws, cache.nbytes, _kv_stream(stream, cache)))
    return ok


def sv_kv_append(cache: KVCache, layer, k, v, n_new=None, stream=None):
    """Write the new tokens' keys and values [batch, T, heads, dim] (bf16, fp16 or fp32;
    slices of a fused projection are fine) into one layer (see specverify.h)."""
    shape, k_row, k_tok = _kv_src(k, "k", cache, cache.heads)
    v_shape, v_row, v_tok = _kv_src(v, "v", cache, cache.heads)
    if shape != v_shape or k.dtype != v.dtype:
        raise ValueError("k and v must have one shape and dtype")
    _kv_counts(n_new, "n_new", cache)
    _check("sv_kv_append", load().sv_kv_append(
        cache.ref, _int32(layer), _addr(k), _addr(v), _kv_dtype(k, "k"), k_row, k_tok,
        v_row, v_tok, shape[1], _addr(n_new), cache.ws, cache.nbytes, _kv_stream(stream, cache)))


def sv_kv_read(cache: KVCache, start, T, count=None, layer=0, n_layers=None,
               dtype=torch.bfloat16, k_out=None, v_out=None, stream=None):
    """The cached values at positions start .. start + count - 1 of each row as numbers (see
    specverify.h). Returns (k, v) [n_layers, batch, T, heads, dim]."""
    c = cache.c
    _kv_counts(start, "start", cache)
    _kv_counts(count, "count", cache)
    if n_layers is None:
        n_layers = c.layers - int(layer)
    shape = (int(n_layers), c.batch, int(T), c.heads, c.dim)
    k_made = v_made = None
    if k_out is None:
        k_out = k_made = start.new_empty(shape, dtype=dtype)
    if v_out is None:
        v_out = v_made = start.new_empty(shape, dtype=dtype)
    for name, t in (("k_out", k_out), ("v_out", v_out)):
        _kv_on(t, name, cache, dtype)
        if tuple(t.shape) != shape:
            raise ValueError(f"{name} must be {list(shape)}")
    _check("sv_kv_read", load().sv_kv_read(
        cache.ref, _int32(layer), _int32(n_layers), _addr(start), _addr(count), _int32(T),
        _addr(k_out), _addr(v_out), _kv_dtype(k_out, "k_out"), cache.ws, cache.nbytes, _kv_stream(stream, cache)))
    if stream is not None:
        _kv_made(stream, cache, k_made, v_made)
    return k_out, v_out


def _kv_attend(name, cache, layer, q, n_new, parent, scale, window, sinks, out, lse, want_lse,
               stream, *share):
    shape, row, tok = _kv_src(q, "q", cache, None)
    T, heads = shape[1], shape[2]
    _kv_counts(n_new, "n_new", cache)
    if parent is not None:
        _kv_on(parent, "parent", cache, torch.int32)
        if parent.shape != shape[:2]:
            raise ValueError(f"parent must be [{cache.batch}, {T}]")
    made = lse_made = None
    if out is None:
        out = made = q.new_empty(shape)
    elif _kv_on(out, "out", cache, q.dtype).shape != shape:
        raise ValueError("out must have q's shape")
    if lse is not None:
        if _kv_on(lse, "lse", cache, torch.float32).shape != shape[:3]:
            raise ValueError("lse must have q's first three dimensions")
    elif want_lse:
        lse = lse_made = q.new_empty(shape[:3], dtype=torch.float32)
    _check(name, getattr(load(), name)(
        cache.ref, _int32(layer), _addr(q), _kv_dtype(q, "q"), row, tok, T, heads, _addr(n_new),
        _addr(parent), float(cache.dim ** -0.5 if scale is None else scale), _int32(window),
        _int32(sinks),
        _addr(out), _addr(lse), *share, cache.ws, cache.nbytes, _kv_stream(stream, cache)))
    if stream is not None:
        _kv_made(stream, cache, made, lse_made)
    return out if lse is None else (out, lse)


def sv_kv_attend(cache: KVCache, layer, q, n_new=None, parent=None, scale=None, window=0,
                 sinks=0, out=None, lse=None, want_lse=False, stream=None):
    """Attention of the new tokens' queries [batch, T, q_heads, dim] (bf16 or fp16) over one
    layer of the cache (see specverify.h); scale defaults to dim ** -0.5. Returns out, or
    (out, lse) when lse is given or wanted."""
    return _kv_attend("sv_kv_attend", cache, layer, q, n_new, parent, scale, window, sinks, out,
                      lse, want_lse, stream)


class KVShare:
    """Which rows of a cache hold the same pages (none at first), and room for the parts of
    results of sv_kv_attend_shared with up to T tokens of q_heads query heads (see
    specverify.h)."""

    def __init__(self, cache: KVCache, T, q_heads, stream=None):
        self.nbytes = int(load().sv_kv_share_bytes(cache.ref, _int32(T), _int32(q_heads)))
        if self.nbytes == 0:
            raise ValueError(f"unsupported sizes T={T}, q_heads={q_heads}")
        self.buf = torch.empty(self.nbytes + 256, dtype=torch.uint8, device=cache.t.device)
        off = (-self.buf.data_ptr()) % 256
        self.t = self.buf[off: off + self.nbytes]
        self.ptr, self.index, self.cache = self.t.data_ptr(), cache.index, cache
        with torch.cuda.device(self.index):
            _check("sv_workspace_init",
                   load().sv_workspace_init(_ptr(self.t), self.nbytes, _kv_stream(stream, cache)))
        # The zeroing must be complete before a call on any other stream uses it.
        torch.cuda.synchronize(self.t.device)


def _kv_share_of(share, cache):
    if share.cache is not cache:
        raise ValueError("share belongs to another cache")
    return share.ptr, share.nbytes


def sv_kv_share(cache: KVCache, share: KVShare, group=None, stream=None):
    """Find the tokens that rows have in common: rows with the same number in group [batch] int32
    (-1: alone), or whose first page is the same (see specverify.h). Until rows are forked, freed
    or shortened, for every layer."""
    _kv_counts(group, "group", cache)
    _check("sv_kv_share", load().sv_kv_share(
        cache.ref, _addr(group), *_kv_share_of(share, cache), cache.ws, cache.nbytes,
        _kv_stream(stream, cache)))


def sv_kv_attend_shared(cache: KVCache, layer, q, share: KVShare, n_new=None, parent=None,
                        scale=None, window=0, sinks=0, out=None, lse=None, want_lse=False,
                        stream=None):
    """sv_kv_attend that reads the tokens which rows have in common (sv_kv_share) once for all of
    them, where that is faster than one by one (where it never is, sv_kv_attend is, by 2 to 11 us)."""
    return _kv_attend("sv_kv_attend_shared", cache, layer, q, n_new, parent, scale, window, sinks,
                      out, lse, want_lse, stream, *_kv_share_of(share, cache))


def sv_kv_commit(cache: KVCache, accepted, N, path=None, stream=None):
    """Keep the accepted part of the last block of N positions and release the pages past
    it (see specverify.h): accepted [batch] int32 and path [batch, N] int32 are what
    sv_verify and sv_verify_tree return."""
    _kv_counts(accepted, "accepted", cache)
    if path is not None:
        _kv_on(path, "path", cache, torch.int32)
        if path.shape != (cache.batch, int(N)):
            raise ValueError(f"path must be [{cache.batch}, {int(N)}]")
    _check("sv_kv_commit", load().sv_kv_commit(
        cache.ref, _addr(accepted), _addr(path), _int32(N), cache.ws, cache.nbytes,
        _kv_stream(stream, cache)))


def sv_kv_fork(cache: KVCache, src, ok=None, stream=None):
    """Row b becomes what row src[b] was, -1 frees it (see specverify.h): beams, samples,
    finished requests. ok [batch] int32, when given, receives 1 per row served. Returns
    ok."""
    _kv_counts(src, "src", cache)
    _kv_counts(ok, "ok", cache)
    _check("sv_kv_fork", load().sv_kv_fork(cache.ref, _addr(src), _addr(ok),
                                           cache.ws, cache.nbytes, _kv_stream(stream, cache)))
    return ok


# ---------------------------------------------------------------------------------------
# Rotary positions.
_SCALINGS = {"none": 0, "linear": 1, "turns": 2, "index": 3}


class Rope:
    """Rotary frequencies on a device (see specverify.h): rot / 2 of them from base and scaling
    ("none", "linear", "turns" or "index", with stretch and, for the last two, original, low and
    high), or from `angles` (radians per position); interleaved pairs or halves; the gain of
    cosine and sine. Holds the status word of sv_rope's calls."""

    what = "rotary table"

    def __init__(self, rot, base=10000.0, interleaved=False, scaling="none", stretch=1.0,
                 original=0.0, low=1.0, high=32.0, gain=1.0, angles=None, device=None):
        rot = int(rot)
        if scaling not in _SCALINGS:
            raise ValueError(f"scaling must be one of {', '.join(_SCALINGS)}, got {scaling!r}")
        if rot < 2 or rot % 2 or rot > 512:
            raise ValueError(f"rot must be even, from 2 to 512, got {rot}")
        if not abs(float(gain)) <= 3.4028234663852886e38:
            raise ValueError(f"gain must be finite, got {gain}")
        freq = (ctypes.c_int64 * (rot // 2))()
        if angles is not None:
            if len(angles) != rot // 2:
                raise ValueError(f"angles must be {rot // 2} numbers")
            _check("sv_rope_fixed", load().sv_rope_fixed(
                (ctypes.c_double * len(freq))(*(float(x) for x in angles)), len(freq), freq))
        else:
            _check("sv_rope_freqs", load().sv_rope_freqs(
                rot, float(base), _SCALINGS[scaling], float(stretch), float(original), float(low),
                float(high), freq))
        dev = torch.device(device or "cuda")
        self.freq = torch.tensor(list(freq), dtype=torch.int64).to(dev)
        self.buf = torch.zeros(512, dtype=torch.uint8, device=dev)
        off = (-self.buf.data_ptr()) % 256
        self.t = self.buf[off: off + 256]
        self.rot, self.index, self.nbytes = rot, self.t.get_device(), 256
        self.c = _RopeStruct(self.freq.data_ptr(), rot, int(bool(interleaved)), float(gain))
        self.ref, self.ws = ctypes.byref(self.c), self.t.data_ptr()
        # Everything above must be complete before a call on any other stream uses it.
        torch.cuda.synchronize(self.t.device)

    def status(self, stream=None, clear=False) -> int:
        _kv_stream(stream, self)
        return Workspace.status(self, stream, clear)


def _rope_src(t, name, index, like=None):
    """Shape of a [batch, T, heads, dim] tensor whose last two dimensions are dense, and the
    element strides of its rows and tokens."""
    if t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}")
    shape = t.shape
    if len(shape) != 4 or (like is not None and (shape != like.shape or t.dtype != like.dtype)):
        raise ValueError(f"{name} must be [batch, T, heads, dim]" if like is None else
                         f"{name} must be {list(like.shape)} of {like.dtype}")
    row, tok, head, one = t.stride()
    B, T, heads, dim = shape
    if one != 1 or (heads > 1 and head != dim):
        raise ValueError(f"{name}: heads and dim must be contiguous")
    # Strides of dimensions of one element are free in torch: use the dense ones.
    if T <= 1:
        tok = heads * dim
    return shape, (row if B > 1 else T * tok), tok


def _rope_ints(t, name, index, shape):
    """The address of a dense int32 tensor of the shape."""
    if t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}")
    if t.dtype != torch.int32 or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous torch.int32 {list(shape)}")
    return t.data_ptr()


def sv_rope(rope: Rope, x, pos=None, start=None, parent=None, n_new=None, inverse=False, out=None,
            stream=None):
    """Rotate x [batch, T, heads, dim] (bf16, fp16 or fp32; slices of a fused projection are
    fine) by positions pos [batch, T], or start [batch] (0 when not given) plus a token's
    number or depth in parent [batch, T] (all int32; see specverify.h). out may be x; inverse
    is the gradient's rotation. Returns out, with its graph where x requires grad (then not
    with out): the backward pass rotates back by pos, start, parent and n_new as they are then."""
    if x.requires_grad and torch.is_grad_enabled():
        if out is not None:
            raise ValueError("out: x requires grad, which a result written to out does not pass on")
        return _RopeGrad.apply(x, rope, pos, start, parent, n_new, inverse, stream)
    index = rope.index
    shape, row, tok = _rope_src(x, "x", index)
    B, T, heads, dim = shape
    made = None
    if out is None:
        out = made = x.new_empty(shape)
        out_tok = heads * dim
        out_row = T * out_tok
    else:
        _, out_row, out_tok = _rope_src(out, "out", index, x)
    code = load().sv_rope(
        rope.ref, x.data_ptr(), _kv_dtype(x, "x"), row, tok, B, _int32(T), _int32(heads), _int32(dim),
        None if pos is None else _rope_ints(pos, "pos", index, shape[:2]),
        None if start is None else _rope_ints(start, "start", index, shape[:1]),
        None if parent is None else _rope_ints(parent, "parent", index, shape[:2]),
        None if n_new is None else _rope_ints(n_new, "n_new", index, shape[:1]),
        1 if inverse else 0, out.data_ptr(), out_row, out_tok, rope.ws, 256, _kv_stream(stream, rope))
    if code != SV_OK:
        raise SpecVerifyError("sv_rope", code)
    if stream is not None:
        _kv_made(stream, rope, made)
    return out


class _RopeGrad(torch.autograd.Function):
    """sv_rope in a graph: a rotation is orthogonal up to its gain, so its gradient is the inverse one
    (which is linear too: gradients of gradients are the same calls)."""

    @staticmethod
    def forward(ctx, x, rope, pos, start, parent, n_new, inverse, stream):
        ctx.rope, ctx.inverse = rope, inverse
        ctx.save_for_backward(pos, start, parent, n_new)
        return sv_rope(rope, x, pos, start, parent, n_new, inverse, stream=stream)

    @staticmethod
    def backward(ctx, g):
        pos, start, parent, n_new = ctx.saved_tensors
        g = g.contiguous()
        if g.data_ptr() % 16:
            g = g.clone()
        return (sv_rope(ctx.rope, g, pos, start, parent, n_new, not ctx.inverse),) + (None,) * 7


def sv_kv_append_rope(cache: KVCache, layer, k, v, rope: Rope, q=None, q_out=None, n_new=None,
                      parent=None, stream=None):
    """sv_kv_append with the keys rotated on the way by their positions in the row (a token's
    depth when parent [batch, T] gives a tree), and the queries q [batch, T, q_heads, dim], if
    given, rotated to q_out (which may be q; see specverify.h). Returns q_out. (No graph is made, as
    by all calls of the cache.)"""
    shape, k_row, k_tok = _kv_src(k, "k", cache, cache.heads)
    v_shape, v_row, v_tok = _kv_src(v, "v", cache, cache.heads)
    if shape != v_shape or k.dtype != v.dtype:
        raise ValueError("k and v must have one shape and dtype")
    if rope.index != cache.index:
        raise ValueError(f"the rotary table must be on {cache.t.device}")
    _kv_counts(n_new, "n_new", cache)
    if parent is not None:
        _kv_on(parent, "parent", cache, torch.int32)
        if parent.shape != shape[:2]:
            raise ValueError(f"parent must be [{cache.batch}, {shape[1]}]")
    q_row = q_tok = out_row = out_tok = heads = 0
    made = None
    if q is not None:
        q_shape, q_row, q_tok = _kv_src(q, "q", cache, None)
        if q_shape[1] != shape[1] or q.dtype != k.dtype:
            raise ValueError("q must have k's tokens and dtype")
        heads = q_shape[2]
        if q_out is None:
            q_out = made = q.new_empty(q_shape)
            out_tok = heads * cache.dim
            out_row = shape[1] * out_tok
        else:
            _, out_row, out_tok = _rope_src(q_out, "q_out", cache.index, q)
    elif q_out is not None:
        raise ValueError("q_out without q")
    _check("sv_kv_append_rope", load().sv_kv_append_rope(
        cache.ref, _int32(layer), _addr(k), _addr(v), _kv_dtype(k, "k"), k_row, k_tok, v_row, v_tok,
        shape[1], _addr(n_new), _addr(parent), rope.ref, _addr(q), q_row, q_tok, heads, _addr(q_out),
        out_row, out_tok, cache.ws, cache.nbytes, _kv_stream(stream, cache)))
    if stream is not None:
        _kv_made(stream, cache, made)
    return q_out
