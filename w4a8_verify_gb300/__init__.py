"""Python binding of ``libw4a8.so`` (the sm_103a library declared in include/w4a8.h).

Argument marshalling only: every function forwards torch tensors' device pointers
and the current CUDA stream to the C ABI function of the same name and raises on a
non-zero status.  The library must be built (``__graft_entry__.build()``); there is
no fallback path.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libw4a8.so")

_lib = None

_c = ctypes
_vp, _i32, _u64, _sz, _f32, _i64 = _c.c_void_p, _c.c_int, _c.c_uint64, _c.c_size_t, _c.c_float, _c.c_int64
_u16, _u32, _dbl = _c.c_uint16, _c.c_uint32, _c.c_double


class ModelDesc(_c.Structure):
    _fields_ = [("n_layers", _i32), ("hidden", _i32), ("n_heads", _i32), ("n_kv_heads", _i32), ("head_dim", _i32),
                ("ffn", _i32), ("vocab", _i32), ("tied", _i32), ("rms_eps", _f32), ("rope_base", _f32)]


class SessionDesc(_c.Structure):
    _fields_ = [("kv_cap", _i32), ("ctx_cap", _i32), ("max_window", _i32), ("eos_id", _i32), ("mem_cap", _i32)]


class Ctl(_c.Structure):
    _fields_ = [("committed_len", _u32), ("ctx_len", _u32), ("n_valid", _u32), ("root_tok", _i32),
                ("n_generated", _u32), ("max_new", _u32), ("flags", _u32), ("step_idx", _u32)]


class Ctl16(_c.Structure):
    _fields_ = [("committed_len", _u32), ("n_generated", _u32), ("flags", _u32), ("root_tok", _i32)]


class StepStats(_c.Structure):
    _fields_ = [("n_accepted_drafts", _u16), ("best_match_len", _u16), ("n_nodes", _u16), ("n_emitted", _u16),
                ("t_lo", _u32)]


class DecodeOpts(_c.Structure):
    _fields_ = [("max_new", _i32), ("window", _i32), ("fixed_width", _i32), ("in_flight", _i32),
                ("timeout_us", _i64), ("n_widths", _i32), ("widths", _i32 * 8), ("t_us", _f32 * 8)]


class DecodeReport(_c.Structure):
    _fields_ = [("n_tokens", _i32), ("n_steps", _i32), ("n_windows", _i32), ("host_syncs", _i32),
                ("accepted_drafts", _i32), ("width_steps", _i32 * 17), ("flags", _u32), ("device_us", _dbl),
                ("kernels", _i64)]


class KV8CacheDesc(_c.Structure):
    _fields_ = [("n_seqs", _i32), ("n_kv_heads", _i32), ("head_dim", _i32), ("max_pages", _i32), ("codes", _vp),
                ("scales", _vp), ("sums", _vp), ("tail", _vp), ("table", _vp), ("len", _vp), ("ctl", _vp)]


class Rows(_c.Structure):
    _fields_ = [("data", _vp), ("seq", _i64), ("row", _i64), ("head", _i64)]


class KV8Attn(_c.Structure):
    _fields_ = [("n", _i32), ("n_heads", _i32), ("dtype", _i32), ("scale", _f32), ("q", Rows), ("out", Rows),
                ("k", Rows), ("v", Rows), ("counts", _vp), ("mask", _vp), ("pages", _vp), ("top_k", _i32),
                ("mass", _vp), ("mass_out", _vp)]


class KV4CacheDesc(_c.Structure):
    _fields_ = [("n_seqs", _i32), ("n_kv_heads", _i32), ("head_dim", _i32), ("max_pages", _i32), ("n_pages", _i32),
                ("pages", _vp), ("table", _vp), ("len", _vp), ("ctl", _vp)]


class KV4Attn(_c.Structure):
    _fields_ = [("n", _i32), ("n_heads", _i32), ("dtype", _i32), ("scale", _f32), ("q", Rows), ("out", Rows),
                ("k", Rows), ("v", Rows), ("counts", _vp), ("mask", _vp)]


class QKRotaryArgs(_c.Structure):
    _fields_ = [("n_seqs", _i32), ("n", _i32), ("n_heads", _i32), ("n_kv_heads", _i32), ("head_dim", _i32),
                ("rot_dim", _i32), ("n_axes", _i32), ("neighbours", _i32), ("dtype", _i32), ("norm", _i32),
                ("eps", _f32), ("factor", _f32), ("turns", _vp), ("axis", _vp), ("pos", _vp), ("start", _vp),
                ("counts", _vp), ("q_gain", _vp), ("k_gain", _vp), ("q", Rows), ("q_out", Rows), ("k", Rows),
                ("k_out", Rows)]


KV4_TICKETS = 16384  # bytes of an attention workspace that are zero between calls
FLAG_TERMINATED, FLAG_ERR_CAPACITY, FLAG_ERR_TOKEN, FLAG_ERR_TREE, FLAG_ERR_TIMEOUT = 1, 2, 4, 8, 16
T_Q, T_K, T_V, T_O, T_GATE, T_UP, T_DOWN, T_EMBED, T_LM_HEAD = range(9)

# name -> argtypes (restype int = w4a8_status unless listed in _RESTYPE)
_SIGNATURES = {
    "w4a8_status_str": [_i32],
    "w4a8_abi_version": [],
    "w4a8_pack_weights": [_vp, _i32, _i32, _vp],
    "w4a8_quantize_weights": [_vp, _i32, _i32, _vp, _vp, _vp],
    "w4a8_weight_layout_bytes": [_i32, _i32, _c.POINTER(_sz), _c.POINTER(_sz)],
    "w4a8_repack_weights": [_vp, _vp, _i32, _i32, _vp, _vp, _vp],
    "w4a8_quantize_rows": [_vp, _i32, _i32, _i32, _vp, _vp, _vp],
    "w4a8_matmul_workspace_bytes": [_i32, _i32, _i32, _c.POINTER(_sz)],
    "w4a8_matmul": [_vp, _vp, _i32, _i32, _vp, _vp, _i32, _vp, _vp, _sz, _vp],
    "w4a8_matmul_slices": [_i32, _i32],
    "w4a8_matmul_inject_timeout": [_vp, _vp, _i32, _i32, _vp, _vp, _i32, _vp, _vp, _sz, _vp],
    "w4a8_matmul_nondet": [_vp, _vp, _i32, _i32, _vp, _vp, _i32, _vp, _vp, _sz, _vp],
    "w4a8_matmul_per32": [_vp, _vp, _i32, _i32, _vp, _vp, _i32, _vp, _vp, _sz, _vp],
    "w4a8_matmul_check": [_vp, _i32, _i32, _i32, _c.POINTER(_c.c_uint32)],
    "w4a8_matmul_noalloc": [_vp, _vp, _i32, _i32, _vp, _vp, _i32, _vp, _vp],
    "w4a8_matmul_noalloc_check": [_c.POINTER(_c.c_uint32)],
    "w4a8_kv8_bytes": [_c.POINTER(KV8CacheDesc), _c.POINTER(_sz)],
    "w4a8_kv8_reset": [_c.POINTER(KV8CacheDesc), _vp],
    "w4a8_kv8_check": [_c.POINTER(KV8CacheDesc), _c.POINTER(_c.c_uint32)],
    "w4a8_kv8_append": [_c.POINTER(KV8CacheDesc), _vp, _vp, _i32, _i32, _i32, _vp, _vp, _vp,
                        _vp],
    "w4a8_kv8_read": [_c.POINTER(KV8CacheDesc), _vp, _vp, _i32, _vp, _vp, _vp],
    "w4a8_kv8_attention_workspace_bytes": [_c.POINTER(KV8CacheDesc), _vp, _c.POINTER(_sz)],
    "w4a8_kv8_attention": [_c.POINTER(KV8CacheDesc), _vp, _vp, _sz, _vp],
    "w4a8_kv8_attention_inject_timeout": [_c.POINTER(KV8CacheDesc), _vp, _vp, _sz, _i32, _vp],
    "w4a8_kv8_select_workspace_bytes": [_c.POINTER(KV8CacheDesc), _vp, _c.POINTER(_sz)],
    "w4a8_kv8_select": [_c.POINTER(KV8CacheDesc), _vp, _i32, _i32, _i32, _vp, _vp, _sz, _vp],
    "w4a8_kv8_evict": [_c.POINTER(KV8CacheDesc), _vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp],
    "w4a8_kv4_bytes": [_c.POINTER(KV4CacheDesc), _c.POINTER(_sz)],
    "w4a8_kv4_reset": [_c.POINTER(KV4CacheDesc), _vp],
    "w4a8_kv4_check": [_c.POINTER(KV4CacheDesc), _c.POINTER(_c.c_uint32)],
    "w4a8_kv4_append": [_c.POINTER(KV4CacheDesc), _vp, _vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp],
    "w4a8_kv4_read": [_c.POINTER(KV4CacheDesc), _vp, _vp, _i32, _i32, _vp, _vp, _vp],
    "w4a8_kv4_attention_workspace_bytes": [_c.POINTER(KV4CacheDesc), _vp, _c.POINTER(_sz)],
    "w4a8_kv4_attention": [_c.POINTER(KV4CacheDesc), _vp, _vp, _sz, _vp],
    "w4a8_kv4_attention_inject_timeout": [_c.POINTER(KV4CacheDesc), _vp, _vp, _sz, _i32, _vp],
    "w4a8_rotary_turns": [_vp, _i32, _vp],
    "w4a8_qk_rotary": [_vp, _vp],
    "w4a8_model_create": [_c.POINTER(ModelDesc), _c.POINTER(_vp)],
    "w4a8_model_load_tensor": [_vp, _i32, _i32, _vp, _vp, _vp],
    "w4a8_model_weight_bytes": [_vp, _c.POINTER(_sz)],
    "w4a8_model_destroy": [_vp],
    "w4a8_session_create": [_vp, _c.POINTER(SessionDesc), _c.POINTER(_vp)],
    "w4a8_session_destroy": [_vp],
    "w4a8_prefill": [_vp, _vp, _i32, _i32, _vp],
    "tree_verify_step": [_vp, _i32, _vp, _vp],
    "w4a8_model_trace_bytes": [_vp, _i32, _c.POINTER(_sz)],
    "w4a8_tree_verify_trace": [_vp, _i32, _vp, _vp, _sz, _vp],
    "accept_greedy": [_vp, _i32, _vp],
    "kv_compact": [_vp, _vp],
    "ngram_draft": [_vp, _vp],
    "w4a8_spec_step": [_vp, _i32, _vp],
    "spec_window": [_vp, _i32, _i32, _vp],
    "spec_poll": [_vp, _c.POINTER(Ctl16), _c.POINTER(StepStats), _c.POINTER(_i32), _c.POINTER(_i32),
                  _c.POINTER(_i32), _i64],
    "w4a8_calibrate": [_vp, _c.POINTER(_i32), _i32, _i32, _i32, _c.POINTER(_f32)],
    "w4a8_decode": [_vp, _c.POINTER(_i32), _i32, _c.POINTER(DecodeOpts), _c.POINTER(_i32), _c.POINTER(_i32),
                    _c.POINTER(DecodeReport), _vp],
    "w4a8_generate": [_vp, _c.POINTER(DecodeOpts), _c.POINTER(_i32), _c.POINTER(_i32), _c.POINTER(DecodeReport),
                      _vp],
    "w4a8_time_matmuls": [_vp, _i32, _i32, _c.POINTER(_dbl), _c.POINTER(_dbl), _c.POINTER(_i32)],
    "w4a8_session_get_ctl": [_vp, _c.POINTER(Ctl)],
    "w4a8_session_raise_flags": [_vp, _u32, _vp],
    "w4a8_session_set_tree": [_vp, _c.POINTER(_i32), _c.POINTER(_i32), _i32],
    "w4a8_session_get_tree": [_vp, _c.POINTER(_i32), _c.POINTER(_i32), _c.POINTER(_i32), _c.POINTER(_i32),
                              _c.POINTER(_i32)],
    "w4a8_session_get_pred": [_vp, _c.POINTER(_i32), _i32],
    "w4a8_session_get_context": [_vp, _c.POINTER(_i32), _i32, _c.POINTER(_i32)],
    "w4a8_session_copy_kv": [_vp, _i32, _i32, _i32, _vp, _vp, _vp],
    "w4a8_session_load_kv": [_vp, _i32, _i32, _i32, _vp, _vp, _vp],
    "w4a8_session_attention": [_vp, _i32, _i32, _vp, _vp, _vp],
    "w4a8_session_memory_append": [_vp, _c.POINTER(_i32), _i32],
    "w4a8_session_memory_clear": [_vp],
    "w4a8_session_memory_get": [_vp, _c.POINTER(_i32), _i32, _c.POINTER(_i32)],
    "w4a8_controller_create": [_c.POINTER(_i32), _c.POINTER(_f32), _i32, _c.POINTER(_vp)],
    "w4a8_controller_destroy": [_vp],
    "w4a8_controller_choose": [_vp],
    "w4a8_controller_observe": [_vp, _i32, _c.POINTER(StepStats), _i32, _dbl],
    "w4a8_controller_expected_tokens": [_vp, _i32],
    "w4a8_controller_cost": [_vp, _i32],
}
_RESTYPE = {"w4a8_status_str": _c.c_char_p, "w4a8_model_destroy": None, "w4a8_session_destroy": None,
            "w4a8_controller_destroy": None, "w4a8_controller_expected_tokens": _dbl, "w4a8_controller_cost": _dbl}


class W4A8Error(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__("%s failed: %s (status %d)" % (fn, status_str(status), status))


def lib():
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libw4a8.so not found at %s: run __graft_entry__.build()" % LIB_PATH)
        L = _c.CDLL(LIB_PATH)
        for name, args in _SIGNATURES.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = _RESTYPE.get(name, _c.c_int)
        _lib = L
    return _lib


def declared_symbols():
    return list(_SIGNATURES)


def status_str(s: int) -> str:
    return lib().w4a8_status_str(int(s)).decode()


def _call(name, *args):
    st = getattr(lib(), name)(*args)
    if st != 0:
        raise W4A8Error(name, st)
    return st


def _ptr(t):
    return None if t is None else _c.c_void_p(t.data_ptr())


def _stream(stream=None):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return _c.c_void_p(s.cuda_stream)


# ----------------------------------------------------------------------------- weights

def w4a8_pack_weights(q):
    """int8 codes (host numpy [N][K]) -> packed u32 words (host numpy [N][K/8])."""
    import numpy as np
    q = np.ascontiguousarray(q, dtype=np.int8)
    N, K = q.shape
    out = np.empty((N, K // 8), dtype=np.uint32)
    _call("w4a8_pack_weights", q.ctypes.data_as(_vp), N, K, out.ctypes.data_as(_vp))
    return out


def w4a8_quantize_weights(w, w_p2=None, s_p2=None, stream=None):
    """fp32 device [N][K] -> (int32-viewed u32 words [N][K/8], int16-viewed fp16 scales [N][K/32])."""
    import torch
    N, K = w.shape
    if w_p2 is None:
        w_p2 = torch.empty((N, K // 8), dtype=torch.int32, device=w.device)
    if s_p2 is None:
        s_p2 = torch.empty((N, K // 32), dtype=torch.int16, device=w.device)
    _call("w4a8_quantize_weights", _ptr(w), N, K, _ptr(w_p2), _ptr(s_p2), _stream(stream))
    return w_p2, s_p2


def w4a8_weight_layout_bytes(N, K):
    wb, sb = _sz(), _sz()
    _call("w4a8_weight_layout_bytes", N, K, _c.byref(wb), _c.byref(sb))
    return wb.value, sb.value


def w4a8_repack_weights(w_p2, s_p2, N, K, stream=None):
    """P2 layout -> tiled layout (device tensors, int32 words / int16 scales)."""
    import torch
    wb, sb = w4a8_weight_layout_bytes(N, K)
    w_t = torch.empty(wb // 4, dtype=torch.int32, device=w_p2.device)
    s_t = torch.empty(sb // 2, dtype=torch.int16, device=w_p2.device)
    _call("w4a8_repack_weights", _ptr(w_p2), _ptr(s_p2), N, K, _ptr(w_t), _ptr(s_t), _stream(stream))
    return w_t, s_t


# ------------------------------------------------------------------------- activations

def w4a8_quantize_rows(x, mode=0, stream=None):
    import torch
    M, K = x.shape
    q = torch.empty((M, K), dtype=torch.int8, device=x.device)
    s = torch.empty((M,) if mode == 0 else (M, K // 32), dtype=torch.float32, device=x.device)
    _call("w4a8_quantize_rows", _ptr(x), M, K, int(mode), _ptr(q), _ptr(s), _stream(stream))
    return q, s


# ------------------------------------------------------------------------------ matmul

def w4a8_matmul_workspace_bytes(M, K, N):
    b = _sz()
    _call("w4a8_matmul_workspace_bytes", M, K, N, _c.byref(b))
    return b.value


def w4a8_matmul_slices(K, N):
    return lib().w4a8_matmul_slices(K, N)


def w4a8_matmul_check(workspace, M, K, N):
    """Device status word of a matmul workspace (0 = every bounded wait completed)."""
    f = _c.c_uint32()
    st = lib().w4a8_matmul_check(_ptr(workspace), M, K, N, _c.byref(f))
    if st not in (0, 7):
        raise W4A8Error("w4a8_matmul_check", st)
    return f.value


def w4a8_matmul_noalloc(a_q, a_s, w_t, s_t, N, y, stream=None):
    """w4a8_matmul with the library's own static scratch (no allocation; y is caller-owned)."""
    M, K = a_q.shape
    _call("w4a8_matmul_noalloc", _ptr(a_q), _ptr(a_s), M, K, _ptr(w_t), _ptr(s_t), N, _ptr(y), _stream(stream))
    return y


def w4a8_matmul_per32(a_q, a_s, w_t, s_t, N, y=None, workspace=None, stream=None):
    """W4A8 product with per-32 activation scales a_s [M][K/32] (w4a8_matmul_per32)."""
    import torch
    M, K = a_q.shape
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=a_q.device)
    need = w4a8_matmul_workspace_bytes(M, K, N)
    if workspace is None:
        workspace = torch.zeros(need, dtype=torch.uint8, device=a_q.device)
    _call("w4a8_matmul_per32", _ptr(a_q), _ptr(a_s), M, K, _ptr(w_t), _ptr(s_t), N, _ptr(y), _ptr(workspace),
          workspace.numel() * workspace.element_size(), _stream(stream))
    return y


def w4a8_matmul_nondet(a_q, a_s, w_t, s_t, N, y=None, workspace=None, stream=None):
    """The non-deterministic fast variant (slices combined with float atomics)."""
    import torch
    M, K = a_q.shape
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=a_q.device)
    need = w4a8_matmul_workspace_bytes(M, K, N)
    if workspace is None:
        workspace = torch.zeros(need, dtype=torch.uint8, device=a_q.device)
    _call("w4a8_matmul_nondet", _ptr(a_q), _ptr(a_s), M, K, _ptr(w_t), _ptr(s_t), N, _ptr(y), _ptr(workspace),
          workspace.numel() * workspace.element_size(), _stream(stream))
    return y


def w4a8_matmul_inject_timeout(a_q, a_s, w_t, s_t, N, y, workspace, stream=None):
    """Test-only: the matmul with a copy warp that issues nothing, so that its bounded waits
    expire and the workspace status word reports the timeout (w4a8_matmul_inject_timeout)."""
    M, K = a_q.shape
    _call("w4a8_matmul_inject_timeout", _ptr(a_q), _ptr(a_s), M, K, _ptr(w_t), _ptr(s_t), N, _ptr(y),
          _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))


def w4a8_matmul_noalloc_check():
    """Status word of the last w4a8_matmul_noalloc call on the current device (0 = every
    bounded wait completed; synchronous: call after that stream has finished)."""
    f = _c.c_uint32()
    st = lib().w4a8_matmul_noalloc_check(_c.byref(f))
    if st not in (0, 7):
        raise W4A8Error("w4a8_matmul_noalloc_check", st)
    return f.value


def w4a8_matmul(a_q, a_s, w_t, s_t, N, y=None, workspace=None, stream=None):
    import torch
    M, K = a_q.shape
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=a_q.device)
    need = w4a8_matmul_workspace_bytes(M, K, N)
    if workspace is None:
        workspace = torch.zeros(need, dtype=torch.uint8, device=a_q.device)
    _call("w4a8_matmul", _ptr(a_q), _ptr(a_s), M, K, _ptr(w_t), _ptr(s_t), N, _ptr(y), _ptr(workspace),
          workspace.numel() * workspace.element_size(), _stream(stream))
    return y


# ------------------------------------------------------------- key/value cache in 8 bits

class _PagedCache:
    """What the paged caches share: their tensors, checks of arguments, streams and workspaces."""

    _ROWS = struct.Struct("@4q")                         # w4a8_rows
    _NONE = (0, 0, 0, 0)

    def _adopt(self, names, shapes, device, tensors):
        """Takes the cache's tensors, or makes new ones."""
        import torch
        self._torch = torch
        self._types = {torch.float32: 0, torch.bfloat16: 1}
        self._name = type(self).__name__
        got = {}
        for (name, dtype), shape in zip(names, shapes):
            dtype = getattr(torch, dtype)
            t = got[name] = torch.empty(shape, dtype=dtype, device=device) if tensors is None else tensors[name]
            if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
                raise ValueError("%s: %s must be a contiguous %s tensor of shape %s" % (self._name, name, dtype, shape))
        self.tensors = got
        one = next(iter(got.values()))
        self.device = one.device
        self._dev = one.get_device()
        if self._dev < 0 or any(t.get_device() != self._dev for t in got.values()):
            raise ValueError("%s: the tensors must be on one CUDA device" % self._name)
        self._sizes, self._kept, self._lock, self._streams = {}, {}, threading.Lock(), set()
        return [t.data_ptr() for t in got.values()]

    @property
    def len(self):
        return self.tensors["len"]

    def _scratch(self, need):
        return self._torch.empty(need, dtype=self._torch.uint8, device=self.device)

    def _elsewhere(self, stream, method, args):
        """The call with ``stream`` as the current one; tensors of other streams are marked as in use on it."""
        torch = self._torch
        if stream.device != self.device:
            raise ValueError(self._name + ": the stream is on another device than the cache")
        with torch.cuda.stream(stream):
            result = method(*args)
        for t in args:
            if isinstance(t, torch.Tensor):
                t.record_stream(stream)
        if stream.cuda_stream not in self._streams:      # the cache's own: once for each stream
            self._streams.add(stream.cuda_stream)
            for t in self.tensors.values():
                t.record_stream(stream)
        return result

    def _run(self, fn, *args):
        """Calls fn(cache, *args, the current stream of the cache's device)."""
        torch = self._torch
        if torch.cuda.current_device() == self._dev:
            status = fn(self._ref, *args, torch._C._cuda_getCurrentRawStream(self._dev))
        else:
            with torch.cuda.device(self._dev):
                status = fn(self._ref, *args, torch._C._cuda_getCurrentRawStream(self._dev))
        if status:
            raise W4A8Error(fn.__name__, status)

    def _vec(self, t, name, dtype, shape):
        """Pointer of a contiguous tensor of this device, type and shape."""
        if t.dtype is not dtype or t.shape != shape or t.get_device() != self._dev or not t.is_contiguous():
            raise ValueError("%s: %s must be a contiguous %s tensor %s on the cache's device"
                             % (self._name, name, str(dtype)[6:], list(shape)))
        return t.data_ptr()

    def _rows(self, t, name, dtype, shape):
        """The fields of a w4a8_rows for t of that shape, [n_seqs][n][heads][head_dim]."""
        a, b, c, d = t.stride() if t.shape == shape else (0, 0, 0, 0)
        if d != 1 or t.dtype is not dtype or t.get_device() != self._dev:
            raise ValueError("%s: %s must be %s %s with unit stride in the last dimension, on the cache's device"
                             % (self._name, name, str(dtype)[6:], list(shape)))
        return t.data_ptr(), a, b, c

    def _query(self, q):
        """(fields, type number, n, heads) of a tensor of query rows."""
        S, D = self.shape[0], self.shape[2]
        shape, dtype = q.shape, q.dtype
        kind = self._types.get(dtype)
        if kind is None or len(shape) != 4 or shape[0] != S or shape[3] != D:
            raise ValueError("%s: q must be fp32 or bf16 [%d][n][heads][%d], not %s %s"
                             % (self._name, S, D, str(dtype)[6:], list(shape)))
        return self._rows(q, "q", dtype, shape), kind, shape[1], shape[2]

    def _launch(self, fn, size_fn, key, args, workspace, *more):
        """fn(cache, args, *more, workspace, its bytes, stream).  Without a workspace of the caller's: the one that the
        cache keeps for the current stream (calls on one stream run in order; the lock keeps the launches of two
        threads' calls apart), or a new one where that does not hold or would stay large: in a capture, whose graph may
        be replayed beside other work, with another device current, above 32 MB."""
        torch = self._torch
        if workspace is not None:
            if workspace.device != self.device or not workspace.is_contiguous():
                raise ValueError(self._name + ": the workspace must be contiguous, on the cache's device")
            return self._run(fn, args, *more, workspace.data_ptr(), workspace.numel() * workspace.element_size())
        need = self._sizes.get(key)
        if need is None:
            n = _sz()
            _call(size_fn, self._ref, args, _c.byref(n))
            need = self._sizes[key] = n.value
        if need > 32 << 20 or torch.cuda.current_device() != self._dev or torch._C._cuda_isCurrentStreamCapturing():
            workspace = self._scratch(need)
            return self._run(fn, args, *more, workspace.data_ptr(), need)
        stream = torch._C._cuda_getCurrentRawStream(self._dev)
        with self._lock:
            ptr, size, _ = self._kept.get(stream, (0, -1, None))
            if size < need:
                t = self._scratch(need)
                ptr, size, _ = self._kept[stream] = (t.data_ptr(), need, t)
            status = fn(self._ref, args, *more, ptr, size, stream)
        if status:
            raise W4A8Error(fn.__name__, status)


class KV8Cache(_PagedCache):
    """One layer of ``n_seqs`` sequences' keys and values in 8 bits (w4a8_kv8_cache).

    Holds the cache's tensors, by name in ``tensors`` (``codes``, ``scales``, ``sums``, ``tail``, ``table``,
    ``len``, ``ctl``: see include/w4a8.h): those given, or new ones of an empty cache.  ``q``, ``k``, ``v`` are
    fp32 or bf16 [n_seqs][n][heads][head_dim] with unit stride in the last dimension.  Asynchronous on the current
    stream of the cache's device, or on ``stream`` (outputs and workspaces are then allocated on it, and the memory of
    the call's tensors is not given to others before it is through with them; work of other streams on them is the
    caller's to order); device state that is out of range is reported by ``check``.

    A decode step is about ten microseconds on the device, so the calls are written out: arguments are marshalled as
    packed bytes (w4a8_kv8_attn, w4a8_rows); the workspace sizes of the shapes seen and one workspace for each
    stream are kept.
    """

    _NAMES = (("codes", "uint8"), ("scales", "float32"), ("sums", "int16"), ("tail", "float32"), ("table", "int32"),
              ("len", "int32"), ("ctl", "int32"))
    _ATTN = struct.Struct("@iiif 4q 4q 4q 4q 3q i 2q")   # w4a8_kv8_attn

    def __init__(self, n_seqs, n_kv_heads, head_dim, max_pages, device="cuda", tensors=None):
        S, H, D, P = self.shape = (n_seqs, n_kv_heads, head_dim, max_pages)
        self.desc = KV8CacheDesc(S, H, D, P)
        _call("w4a8_kv8_bytes", _c.byref(self.desc), (_sz * 7)())     # refuses dimensions out of range
        shapes = ((S, H, P, 2, 64 * D), (S, H, P, 2), (S, H, P, D), (S, H, 2, 64, D), (S, H, P), (S,), (1,))
        self.desc = KV8CacheDesc(S, H, D, P, *self._adopt(self._NAMES, shapes, device, tensors))
        self._ref = _c.byref(self.desc)
        L = lib()
        self._attention, self._select, self._evict = L.w4a8_kv8_attention, L.w4a8_kv8_select, L.w4a8_kv8_evict
        self._append, self._read = L.w4a8_kv8_append, L.w4a8_kv8_read
        if tensors is None:
            self.reset()

    def reset(self, stream=None):
        """Empties the cache (w4a8_kv8_reset)."""
        if stream is not None:
            return self._elsewhere(stream, self.reset, ())
        self._run(lib().w4a8_kv8_reset)

    def check(self, stream=None):
        """The status word (0 = every call's device state was in range); waits for the calls on the current stream of the
        cache's device, or on ``stream``."""
        if stream is not None:
            return self._elsewhere(stream, self.check, ())
        self._torch.cuda.current_stream(self.device).synchronize()
        f = _c.c_uint32()
        st = lib().w4a8_kv8_check(self._ref, _c.byref(f))
        if st not in (0, 7):
            raise W4A8Error("w4a8_kv8_check", st)
        return f.value

    def append(self, k, v, counts=None, index=None, len_out=None, stream=None):
        """Commits rows of k and v, advancing the cache's lengths, or storing the new ones in ``len_out`` instead
        (w4a8_kv8_append): a sequence that completes a page is then right at its new length alone.  ``index``
        [n_seqs][n]: the source row of each new position."""
        if stream is not None:
            return self._elsewhere(stream, self.append, (k, v, counts, index, len_out))
        S, H, D, _ = self.shape
        dtype, i32 = k.dtype, self._torch.int32
        kind = self._types.get(dtype)
        if kind is None or k.dim() != 4:
            raise ValueError("KV8Cache: k must be fp32 or bf16 [n_seqs][n][n_kv_heads][head_dim]")
        n_src = k.shape[1]
        shape = (S, n_src, H, D)
        kr = self._ROWS.pack(*self._rows(k, "k", dtype, shape))
        vr = self._ROWS.pack(*self._rows(v, "v", dtype, shape))
        n = n_src if index is None else index.shape[1]
        self._run(self._append, kr, vr, kind, n_src, n, 0 if counts is None else self._vec(counts, "counts", i32, (S,)),
                  0 if index is None else self._vec(index, "index", i32, (S, n)),
                  self.desc.len if len_out is None else self._vec(len_out, "len_out", i32, (S,)))

    def read(self, first, n, length=None, stream=None):
        """fp32 keys and values [n_seqs][n][n_kv_heads][head_dim] of positions first[s].. as held (w4a8_kv8_read)."""
        if stream is not None:
            return self._elsewhere(stream, self.read, (first, n, length))
        torch = self._torch
        S, H, D, _ = self.shape
        k = torch.empty((S, n, H, D), dtype=torch.float32, device=self.device)
        v = torch.empty_like(k)
        self._run(self._read, self._vec(first, "first", torch.int32, (S,)),
                  0 if length is None else self._vec(length, "length", torch.int32, (S,)), n, k.data_ptr(), v.data_ptr())
        return k, v

    def attention(self, q, k=None, v=None, scale=1.0, counts=None, mask=None, pages=None, mass=None, mass_out=None,
                  out=None, workspace=None, stream=None):
        """Attention of q's rows over the cache and the new rows k, v (w4a8_kv8_attention); returns ``out``, a new
        tensor if not given (its allocation is a third of a small call's time)."""
        if stream is not None:
            return self._elsewhere(stream, self.attention,
                                   (q, k, v, scale, counts, mask, pages, mass, mass_out, out, workspace))
        torch = self._torch
        S, H, D, P = self.shape
        qr, kind, n, heads = self._query(q)
        dtype = q.dtype
        if k is None and v is None:
            kr = vr = self._NONE
        elif k is None or v is None:
            raise ValueError("KV8Cache: k and v come together")
        else:
            kr, vr = self._rows(k, "k", dtype, (S, n, H, D)), self._rows(v, "v", dtype, (S, n, H, D))
        if out is None:
            out = torch.empty_like(q, memory_format=torch.contiguous_format)
            outr = (out.data_ptr(), n * heads * D, heads * D, D)
        else:
            outr = self._rows(out, "out", dtype, (S, n, heads, D))
        top_k = pp = mi = mo = 0
        if pages is not None:
            top_k = pages.shape[-1]
            pp = self._vec(pages, "pages", torch.int32, (S, n, H, top_k))
        if mass_out is not None:
            mi = 0 if mass is None else self._vec(mass, "mass", torch.float32, (S, H, P))
            mo = self._vec(mass_out, "mass_out", torch.float32, (S, H, P))
        elif mass is not None:
            raise ValueError("KV8Cache: mass needs mass_out")
        a = self._ATTN.pack(n, heads, kind, scale, *qr, *outr, *kr, *vr,
                            0 if counts is None else self._vec(counts, "counts", torch.int32, (S,)),
                            0 if mask is None else self._vec(mask, "mask", torch.int64, (S, n)), pp, top_k, mi, mo)
        self._launch(self._attention, "w4a8_kv8_attention_workspace_bytes",
                     (n, heads, kind, k is None, pages is None, top_k, mo == 0), a, workspace)
        return out

    def select(self, q, top_k, first_pages=0, last_pages=0, counts=None, out=None, workspace=None, stream=None):
        """The whole pages of best score for every row and KV head, int32 [n_seqs][n][n_kv_heads][top_k], ascending,
        -1 behind the last (w4a8_kv8_select)."""
        if stream is not None:
            return self._elsewhere(stream, self.select, (q, top_k, first_pages, last_pages, counts, out, workspace))
        torch = self._torch
        S, H = self.shape[:2]
        qr, kind, n, heads = self._query(q)
        if out is None:
            out = torch.empty((S, n, H, top_k), dtype=torch.int32, device=self.device)
            po = out.data_ptr()
        else:
            po = self._vec(out, "out", torch.int32, (S, n, H, top_k))
        none = self._NONE
        a = self._ATTN.pack(n, heads, kind, 1.0, *qr, *none, *none, *none,
                            0 if counts is None else self._vec(counts, "counts", torch.int32, (S,)), 0, 0, 0, 0, 0)
        self._launch(self._select, "w4a8_kv8_select_workspace_bytes", (n, heads, kind), a, workspace, top_k, first_pages,
                     last_pages, po)
        return out

    def evict(self, mass, keep, first_pages=0, last_pages=0, in_place=False, stream=None):
        """Keeps at most ``keep`` whole pages per KV head (w4a8_kv8_evict); returns (table, mass, len), new tensors,
        or the cache's own and ``mass`` itself when ``in_place``."""
        if stream is not None:
            return self._elsewhere(stream, self.evict, (mass, keep, first_pages, last_pages, in_place))
        torch = self._torch
        S, H, _, P = self.shape
        pm = self._vec(mass, "mass", torch.float32, (S, H, P))
        table, length = self.tensors["table"], self.tensors["len"]
        if not in_place:
            table, mass, length = torch.empty_like(table), torch.empty_like(mass), torch.empty_like(length)
        self._run(self._evict, pm, keep, first_pages, last_pages, table.data_ptr(), mass.data_ptr(), length.data_ptr())
        return table, mass, length


# ------------------------------------------------------------- key/value cache in 4 bits

class KV4Cache(_PagedCache):
    """One layer of ``n_seqs`` sequences' keys and values in 4 bits with a scale for every 32 dims, in a pool of ``n_pages``
    pages of 64 tokens (w4a8_kv4_cache); ``tensors["table"]`` [n_seqs][max_pages] names each sequence's pages, which
    sequences may share as long as no append writes to them.

    Holds the cache's tensors, by name in ``tensors`` (``pages``, ``table``, ``len``, ``ctl``: see include/w4a8.h): those given,
    or new ones of an empty cache, whose sequences own ``max_pages`` pages each where ``n_pages`` is not given.  ``q``, ``k``, ``v``
    are fp32 or bf16 [n_seqs][n][heads][head_dim] with unit stride in the last dimension.  Streams, workspaces and device
    state that is out of range: as KV8Cache.
    """

    _NAMES = (("pages", "uint8"), ("table", "int32"), ("len", "int32"), ("ctl", "int32"))
    _ATTN = struct.Struct("@iiif 4q 4q 4q 4q 2q")        # w4a8_kv4_attn

    def __init__(self, n_seqs, n_kv_heads, head_dim, max_pages, n_pages=None, device="cuda", tensors=None):
        if n_pages is None:
            n_pages = n_seqs * max_pages
        S, H, D, P, N = self.shape = (n_seqs, n_kv_heads, head_dim, max_pages, n_pages)
        self.desc = KV4CacheDesc(S, H, D, P, N)
        _call("w4a8_kv4_bytes", _c.byref(self.desc), (_sz * 4)())     # refuses dimensions out of range
        shapes = ((N, H, 68 * D), (S, P), (S,), (1,))
        self.desc = KV4CacheDesc(S, H, D, P, N, *self._adopt(self._NAMES, shapes, device, tensors))
        self._ref = _c.byref(self.desc)
        L = lib()
        self._attention, self._append, self._read = L.w4a8_kv4_attention, L.w4a8_kv4_append, L.w4a8_kv4_read
        if tensors is None:
            self.reset()

    def _scratch(self, need):
        t = super()._scratch(need)
        t[:KV4_TICKETS].zero_()
        return t

    def reset(self, stream=None):
        """Empties the cache: lengths 0, every sequence its own pages as far as the pool goes and no page (-1) behind that
        (w4a8_kv4_reset)."""
        if stream is not None:
            return self._elsewhere(stream, self.reset, ())
        self._run(lib().w4a8_kv4_reset)

    def check(self, stream=None):
        """The status word (0 = every call's device state was in range); waits for the calls on the current stream of the
        cache's device, or on ``stream``."""
        if stream is not None:
            return self._elsewhere(stream, self.check, ())
        self._torch.cuda.current_stream(self.device).synchronize()
        f = _c.c_uint32()
        st = lib().w4a8_kv4_check(self._ref, _c.byref(f))
        if st not in (0, 7):
            raise W4A8Error("w4a8_kv4_check", st)
        return f.value

    def append(self, k, v, counts=None, index=None, len_out=None, stream=None):
        """Commits rows of k and v, advancing the cache's lengths, or storing the new ones in ``len_out`` instead
        (w4a8_kv4_append).  ``index`` [n_seqs][n]: the source row of each new position."""
        if stream is not None:
            return self._elsewhere(stream, self.append, (k, v, counts, index, len_out))
        S, H, D = self.shape[:3]
        dtype, i32 = k.dtype, self._torch.int32
        kind = self._types.get(dtype)
        if kind is None or k.dim() != 4:
            raise ValueError("KV4Cache: k must be fp32 or bf16 [n_seqs][n][n_kv_heads][head_dim]")
        n_src = k.shape[1]
        shape = (S, n_src, H, D)
        kr = self._ROWS.pack(*self._rows(k, "k", dtype, shape))
        vr = self._ROWS.pack(*self._rows(v, "v", dtype, shape))
        n = n_src if index is None else index.shape[1]
        self._run(self._append, kr, vr, kind, n_src, n, 0 if counts is None else self._vec(counts, "counts", i32, (S,)),
                  0 if index is None else self._vec(index, "index", i32, (S, n)),
                  self.desc.len if len_out is None else self._vec(len_out, "len_out", i32, (S,)))

    def read(self, first, n, length=None, dtype=None, stream=None):
        """Keys and values [n_seqs][n][n_kv_heads][head_dim] of positions first[s].. as held, in fp32 or bf16 (exact in
        either; fp32 by default) (w4a8_kv4_read)."""
        if stream is not None:
            return self._elsewhere(stream, self.read, (first, n, length, dtype))
        torch = self._torch
        S, H, D = self.shape[:3]
        dtype = torch.float32 if dtype is None else dtype
        kind = self._types.get(dtype)
        if kind is None:
            raise ValueError("KV4Cache: dtype must be fp32 or bf16")
        k = torch.empty((S, n, H, D), dtype=dtype, device=self.device)
        v = torch.empty_like(k)
        self._run(self._read, self._vec(first, "first", torch.int32, (S,)),
                  0 if length is None else self._vec(length, "length", torch.int32, (S,)), n, kind, k.data_ptr(),
                  v.data_ptr())
        return k, v

    def attention(self, q, k=None, v=None, scale=1.0, counts=None, mask=None, out=None, workspace=None, stream=None):
        """Attention of q's rows over the cache and the new rows k, v (w4a8_kv4_attention); returns ``out``, a new tensor if
        not given, whose rows behind the counts and of sequences that are left out hold anything.  A ``workspace`` of the caller's needs no initialisation: its first KV4_TICKETS bytes are set to zero by the
        call (a small launch that the cache's own workspaces do without)."""
        if stream is not None:
            return self._elsewhere(stream, self.attention, (q, k, v, scale, counts, mask, out, workspace))
        if workspace is not None:
            if workspace.get_device() != self._dev or not workspace.is_contiguous():
                raise ValueError("KV4Cache: the workspace must be contiguous, on the cache's device")
            with self._torch.cuda.device(self._dev):
                workspace.view(-1).view(self._torch.uint8)[:KV4_TICKETS].zero_()
        torch = self._torch
        S, H, D = self.shape[:3]
        qr, kind, n, heads = self._query(q)
        dtype = q.dtype
        if k is None and v is None:
            kr = vr = self._NONE
        elif k is None or v is None:
            raise ValueError("KV4Cache: k and v come together")
        else:
            kr, vr = self._rows(k, "k", dtype, (S, n, H, D)), self._rows(v, "v", dtype, (S, n, H, D))
        if out is None:
            out = torch.empty_like(q, memory_format=torch.contiguous_format)
            outr = (out.data_ptr(), n * heads * D, heads * D, D)
        else:
            outr = self._rows(out, "out", dtype, (S, n, heads, D))
        a = self._ATTN.pack(n, heads, kind, scale, *qr, *outr, *kr, *vr,
                            0 if counts is None else self._vec(counts, "counts", torch.int32, (S,)),
                            0 if mask is None else self._vec(mask, "mask", torch.int64, (S, n)))
        self._launch(self._attention, "w4a8_kv4_attention_workspace_bytes", (n, heads, kind, k is None), a, workspace)
        return out


# ------------------------------------------------------- norm and rotation of queries and keys

class Rotary:
    """Rotary positions of one head size, with the norm of queries and keys in the same pass (w4a8_qk_rotary).

    ``rot_dim``: dims that are turned (all by default).  The frequencies, radians for each position, are ``base`` to the powers
    -2 i / rot_dim, or ``inv_freq`` [rot_dim / 2] (64-bit values; any stretching of the context is in them).  ``axis``
    [rot_dim / 2]: for positions of several axes (time, height, width), the axis of each frequency.  ``neighbours``: pairs
    are dims (2 i, 2 i + 1) instead of (i, i + rot_dim / 2).  ``factor`` multiplies the turned dims.
    """

    _ARGS = struct.Struct("@10i 2f 7q 16q")              # w4a8_qk_rotary_args
    _NONE = (0, 0, 0, 0)

    def __init__(self, head_dim, rot_dim=None, base=10000.0, inv_freq=None, axis=None, neighbours=False, factor=1.0,
                 device="cuda"):
        import numpy as np
        import torch
        self._torch = torch
        self._types = {torch.float32: 0, torch.bfloat16: 1}
        rot = head_dim if rot_dim is None else rot_dim
        if head_dim < 16 or head_dim > 256 or head_dim % 16 or rot < 0 or rot > head_dim or rot % 16:
            raise ValueError("Rotary: head_dim and rot_dim must be multiples of 16, at most 256 and head_dim")
        half = rot // 2
        inv = float(base) ** (-np.arange(half) / max(half, 1)) if inv_freq is None else np.asarray(inv_freq)
        inv = np.ascontiguousarray(inv, dtype=np.float64)
        axis = np.zeros(half, np.int64) if axis is None else np.asarray(axis)
        if inv.shape != (half,) or axis.shape != (half,):
            raise ValueError("Rotary: inv_freq and axis must have rot_dim / 2 = %d entries" % half)
        if half and (axis.min() < 0 or axis.max() > 3):
            raise ValueError("Rotary: at most four axes")
        turns = np.zeros(half, np.uint64)
        if half:
            _call("w4a8_rotary_turns", inv.ctypes.data_as(_vp), half, turns.ctypes.data_as(_vp))
        self.n_axes = int(axis.max()) + 1 if half else 1
        self.head_dim, self.rot_dim, self.neighbours, self.factor = head_dim, rot, bool(neighbours), float(factor)
        self._turns = torch.from_numpy(turns.view(np.int64)).to(device)
        self._axis = torch.from_numpy(axis.astype(np.uint8)).to(device)
        self.device = self._turns.device
        self._dev = self._turns.get_device()
        if self._dev < 0:
            raise ValueError("Rotary: needs a CUDA device")
        self._fn = lib().w4a8_qk_rotary
        self._mine = (self._turns.data_ptr() if half else 0, self._axis.data_ptr() if self.n_axes > 1 else 0)

    def _rows(self, t, name, dtype, shape):
        a, b, c, d = t.stride() if t.shape == shape else (0, 0, 0, 0)
        if d != 1 or t.dtype is not dtype or t.get_device() != self._dev:
            raise ValueError("Rotary: %s must be %s %s with unit stride in the last dimension, on the tables' device"
                             % (name, str(dtype)[6:], list(shape)))
        return t.data_ptr(), a, b, c

    def _vec(self, t, name, dtype, shape):
        if t is None:
            return 0
        if t.dtype is not dtype or t.shape != shape or t.get_device() != self._dev or not t.is_contiguous():
            raise ValueError("Rotary: %s must be a contiguous %s tensor %s on the tables' device"
                             % (name, str(dtype)[6:], list(shape)))
        return t.data_ptr()

    def apply(self, q, k=None, positions=None, start=None, eps=None, q_gain=None, k_gain=None, counts=None, q_out=None,
              k_out=None, stream=None):
        """(q, k) turned, in new tensors or in ``q_out`` and ``k_out`` (which may be q and k themselves); q alone where k is not
        given.  q, k: fp32 or bf16 [n_seqs][n][heads][head_dim], unit stride in the last dimension.  ``positions`` int32
        [n_axes][n_seqs][n] ([n_seqs][n] does for one axis), the row's number by default; ``start`` int32 [n_seqs] is added to
        them (e.g. a cache's ``len``).  ``eps``: divide each head by the root of its mean square plus eps, times ``q_gain``,
        ``k_gain`` (fp32 [head_dim], 1 by default); None: no norm.  ``counts`` int32 [n_seqs]: rows behind them are left as
        they were in given outputs, and hold anything in new ones."""
        torch = self._torch
        if stream is not None:
            if stream.device != self.device:
                raise ValueError("Rotary: the stream is on another device than the tables")
            args = (q, k, positions, start, eps, q_gain, k_gain, counts, q_out, k_out)
            with torch.cuda.stream(stream):
                result = self.apply(*args)
            for t in args + (self._turns, self._axis):
                if isinstance(t, torch.Tensor):
                    t.record_stream(stream)
            return result
        shape, dtype, D = q.shape, q.dtype, self.head_dim
        kind = self._types.get(dtype)
        if kind is None or len(shape) != 4 or shape[3] != D:
            raise ValueError("Rotary: q must be fp32 or bf16 [n_seqs][n][heads][%d], not %s %s"
                             % (D, str(dtype)[6:], list(shape)))
        S, n, heads, _ = shape
        qr = self._rows(q, "q", dtype, shape)
        if q_out is None:
            q_out = torch.empty(shape, dtype=dtype, device=self.device)
            qo = (q_out.data_ptr(), n * heads * D, heads * D, D)
        else:
            qo = self._rows(q_out, "q_out", dtype, shape)
        kv_heads, kr, ko = 0, self._NONE, self._NONE
        if k is not None:
            kv_heads = k.shape[2] if k.dim() == 4 else 0
            kshape = (S, n, kv_heads, D)
            kr = self._rows(k, "k", dtype, kshape)
            if k_out is None:
                k_out = torch.empty(kshape, dtype=dtype, device=self.device)
                ko = (k_out.data_ptr(), n * kv_heads * D, kv_heads * D, D)
            else:
                ko = self._rows(k_out, "k_out", dtype, kshape)
        elif k_out is not None or k_gain is not None:
            raise ValueError("Rotary: k_out and k_gain need k")
        if eps is None and (q_gain is not None or k_gain is not None):
            raise ValueError("Rotary: gains need eps")
        i32, f32 = torch.int32, torch.float32
        pos = 0
        if positions is not None:
            pshape = (S, n) if self.n_axes == 1 and positions.dim() == 2 else (self.n_axes, S, n)
            pos = self._vec(positions, "positions", i32, pshape)
        a = self._ARGS.pack(S, n, heads, kv_heads, D, self.rot_dim, self.n_axes, self.neighbours, kind, eps is not None,
                            0.0 if eps is None else eps, self.factor, *self._mine, pos,
                            self._vec(start, "start", i32, (S,)), self._vec(counts, "counts", i32, (S,)),
                            self._vec(q_gain, "q_gain", f32, (D,)), self._vec(k_gain, "k_gain", f32, (D,)),
                            *qr, *qo, *kr, *ko)
        if torch.cuda.current_device() == self._dev:
            status = self._fn(a, torch._C._cuda_getCurrentRawStream(self._dev))
        else:
            with torch.cuda.device(self._dev):
                status = self._fn(a, torch._C._cuda_getCurrentRawStream(self._dev))
        if status:
            raise W4A8Error("w4a8_qk_rotary", status)
        return q_out if k is None else (q_out, k_out)


# ------------------------------------------------------------------------ model/session

def _arr(vals, ctype=_i32):
    vals = list(vals)
    return (ctype * max(1, len(vals)))(*vals)


class Model:
    """A decoder held by the library (w4a8_model)."""

    def __init__(self, n_layers, hidden, n_heads, n_kv_heads, head_dim, ffn, vocab, tied,
                 rms_eps=1e-6, rope_base=10000.0):
        self.desc = ModelDesc(n_layers, hidden, n_heads, n_kv_heads, head_dim, ffn, vocab, int(bool(tied)),
                              rms_eps, rope_base)
        h = _vp()
        _call("w4a8_model_create", _c.byref(self.desc), _c.byref(h))
        self.h = h

    def load_tensor(self, kind, layer, w_p2, s_p2, stream=None):
        _call("w4a8_model_load_tensor", self.h, int(kind), int(layer), _ptr(w_p2), _ptr(s_p2), _stream(stream))

    def weight_bytes(self):
        b = _sz()
        _call("w4a8_model_weight_bytes", self.h, _c.byref(b))
        return b.value

    def close(self):
        if getattr(self, "h", None):
            lib().w4a8_model_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Session:
    """A decoding session (w4a8_session) on a Model."""

    def __init__(self, model, kv_cap, ctx_cap, max_window=16, eos_id=-1, mem_cap=0):
        self.model = model
        self.desc = SessionDesc(kv_cap, ctx_cap, max_window, eos_id, mem_cap)
        h = _vp()
        _call("w4a8_session_create", model.h, _c.byref(self.desc), _c.byref(h))
        self.h = h

    def close(self):
        if getattr(self, "h", None):
            lib().w4a8_session_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # device-side operations (asynchronous on the current stream)
    def prefill(self, prompt_dev, max_new, stream=None):
        _call("w4a8_prefill", self.h, _ptr(prompt_dev), int(prompt_dev.numel()), int(max_new), _stream(stream))

    def tree_verify_step(self, N, logits=None, stream=None):
        _call("tree_verify_step", self.h, int(N), _ptr(logits), _stream(stream))

    def trace_bytes(self, N):
        n = _sz()
        _call("w4a8_model_trace_bytes", self.model.h, int(N), _c.byref(n))
        return n.value

    def tree_verify_trace(self, N, codes, logits=None, stream=None):
        """tree_verify_step that also writes the int8 codes of every quantisation point into
        the device int8 buffer ``codes`` (w4a8_tree_verify_trace)."""
        _call("w4a8_tree_verify_trace", self.h, int(N), _ptr(logits), _ptr(codes),
              codes.numel() * codes.element_size(), _stream(stream))

    def accept_greedy(self, N, stream=None):
        _call("accept_greedy", self.h, int(N), _stream(stream))

    def kv_compact(self, stream=None):
        _call("kv_compact", self.h, _stream(stream))

    def ngram_draft(self, stream=None):
        _call("ngram_draft", self.h, _stream(stream))

    def spec_step(self, N, stream=None):
        _call("w4a8_spec_step", self.h, int(N), _stream(stream))

    def spec_window(self, N, W, stream=None):
        _call("spec_window", self.h, int(N), int(W), _stream(stream))

    def spec_poll(self, W, timeout_us=-1):
        c = Ctl16()
        st = (StepStats * max(1, W))()
        toks = (_i32 * (16 * max(1, W)))()
        ns, nt = _i32(), _i32()
        _call("spec_poll", self.h, _c.byref(c), st, _c.byref(ns), toks, _c.byref(nt), int(timeout_us))
        return c, list(st)[:ns.value], list(toks)[:nt.value]

    def calibrate(self, widths, reps=20, trials=5):
        out = (_f32 * len(widths))()
        _call("w4a8_calibrate", self.h, _arr(widths), len(widths), int(reps), int(trials), out)
        return list(out)

    @staticmethod
    def _opts(max_new, window, fixed_width, in_flight, widths, t_us, timeout_us):
        o = DecodeOpts()
        o.max_new, o.window, o.fixed_width, o.in_flight, o.timeout_us = max_new, window, fixed_width, in_flight, timeout_us
        o.n_widths = len(widths)
        for i, (w, t) in enumerate(zip(widths, t_us)):
            o.widths[i], o.t_us[i] = int(w), float(t)
        return o

    def generate(self, max_new, window=4, fixed_width=0, in_flight=2, widths=(), t_us=(), timeout_us=-1,
                 stream=None):
        """Window loop on a prefilled session; returns (tokens, DecodeReport)."""
        o = self._opts(max_new, window, fixed_width, in_flight, widths, t_us, timeout_us)
        out = (_i32 * max(1, max_new))()
        n_out = _i32()
        rep = DecodeReport()
        _call("w4a8_generate", self.h, _c.byref(o), out, _c.byref(n_out), _c.byref(rep), _stream(stream))
        return list(out)[:n_out.value], rep

    def time_matmuls(self, N, reps=5):
        us, by, nl = _dbl(), _dbl(), _i32()
        _call("w4a8_time_matmuls", self.h, int(N), int(reps), _c.byref(us), _c.byref(by), _c.byref(nl))
        return us.value, by.value, nl.value

    def decode(self, prompt, max_new, window=4, fixed_width=0, in_flight=2, widths=(), t_us=(),
               timeout_us=-1, stream=None):
        """End-to-end decode from a host prompt; returns (tokens, DecodeReport)."""
        o = DecodeOpts()
        o.max_new, o.window, o.fixed_width, o.in_flight, o.timeout_us = max_new, window, fixed_width, in_flight, timeout_us
        o.n_widths = len(widths)
        for i, (w, t) in enumerate(zip(widths, t_us)):
            o.widths[i], o.t_us[i] = int(w), float(t)
        p = _arr([int(t) for t in prompt])
        out = (_i32 * max(1, max_new))()
        n_out = _i32()
        rep = DecodeReport()
        _call("w4a8_decode", self.h, p, len(prompt), _c.byref(o), out, _c.byref(n_out), _c.byref(rep),
              _stream(stream))
        return list(out)[:n_out.value], rep

    def raise_flags(self, flags, stream=None):
        _call("w4a8_session_raise_flags", self.h, int(flags), _stream(stream))

    # synchronous state access
    def ctl(self):
        c = Ctl()
        _call("w4a8_session_get_ctl", self.h, _c.byref(c))
        return c

    def set_tree(self, tok, parent):
        n = len(tok)
        _call("w4a8_session_set_tree", self.h, _arr(tok), _arr(parent), n)

    def tree(self):
        tok, par, dep = (_i32 * 16)(), (_i32 * 16)(), (_i32 * 16)()
        nv, bl = _i32(), _i32()
        _call("w4a8_session_get_tree", self.h, tok, par, dep, _c.byref(nv), _c.byref(bl))
        return list(tok), list(par), list(dep), nv.value, bl.value

    def pred(self, n):
        out = (_i32 * n)()
        _call("w4a8_session_get_pred", self.h, out, int(n))
        return list(out)

    def context(self, cap=1 << 16):
        out = (_i32 * cap)()
        n = _i32()
        _call("w4a8_session_get_context", self.h, out, cap, _c.byref(n))
        return list(out)[:min(cap, n.value)]

    def copy_kv(self, layer, slot0, n, k_out, v_out, stream=None):
        _call("w4a8_session_copy_kv", self.h, int(layer), int(slot0), int(n), _ptr(k_out), _ptr(v_out),
              _stream(stream))

    def memory_append(self, tokens):
        """Appends an earlier output to the session memory (w4a8_session_memory_append)."""
        _call("w4a8_session_memory_append", self.h, _arr([int(t) for t in tokens]), len(tokens))

    def memory_clear(self):
        _call("w4a8_session_memory_clear", self.h)

    def memory(self, cap=1 << 16):
        out = (_i32 * cap)()
        n = _i32()
        _call("w4a8_session_memory_get", self.h, out, cap, _c.byref(n))
        return list(out)[:min(cap, n.value)]

    def load_kv(self, layer, slot0, n, k_in, v_in, stream=None):
        _call("w4a8_session_load_kv", self.h, int(layer), int(slot0), int(n), _ptr(k_in), _ptr(v_in),
              _stream(stream))

    def attention(self, layer, n, q, out, stream=None):
        """Tree attention of one layer for device queries q [n][n_heads][head_dim] (after RoPE
        and the 1/sqrt(head_dim) scale) into out [n][n_heads * head_dim] (w4a8_session_attention)."""
        _call("w4a8_session_attention", self.h, int(layer), int(n), _ptr(q), _ptr(out), _stream(stream))


class Controller:
    """The host width controller (w4a8_controller)."""

    def __init__(self, widths, t_us):
        h = _vp()
        _call("w4a8_controller_create", _arr(widths), _arr(t_us, _f32), len(widths), _c.byref(h))
        self.h = h

    def choose(self):
        return lib().w4a8_controller_choose(self.h)

    def observe(self, width, stats, interval_us=0.0):
        arr = (StepStats * max(1, len(stats)))()
        for i, st in enumerate(stats):
            arr[i] = st if isinstance(st, StepStats) else StepStats(*st)
        _call("w4a8_controller_observe", self.h, int(width), arr, len(stats), float(interval_us))

    def expected_tokens(self, width):
        return lib().w4a8_controller_expected_tokens(self.h, int(width))

    def cost(self, width):
        return lib().w4a8_controller_cost(self.h, int(width))

    def __del__(self):
        try:
            if getattr(self, "h", None):
                lib().w4a8_controller_destroy(self.h)
                self.h = None
        except Exception:
            pass
