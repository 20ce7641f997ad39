"""Python binding of the OSCAR INT2 KV-cache library (liboscar.so, CUDA sm_103a).

Argument marshalling only: every step of the write and decode paths runs in
the library's CUDA kernels. PyTorch supplies device memory and the current
stream. If the compiled library is missing, importing the binding raises; there
is no fallback.

The C entry points, layouts and error behaviour are documented in
``include/oscar.h``; the names here follow them.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "liboscar.so")

OK = 0
ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_DEVICE_STATUS, ERR_TIMEOUT, ERR_NOT_ORTHOGONAL = -1, -2, -3, -4, -5, -6
ERR_TOO_LARGE = -7
STATUS_BAD_PAGE, STATUS_BAD_SEQLEN, STATUS_TIMEOUT, STATUS_NONFINITE, STATUS_SATURATED = 1, 2, 4, 8, 16
STATUS_NO_PAGES, STATUS_BAD_TREE = 32, 64
V_ABSORBED, V_EXPLICIT = 0, 1
OUT_BF16, OUT_FP32 = 0, 1
KIND_K, KIND_V = 0, 1
DECODE_SIMT, DECODE_MMA, DECODE_TC = 0, 1, 2
META_F16, META_U8, META_CB = 0, 1, 2
ROPE_NONE, ROPE_LINEAR, ROPE_NTK, ROPE_YARN = 0, 1, 2, 3
ROPE_HALF, ROPE_PAIRS = 0, 1
DTYPE_BF16, DTYPE_FP32, DTYPE_FP16 = 0, 1, 2
MAX_DRAFT = 256
MAX_ROPE_AXES = 4

# every symbol include/oscar.h declares
EXPORTS = (
    "oscar_cache_bytes", "oscar_cache_create", "oscar_cache_destroy", "oscar_layer_offsets", "oscar_set_rotation",
    "oscar_quantize_prefill", "oscar_project_quantize_prefill", "oscar_append_kv", "oscar_decode_attention", "oscar_set_decode_algo",
    "oscar_get_status", "oscar_pack_rotated", "oscar_rotate", "oscar_bf16_decode_workspace_bytes",
    "oscar_bf16_decode", "oscar_calibrate", "oscar_profile_begin", "oscar_profile_read", "oscar_error_string",
    "oscar_decode_attention_noalloc", "oscar_trace_ctas", "oscar_decode_step",
    "oscar_decode_attention_shared", "oscar_decode_step_shared",
    "oscar_trace_timeline", "oscar_check_wait_timeout", "oscar_set_codebook", "oscar_calibrate_codebook",
    "oscar_build_tables", "oscar_tree_layout", "oscar_rope_frequencies", "oscar_rope_turns", "oscar_rope",
    "oscar_tree_workspace_bytes", "oscar_tree_attention", "oscar_commit_draft",
    "oscar_rope_axes", "oscar_norm_rope", "oscar_norm_rope_backward", "oscar_norm_rope_workspace_bytes",
    "oscar_append_kv_rope", "oscar_decode_step_rope", "oscar_prompt_attention",
)


class OscarError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {_lib.oscar_error_string(code).decode()} ({code})")


class Layout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "num_layers", "num_kv_heads", "num_q_heads", "head_dim", "group", "page_size", "sink", "recent",
        "num_int2_pages", "num_bf16_pages", "v_mode", "max_batch", "max_splits", "meta_format")]


class RopeTensor(ctypes.Structure):
    _fields_ = [("inp", ctypes.c_void_p), ("out", ctypes.c_void_p)] + [
        (n, ctypes.c_int64) for n in ("in_token", "in_head", "out_token", "out_head")] + [("heads", ctypes.c_int)]


class Rotary(ctypes.Structure):
    _fields_ = [("turns", ctypes.c_void_p), ("axes", ctypes.c_void_p), ("num_axes", ctypes.c_int),
                ("rotary_dim", ctypes.c_int), ("layout", ctypes.c_int), ("scale", ctypes.c_float)]


class Heads(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("token", ctypes.c_int64), ("head", ctypes.c_int64)]


class RawStep(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in "qkv"] + [(n, ctypes.c_int64) for n in ("q_row", "k_row", "v_row")] + [
        (n, ctypes.c_void_p) for n in ("q_out", "positions", "rotary", "norm")]


class HeadNorm(ctypes.Structure):
    _fields_ = [("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("eps", ctypes.c_float)]


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"OSCAR CUDA library not built ({LIB_PATH} missing); run __graft_entry__.build()")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32p, sz = ctypes.c_void_p, ctypes.c_void_p, ctypes.POINTER(ctypes.c_size_t)
    c_int, c_float, c_double = ctypes.c_int, ctypes.c_float, ctypes.c_double
    sig = {
        "oscar_cache_bytes": [ctypes.POINTER(Layout), sz, sz],
        "oscar_cache_create": [ctypes.POINTER(Layout), vp, vp, ctypes.POINTER(vp)],
        "oscar_cache_destroy": [vp],
        "oscar_layer_offsets": [vp, c_int, sz, sz, sz],
        "oscar_set_rotation": [vp, c_int, vp, vp, vp, vp, vp],
        "oscar_set_codebook": [vp, c_int, vp, vp, vp],
        "oscar_calibrate_codebook": [vp, c_int, vp, vp],
        "oscar_quantize_prefill": [vp, c_int, c_int, vp, vp, i32p, c_int, i32p, c_int, i32p, vp],
        "oscar_project_quantize_prefill": [vp, c_int, c_int, vp, c_int, vp, vp, i32p, c_int, i32p, c_int, i32p, vp],
        "oscar_append_kv": [vp, c_int, c_int, vp, vp, i32p, i32p, c_int, i32p, vp],
        "oscar_decode_attention": [vp, c_int, c_int, vp, i32p, i32p, c_int, i32p, c_float, vp, c_int, vp, vp],
        "oscar_set_decode_algo": [vp, c_int],
        "oscar_get_status": [vp, ctypes.POINTER(c_int)],
        "oscar_pack_rotated": [vp, c_int, c_int, vp, i32p, i32p, c_int, vp],
        "oscar_rotate": [vp, c_int, c_int, vp, vp, c_int, vp],
        "oscar_bf16_decode_workspace_bytes": [c_int, c_int, c_int, sz],
        "oscar_bf16_decode": [c_int, c_int, c_int, vp, c_int, vp, i32p, i32p, c_int, c_float, vp, c_int, vp, vp,
                              ctypes.c_size_t, c_int, vp],
        "oscar_calibrate": [vp, vp, vp, c_int, c_float, c_float, c_float, vp, vp, vp, vp, vp, vp],
        "oscar_profile_begin": [vp, c_int],
        "oscar_profile_read": [vp, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(c_int)],
        "oscar_trace_ctas": [vp, vp, c_int],
        "oscar_trace_timeline": [vp, vp, c_int],
        "oscar_check_wait_timeout": [vp, vp],
        "oscar_decode_step": [vp, c_int, c_int, vp, vp, vp, i32p, i32p, c_int, i32p, c_float, vp, c_int, vp, vp],
        "oscar_decode_attention_shared": [vp, c_int, c_int, vp, i32p, i32p, c_int, c_int, i32p, c_float, vp, c_int,
                                          vp, vp],
        "oscar_decode_step_shared": [vp, c_int, c_int, vp, vp, vp, i32p, i32p, c_int, c_int, i32p, c_float, vp,
                                     c_int, vp, vp],
        "oscar_build_tables": [vp, c_int, i32p, i32p, i32p, c_int, i32p, i32p, i32p, i32p, i32p, i32p, i32p, c_int, vp],
        "oscar_tree_layout": [vp, c_int, c_int, i32p, i32p, i32p, vp, i32p, vp],
        "oscar_rope_frequencies": [c_int, c_double, c_int, c_double, c_double, c_double, c_double, vp,
                                   ctypes.POINTER(c_float)],
        "oscar_rope_turns": [vp, c_int, vp],
        "oscar_rope": [ctypes.POINTER(RopeTensor), ctypes.POINTER(RopeTensor), c_int, c_int, c_int, i32p, vp, c_int,
                       c_int, c_float, c_int, vp],
        "oscar_rope_axes": [ctypes.POINTER(RopeTensor), ctypes.POINTER(RopeTensor), c_int, c_int, c_int, i32p,
                            ctypes.POINTER(Rotary), c_int, vp],
        "oscar_norm_rope": [ctypes.POINTER(RopeTensor), ctypes.POINTER(RopeTensor), c_int, c_int, c_int, i32p,
                            ctypes.POINTER(Rotary), ctypes.POINTER(HeadNorm), vp],
        "oscar_prompt_attention": [vp, c_int] + [ctypes.POINTER(Heads)] * 3 + [i32p, c_int, c_float, vp, c_int, vp, vp],
        "oscar_append_kv_rope": [vp, c_int, c_int, ctypes.POINTER(RawStep), i32p, i32p, c_int, i32p, vp],
        "oscar_decode_step_rope": [vp, c_int, c_int, ctypes.POINTER(RawStep), i32p, i32p, c_int, c_int, i32p, c_float, vp,
                                   c_int, vp, vp],
        "oscar_norm_rope_workspace_bytes": [c_int, sz],
        "oscar_norm_rope_backward": [ctypes.POINTER(RopeTensor)] * 4 + [c_int, c_int, c_int, i32p, ctypes.POINTER(Rotary),
                                                                        ctypes.POINTER(HeadNorm), vp, vp, vp,
                                                                        ctypes.c_size_t, vp],
        "oscar_tree_workspace_bytes": [vp, c_int, c_int, c_int, sz],
        "oscar_tree_attention": [vp, c_int, c_int, c_int, vp, vp, vp, vp, i32p, i32p, i32p, c_int, i32p, c_float, vp,
                                 c_int, vp, vp, ctypes.c_size_t, vp],
        "oscar_commit_draft": [vp, c_int, c_int, c_int, vp, vp, i32p, i32p, c_int, i32p, i32p, c_int, i32p, vp],
        "oscar_decode_attention_noalloc": [ctypes.POINTER(Layout), vp, c_int, c_int, vp, i32p, i32p, c_int, i32p,
                                           c_float, vp, c_int, vp, vp, vp],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = c_int
    lib.oscar_error_string.argtypes = [c_int]
    lib.oscar_error_string.restype = ctypes.c_char_p
    return lib


_lib = _load()


def lib() -> ctypes.CDLL:
    return _lib


def _check(rc: int, what: str):
    if rc != OK:
        raise OscarError(rc, what)


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, np.ndarray):
        return t.ctypes.data
    return t.data_ptr()


def _stream(stream=None) -> int:
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _dev_i32(x, device):
    import torch
    if isinstance(x, torch.Tensor):
        assert x.dtype == torch.int32 and x.is_cuda and x.is_contiguous()
        return x
    return torch.as_tensor(np.ascontiguousarray(x, dtype=np.int32), device=device)


# torch's names that the calls below look up on every call, bound by the first of them: a call costs about 9 us on the
# host, and looking them up afresh was 2 us of it
_tensor = _i32 = _words = _bf16 = _f32 = _f16 = _u8 = _empty = _get_device = _get_stream = None


def _bind_torch():
    global _tensor, _i32, _words, _bf16, _f32, _f16, _u8, _empty, _get_device, _get_stream
    import torch
    _i32, _words, _bf16, _f32, _f16 = torch.int32, (torch.int64, torch.uint64), torch.bfloat16, torch.float32, torch.float16
    _u8 = torch.uint8
    _empty, _get_device, _get_stream = torch.empty, torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
    _tensor = torch.Tensor


def _on(stream):
    import torch
    return torch.cuda.stream(stream)


def _here(t) -> tuple[int, int]:
    """The current device, which t has to be on, and its current stream. (The handle is asked for directly: building
    torch's stream object costs 3 us of a call.)"""
    if _tensor is None:
        _bind_torch()
    dev = _get_device()
    if t.get_device() != dev:
        raise OscarError(ERR_INVALID_ARG, "tensors on the current device")
    return dev, _get_stream(dev)


def _in_i32(x, dev: int):
    """int32 values for the library to read: a contiguous tensor on device dev, or host values that are copied."""
    if isinstance(x, _tensor):
        if x.dtype is not _i32 or x.get_device() != dev or not x.is_contiguous():
            raise OscarError(ERR_INVALID_ARG, "contiguous int32 tensor on the current device")
        return x
    import torch
    return torch.as_tensor(np.ascontiguousarray(x, dtype=np.int32), device=dev)


def _own_i32(t, numel: int, dev: int):
    """An int32 device tensor the library writes (never copied): contiguous, of at least numel elements."""
    if not isinstance(t, _tensor) or t.dtype is not _i32 or t.get_device() != dev or not t.is_contiguous() or \
            t.numel() < numel:
        raise OscarError(ERR_INVALID_ARG, f"contiguous int32 tensor of at least {numel} elements on the current device")
    return t


def _check_words(t, B: int, T: int, dev: int, what: str):
    if t.dtype not in _words or t.get_device() != dev or not t.is_contiguous() or t.shape != (B, T, (T + 63) // 64):
        raise OscarError(ERR_INVALID_ARG, what)


def _check_like(t, dtype, shape, dev: int, what: str):
    if t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous() or t.shape != shape:
        raise OscarError(ERR_INVALID_ARG, what)


@dataclass
class CacheConfig:
    num_layers: int
    num_kv_heads: int
    num_q_heads: int
    num_int2_pages: int
    num_bf16_pages: int
    max_batch: int = 1
    max_splits: int = 256
    v_mode: int = V_ABSORBED
    head_dim: int = 128
    group: int = 64
    page_size: int = 64
    sink: int = 64
    recent: int = 256
    meta_format: int = META_F16        # META_U8: 16-bit (mn8, mx8) group metadata, 4608-byte INT2 blocks;
    #                                    META_CB: Lloyd-Max codebook levels with fp16 (range, zero) metadata

    def layout(self) -> Layout:
        return Layout(self.num_layers, self.num_kv_heads, self.num_q_heads, self.head_dim, self.group,
                      self.page_size, self.sink, self.recent, self.num_int2_pages, self.num_bf16_pages, self.v_mode,
                      self.max_batch, self.max_splits, self.meta_format)


def cache_bytes(cfg: CacheConfig) -> tuple[int, int]:
    lay = cfg.layout()
    pb, wb = ctypes.c_size_t(), ctypes.c_size_t()
    _check(_lib.oscar_cache_bytes(ctypes.byref(lay), ctypes.byref(pb), ctypes.byref(wb)), "oscar_cache_bytes")
    return pb.value, wb.value


class OscarCache:
    """A mixed-precision KV cache: caller-owned pool and workspace (torch uint8 tensors) plus the library handle."""

    def __init__(self, cfg: CacheConfig, device="cuda", pool=None, workspace=None):
        import torch
        self.cfg = cfg
        self.device = torch.device(device)
        pb, wb = cache_bytes(cfg)
        self.pool = torch.zeros(pb, dtype=torch.uint8, device=self.device) if pool is None else pool
        self.workspace = torch.zeros(wb, dtype=torch.uint8, device=self.device) if workspace is None else workspace
        lay = cfg.layout()
        h = ctypes.c_void_p()
        _check(_lib.oscar_cache_create(ctypes.byref(lay), _ptr(self.pool), _ptr(self.workspace), ctypes.byref(h)),
               "oscar_cache_create")
        self._h = h

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            _lib.oscar_cache_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def handle(self):
        return self._h

    # ---- layout views --------------------------------------------------------------
    def layer_offsets(self, layer: int) -> tuple[int, int, int]:
        a, b, c = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
        _check(_lib.oscar_layer_offsets(self._h, layer, ctypes.byref(a), ctypes.byref(b), ctypes.byref(c)),
               "oscar_layer_offsets")
        return a.value, b.value, c.value

    def int2_pages(self, layer: int):
        """uint8 view [num_int2_pages, Hkv, block] of a layer's INT2 page blocks (block = 5120 bytes,
        or 4608 with the compact META_U8 metadata)."""
        o, _, _ = self.layer_offsets(layer)
        blk = 4608 if self.cfg.meta_format == META_U8 else 5120
        n = self.cfg.num_int2_pages * self.cfg.num_kv_heads * blk
        return self.pool[o:o + n].view(self.cfg.num_int2_pages, self.cfg.num_kv_heads, blk)

    def bf16_pages(self, layer: int):
        """uint8 view [num_bf16_pages, Hkv, 32768] of a layer's BF16 page blocks."""
        _, o, _ = self.layer_offsets(layer)
        n = self.cfg.num_bf16_pages * self.cfg.num_kv_heads * 32768
        return self.pool[o:o + n].view(self.cfg.num_bf16_pages, self.cfg.num_kv_heads, 32768)

    # ---- entry points ---------------------------------------------------------------
    def set_rotation(self, layer: int, U_K, U_V, tau_K, tau_V, stream=None):
        import torch
        stream = torch.cuda.current_stream(self.pool.device) if stream is None else stream
        f32 = lambda a: None if a is None else np.ascontiguousarray(a, dtype=np.float32)
        uk, uv, tk, tv = f32(U_K), f32(U_V), f32(tau_K), f32(tau_V)
        _check(_lib.oscar_set_rotation(self._h, layer, _ptr(uk), _ptr(uv), _ptr(tk), _ptr(tv), _stream(stream)),
               "oscar_set_rotation")

    def set_codebook(self, layer: int, cb_K, cb_V, stream=None):
        """Codebook bytes uint8 [Hkv][4] of K and V (META_CB layouts); call after set_rotation."""
        ck = np.ascontiguousarray(cb_K, dtype=np.uint8)
        cv = np.ascontiguousarray(cb_V, dtype=np.uint8)
        _check(_lib.oscar_set_codebook(self._h, layer, _ptr(ck), _ptr(cv), _stream(stream)), "oscar_set_codebook")

    def quantize_prefill(self, layer: int, k, v, cu_seqlens, hist_pt, bf16_pt, total_tokens: int | None = None,
                         stream=None):
        cu = _dev_i32(cu_seqlens, self.device)
        hp = _dev_i32(hist_pt, self.device)
        bp = _dev_i32(bf16_pt, self.device)
        B = cu.numel() - 1
        total = int(k.shape[0]) if total_tokens is None else total_tokens
        mhp = hp.shape[1] if hp.dim() == 2 else 0
        _check(_lib.oscar_quantize_prefill(self._h, layer, B, _ptr(k), _ptr(v), _ptr(cu), total, _ptr(hp), mhp,
                                           _ptr(bp), _stream(stream)), "oscar_quantize_prefill")

    def project_quantize_prefill(self, layer: int, x, w_k, w_v, cu_seqlens, hist_pt, bf16_pt,
                                 total_tokens: int | None = None, stream=None):
        """quantize_prefill of K = bf16(x W_k^T), V = bf16(x W_v^T): x bf16 [T, d_model], w bf16 [Hkv*128, d_model]."""
        cu = _dev_i32(cu_seqlens, self.device)
        hp = _dev_i32(hist_pt, self.device)
        bp = _dev_i32(bf16_pt, self.device)
        B = cu.numel() - 1
        total = int(x.shape[0]) if total_tokens is None else total_tokens
        mhp = hp.shape[1] if hp.dim() == 2 else 0
        _check(_lib.oscar_project_quantize_prefill(self._h, layer, B, _ptr(x), int(x.shape[1]), _ptr(w_k), _ptr(w_v),
                                                   _ptr(cu), total, _ptr(hp), mhp, _ptr(bp), _stream(stream)),
               "oscar_project_quantize_prefill")

    def append_kv(self, layer: int, k, v, seq_lens_before, hist_pt, bf16_pt, stream=None):
        """Append one token per request. Lengths and tables on the device are read before the kernel just before this
        call on the stream is waited for: of a kernel of the caller's launched there only k and v may come."""
        sl = _dev_i32(seq_lens_before, self.device)
        hp = _dev_i32(hist_pt, self.device)
        bp = _dev_i32(bf16_pt, self.device)
        _check(_lib.oscar_append_kv(self._h, layer, sl.numel(), _ptr(k), _ptr(v), _ptr(sl), _ptr(hp),
                                    hp.shape[1] if hp.dim() == 2 else 0, _ptr(bp), _stream(stream)),
               "oscar_append_kv")

    def decode_attention(self, layer: int, q, seq_lens, hist_pt, bf16_pt, sm_scale: float, out=None,
                         out_dtype: int = OUT_BF16, lse=None, stream=None, shared_hist_pages: int = 0):
        """Decode attention; shared_hist_pages > 0 states that history pages [0, shared_hist_pages) of every
        request are the same pages (oscar_decode_attention_shared)."""
        import torch
        sl = _dev_i32(seq_lens, self.device)
        hp = _dev_i32(hist_pt, self.device)
        bp = _dev_i32(bf16_pt, self.device)
        if out is None:
            out = torch.empty(q.shape, dtype=torch.float32 if out_dtype == OUT_FP32 else torch.bfloat16,
                              device=self.device)
        mhp = hp.shape[1] if hp.dim() == 2 else 0
        if shared_hist_pages:
            _check(_lib.oscar_decode_attention_shared(self._h, layer, sl.numel(), _ptr(q), _ptr(sl), _ptr(hp), mhp,
                                                      int(shared_hist_pages), _ptr(bp), float(sm_scale), _ptr(out),
                                                      out_dtype, _ptr(lse), _stream(stream)),
                   "oscar_decode_attention_shared")
        else:
            _check(_lib.oscar_decode_attention(self._h, layer, sl.numel(), _ptr(q), _ptr(sl), _ptr(hp), mhp,
                                               _ptr(bp), float(sm_scale), _ptr(out), out_dtype, _ptr(lse),
                                               _stream(stream)), "oscar_decode_attention")
        return out

    def decode_step(self, layer: int, q, k, v, seq_lens_before, hist_pt, bf16_pt, sm_scale: float, out=None,
                    out_dtype: int = OUT_BF16, lse=None, stream=None, shared_hist_pages: int = 0):
        """append_kv(k, v) then decode_attention(q) over seq_lens_before + 1 tokens, in one call
        (oscar_decode_step_shared when shared_hist_pages > 0). As for append_kv, only q, k and v may come from a kernel
        of the caller's launched just before."""
        import torch
        sl = _dev_i32(seq_lens_before, self.device)
        hp = _dev_i32(hist_pt, self.device)
        bp = _dev_i32(bf16_pt, self.device)
        if out is None:
            out = torch.empty(q.shape, dtype=torch.float32 if out_dtype == OUT_FP32 else torch.bfloat16,
                              device=self.device)
        mhp = hp.shape[1] if hp.dim() == 2 else 0
        if shared_hist_pages:
            _check(_lib.oscar_decode_step_shared(self._h, layer, sl.numel(), _ptr(q), _ptr(k), _ptr(v), _ptr(sl),
                                                 _ptr(hp), mhp, int(shared_hist_pages), _ptr(bp), float(sm_scale),
                                                 _ptr(out), out_dtype, _ptr(lse), _stream(stream)),
                   "oscar_decode_step_shared")
        else:
            _check(_lib.oscar_decode_step(self._h, layer, sl.numel(), _ptr(q), _ptr(k), _ptr(v), _ptr(sl), _ptr(hp),
                                          mhp, _ptr(bp), float(sm_scale), _ptr(out), out_dtype, _ptr(lse),
                                          _stream(stream)), "oscar_decode_step")
        return out

    # ---- a prompt over itself ----------------------------------------------------------
    def prompt_attention(self, q, k, v, cu_seqlens, sm_scale: float, out=None, out_dtype: int = OUT_BF16, lse=None,
                         stream=None):
        """Causal attention of whole prompts, packed one behind the other as for quantize_prefill: q [N, Hq, 128],
        k, v [N, Hkv, 128] with free token and head strides (views of one projection), cu_seqlens [B + 1]. Rows of tokens
        that belong to no prompt stay as they are: a new out holds them unset. Returns out [N, Hq, 128]."""
        if stream is not None:
            with _on(stream):
                return self.prompt_attention(q, k, v, cu_seqlens, sm_scale, out, out_dtype, lse)
        what = "oscar_prompt_attention"
        dev, st = _here(self.pool)
        cu = _in_i32(cu_seqlens, dev)
        N, d = int(q.shape[0]), self.cfg.head_dim
        heads = []
        for x, h in ((q, self.cfg.num_q_heads), (k, self.cfg.num_kv_heads), (v, self.cfg.num_kv_heads)):
            if x.dtype is not _bf16 or x.get_device() != dev or x.shape != (N, h, d) or x.stride(2) != 1:
                raise OscarError(ERR_INVALID_ARG, what)
            heads.append(Heads(x.data_ptr(), x.stride(0), x.stride(1)))
        rows, out_type = (N, self.cfg.num_q_heads, d), _f32 if out_dtype == OUT_FP32 else _bf16
        if cu.dim() != 1 or cu.numel() < 1 or N >> 31:
            raise OscarError(ERR_INVALID_ARG, what)
        if out is None:
            out = _empty(rows, dtype=out_type, device=dev)
        else:
            _check_like(out, out_type, rows, dev, what)
        if lse is not None:
            _check_like(lse, _f32, rows[:2], dev, what)
        _check(_lib.oscar_prompt_attention(self._h, cu.numel() - 1, heads[0], heads[1], heads[2], cu.data_ptr(), N,
                                           float(sm_scale), out.data_ptr(), out_dtype, _ptr(lse), st), what)
        return out

    # ---- a token's raw projections ---------------------------------------------------
    def _raw_step(self, plan, q, k, v, q_weight, k_weight, eps, positions, layout, q_out, B: int, dev: int, what: str):
        """(RawStep, q_out, what has to live until the call) of raw rows q [B, Hq, 128] (or None), k and v [B, Hkv, 128]."""
        heads, d = (self.cfg.num_q_heads, self.cfg.num_kv_heads, self.cfg.num_kv_heads), self.cfg.head_dim
        rows = []
        for x, h in zip((q, k, v), heads):
            if x is None and not rows:   # no queries: k and v are appended
                rows.append(0)
                continue
            if x is None or x.dtype is not _bf16 or x.get_device() != dev or x.shape != (B, h, d):
                raise OscarError(ERR_INVALID_ARG, what)
            row, head, channel = x.stride()
            if channel != 1 or (h > 1 and head != d):
                raise OscarError(ERR_INVALID_ARG, what)
            rows.append(row if B > 1 else h * d)
        if q is not None:
            if q_out is None:
                q_out = _empty((B, heads[0], d), dtype=_bf16, device=dev)
            else:
                _check_like(q_out, _bf16, (B, heads[0], d), dev, what)
        pos = None
        if positions is None:
            if plan.turns.get_device() != dev:
                raise OscarError(ERR_INVALID_ARG, what)
        else:
            pos, n = plan.positions(positions, dev, what)
            if n != B:
                raise OscarError(ERR_INVALID_ARG, what)
        rotary = plan.rotary(layout)
        norm = None if eps is None else _head_norm(q_weight, k_weight, eps, _bf16, d, dev, what)
        step = RawStep(_ptr(q), k.data_ptr(), v.data_ptr(), *rows, _ptr(q_out), _ptr(pos), ctypes.addressof(rotary),
                       None if norm is None else ctypes.addressof(norm))
        return step, q_out, (rotary, norm, pos)

    def _step_tables(self, seq_lens, hist_pt, bf16_pt, dev: int, what: str):
        sl, hp, bp = _in_i32(seq_lens, dev), _in_i32(hist_pt, dev), _in_i32(bf16_pt, dev)
        B, mhp = sl.numel(), hp.shape[1] if hp.dim() == 2 else 0
        if hp.numel() != B * mhp or bp.numel() != B * ((self.cfg.sink + self.cfg.recent) // self.cfg.page_size):
            raise OscarError(ERR_INVALID_ARG, what)
        return sl, hp, bp, B, mhp

    def append_kv_rope(self, layer: int, plan: RopePlan, q, k, v, seq_lens_before, hist_pt, bf16_pt, q_weight=None,
                       k_weight=None, eps: float | None = 1e-6, positions=None, layout: int = ROPE_HALF, q_out=None,
                       stream=None):
        """append_kv of one token per request from its raw projections: norm_rope() of q [B, Hq, 128] (or None) and k
        [B, Hkv, 128] on the way (eps None: the rotation alone), at positions [B] ([num_axes, B] where the plan has axes),
        seq_lens_before by default. Rows of q, k and v may be views of one projection. Returns q_out, the queries for
        decode_attention."""
        if stream is not None:
            with _on(stream):
                return self.append_kv_rope(layer, plan, q, k, v, seq_lens_before, hist_pt, bf16_pt, q_weight, k_weight, eps,
                                           positions, layout, q_out)
        dev, st = _here(self.pool)
        sl, hp, bp, B, mhp = self._step_tables(seq_lens_before, hist_pt, bf16_pt, dev, "oscar_append_kv_rope")
        step, q_out, _keep = self._raw_step(plan, q, k, v, q_weight, k_weight, eps, positions, layout, q_out, B, dev,
                                            "oscar_append_kv_rope")
        _check(_lib.oscar_append_kv_rope(self._h, layer, B, step, sl.data_ptr(), hp.data_ptr(), mhp, bp.data_ptr(), st),
               "oscar_append_kv_rope")
        return q_out

    def decode_step_rope(self, layer: int, plan: RopePlan, q, k, v, seq_lens_before, hist_pt, bf16_pt, sm_scale: float,
                         q_weight=None, k_weight=None, eps: float | None = 1e-6, positions=None, layout: int = ROPE_HALF,
                         q_out=None, out=None, out_dtype: int = OUT_BF16, lse=None, stream=None,
                         shared_hist_pages: int = 0):
        """decode_step from raw projections, arguments as for append_kv_rope: the same three launches, with the norm and
        the rotation in the first. q_out [B, Hq, 128] receives the queries (allocated per call when not given)."""
        if stream is not None:
            with _on(stream):
                return self.decode_step_rope(layer, plan, q, k, v, seq_lens_before, hist_pt, bf16_pt, sm_scale, q_weight,
                                             k_weight, eps, positions, layout, q_out, out, out_dtype, lse,
                                             shared_hist_pages=shared_hist_pages)
        dev, st = _here(self.pool)
        sl, hp, bp, B, mhp = self._step_tables(seq_lens_before, hist_pt, bf16_pt, dev, "oscar_decode_step_rope")
        if q is None:
            raise OscarError(ERR_INVALID_ARG, "oscar_decode_step_rope")
        step, q_out, _keep = self._raw_step(plan, q, k, v, q_weight, k_weight, eps, positions, layout, q_out, B, dev,
                                            "oscar_decode_step_rope")
        rows, out_type = (B, self.cfg.num_q_heads, self.cfg.head_dim), _f32 if out_dtype == OUT_FP32 else _bf16
        if out is None:
            out = _empty(rows, dtype=out_type, device=dev)
        else:
            _check_like(out, out_type, rows, dev, "oscar_decode_step_rope")
        if lse is not None:
            _check_like(lse, _f32, rows[:2], dev, "oscar_decode_step_rope")
        _check(_lib.oscar_decode_step_rope(self._h, layer, B, step, sl.data_ptr(), hp.data_ptr(), mhp, int(shared_hist_pages),
                                           bp.data_ptr(), float(sm_scale), out.data_ptr(), out_dtype, _ptr(lse), st),
               "oscar_decode_step_rope")
        return out

    # ---- verifying drafted tokens -----------------------------------------------------
    def build_tables(self, old_lens, new_lens, hist_pt, bf16_pt, free_int2, free_bf16, rings, max_tokens: int = 0,
                     rings_out=None, cu_tokens=None, slots=None, stream=None):
        """Page tables and token slots of requests growing (or released) from old_lens, the lengths the last call left,
        to new_lens; the tables and the free rings are int32 device tensors updated in place, the ring positions too
        unless rings_out is given. A draft needs no pages: grow by what was accepted of it.
        With max_tokens, or a slots tensor [max_tokens, 4], each new token's (position, region, page, row) is
        written. Returns (rings_out, cu_tokens, slots)."""
        if stream is not None:
            with _on(stream):
                return self.build_tables(old_lens, new_lens, hist_pt, bf16_pt, free_int2, free_bf16, rings, max_tokens,
                                         rings_out, cu_tokens, slots)
        dev, st = _here(self.pool)
        old, new = _in_i32(old_lens, dev), _in_i32(new_lens, dev)
        B = old.numel()
        _own_i32(hist_pt, 0, dev)
        _own_i32(bf16_pt, B * (self.cfg.sink + self.cfg.recent) // self.cfg.page_size, dev)
        _own_i32(free_int2, self.cfg.num_int2_pages, dev)
        _own_i32(free_bf16, self.cfg.num_bf16_pages, dev)
        _own_i32(rings, 4, dev)
        rings_out = rings if rings_out is None else _own_i32(rings_out, 4, dev)
        cu_tokens = _empty(B + 1, dtype=_i32, device=dev) if cu_tokens is None else \
            _own_i32(cu_tokens, B + 1, dev)
        if slots is None and max_tokens:
            slots = _empty(max_tokens, 4, dtype=_i32, device=dev)
        if slots is not None:
            max_tokens = _own_i32(slots, 0, dev).numel() // 4
        if new.numel() != B or hist_pt.dim() != 2 or hist_pt.shape[0] != B:
            raise OscarError(ERR_INVALID_ARG, "oscar_build_tables")
        _check(_lib.oscar_build_tables(self._h, B, old.data_ptr(), new.data_ptr(), hist_pt.data_ptr(), hist_pt.shape[1],
                                       bf16_pt.data_ptr(), free_int2.data_ptr(), free_bf16.data_ptr(),
                                       rings.data_ptr(), rings_out.data_ptr(), cu_tokens.data_ptr(), _ptr(slots),
                                       max_tokens, st), "oscar_build_tables")
        return rings_out, cu_tokens, slots

    def tree_layout(self, parents, seq_lens, n_draft=None, mask=None, positions=None, stream=None):
        """Ancestor masks (int64 [B, T, ceil(T / 64)], 64 nodes a word) and positions (int32 [B, T]) of the trees
        given by parents [B, T]."""
        if stream is not None:
            with _on(stream):
                return self.tree_layout(parents, seq_lens, n_draft, mask, positions)
        dev, st = _here(self.pool)
        pa, sl = _in_i32(parents, dev), _in_i32(seq_lens, dev)
        nd = None if n_draft is None else _in_i32(n_draft, dev)
        if pa.dim() != 2 or sl.numel() != pa.shape[0] or (nd is not None and nd.numel() != pa.shape[0]):
            raise OscarError(ERR_INVALID_ARG, "oscar_tree_layout")
        B, T = pa.shape
        if mask is None:
            mask = _empty((B, T, (T + 63) // 64), dtype=_words[0], device=dev)
        else:
            _check_words(mask, B, T, dev, "oscar_tree_layout")
        if positions is None:
            positions = _empty((B, T), dtype=_i32, device=dev)
        else:
            _own_i32(positions, B * T, dev)
        _check(_lib.oscar_tree_layout(self._h, B, T, pa.data_ptr(), _ptr(nd), sl.data_ptr(), mask.data_ptr(),
                                      positions.data_ptr(), st), "oscar_tree_layout")
        return mask, positions

    def tree_workspace_bytes(self, batch: int, T: int, max_hist_pages: int) -> int:
        n = ctypes.c_size_t()
        _check(_lib.oscar_tree_workspace_bytes(self._h, batch, T, max_hist_pages, ctypes.byref(n)),
               "oscar_tree_workspace_bytes")
        return n.value

    def tree_attention(self, layer: int, q, k_draft, v_draft, mask, seq_lens, hist_pt, bf16_pt, sm_scale: float,
                       n_draft=None, out=None, out_dtype: int = OUT_BF16, lse=None, workspace=None, stream=None):
        """Attention of drafted nodes q [B, T, Hq, 128] over the cache's seq_lens tokens and, by mask, the drafted
        k_draft, v_draft [B, T, Hkv, 128]. A NaN or infinity in a row of q makes that row NaN. workspace: a uint8 tensor of tree_workspace_bytes, allocated per call
        when not given; calls that may overlap need one each."""
        if stream is not None:
            with _on(stream):
                return self.tree_attention(layer, q, k_draft, v_draft, mask, seq_lens, hist_pt, bf16_pt, sm_scale,
                                           n_draft, out, out_dtype, lse, workspace)
        dev, st = _here(self.pool)
        sl, hp, bp = _in_i32(seq_lens, dev), _in_i32(hist_pt, dev), _in_i32(bf16_pt, dev)
        nd = None if n_draft is None else _in_i32(n_draft, dev)
        if q.dim() != 4:
            raise OscarError(ERR_INVALID_ARG, "oscar_tree_attention")
        B, T = int(q.shape[0]), int(q.shape[1])
        rows = (B, T, self.cfg.num_q_heads, self.cfg.head_dim)
        drafted = (B, T, self.cfg.num_kv_heads, self.cfg.head_dim)
        _check_like(q, _bf16, rows, dev, "oscar_tree_attention")
        _check_like(k_draft, _bf16, drafted, dev, "oscar_tree_attention")
        _check_like(v_draft, _bf16, drafted, dev, "oscar_tree_attention")
        _check_words(mask, B, T, dev, "oscar_tree_attention")
        mhp = hp.shape[1] if hp.dim() == 2 else 0
        if sl.numel() != B or (nd is not None and nd.numel() != B) or hp.numel() != B * mhp or \
                bp.numel() != B * ((self.cfg.sink + self.cfg.recent) // self.cfg.page_size):
            raise OscarError(ERR_INVALID_ARG, "oscar_tree_attention")
        out_type = _f32 if out_dtype == OUT_FP32 else _bf16
        if out is None:
            out = _empty(rows, dtype=out_type, device=dev)
        else:
            _check_like(out, out_type, rows, dev, "oscar_tree_attention")
        if lse is not None:
            _check_like(lse, _f32, rows[:3], dev, "oscar_tree_attention")
        if workspace is None:
            workspace = self.pool.new_empty(self.tree_workspace_bytes(B, T, mhp))
        elif workspace.get_device() != dev or not workspace.is_contiguous():
            raise OscarError(ERR_INVALID_ARG, "oscar_tree_attention")
        _check(_lib.oscar_tree_attention(self._h, layer, B, T, q.data_ptr(), k_draft.data_ptr(), v_draft.data_ptr(),
                                         mask.data_ptr(), _ptr(nd), sl.data_ptr(), hp.data_ptr(), mhp, bp.data_ptr(),
                                         float(sm_scale), out.data_ptr(), out_dtype, _ptr(lse), workspace.data_ptr(),
                                         workspace.nbytes, st), "oscar_tree_attention")
        return out

    def commit_draft(self, layer: int, k_draft, v_draft, seq_lens_before, n_accept, hist_pt, bf16_pt, path=None,
                     max_accept: int | None = None, stream=None):
        """Append nodes path[r, :n_accept[r]] of k_draft, v_draft [B, T, Hkv, 128] at seq_lens_before[r]; without a
        path nodes 0 .. n_accept[r] - 1 (max_accept of them at most, T by default)."""
        if stream is not None:
            with _on(stream):
                return self.commit_draft(layer, k_draft, v_draft, seq_lens_before, n_accept, hist_pt, bf16_pt, path,
                                         max_accept)
        dev, st = _here(self.pool)
        sl, na = _in_i32(seq_lens_before, dev), _in_i32(n_accept, dev)
        hp, bp = _in_i32(hist_pt, dev), _in_i32(bf16_pt, dev)
        pa = None if path is None else _in_i32(path, dev)
        if k_draft.dim() != 4:
            raise OscarError(ERR_INVALID_ARG, "oscar_commit_draft")
        B, T = int(k_draft.shape[0]), int(k_draft.shape[1])
        drafted = (B, T, self.cfg.num_kv_heads, self.cfg.head_dim)
        _check_like(k_draft, _bf16, drafted, dev, "oscar_commit_draft")
        _check_like(v_draft, _bf16, drafted, dev, "oscar_commit_draft")
        mhp = hp.shape[1] if hp.dim() == 2 else 0
        if sl.numel() != B or na.numel() != B or hp.numel() != B * mhp or \
                bp.numel() != B * ((self.cfg.sink + self.cfg.recent) // self.cfg.page_size) or \
                (pa is not None and (pa.dim() != 2 or pa.shape[0] != B)):
            raise OscarError(ERR_INVALID_ARG, "oscar_commit_draft")
        if pa is not None:
            max_accept = pa.shape[1]
        elif max_accept is None:
            max_accept = T
        _check(_lib.oscar_commit_draft(self._h, layer, B, T, k_draft.data_ptr(), v_draft.data_ptr(), sl.data_ptr(),
                                       na.data_ptr(), max_accept, _ptr(pa), hp.data_ptr(), mhp, bp.data_ptr(), st),
               "oscar_commit_draft")

    def set_decode_algo(self, algo: int):
        _check(_lib.oscar_set_decode_algo(self._h, algo), "oscar_set_decode_algo")

    def get_status(self) -> int:
        code = ctypes.c_int()
        rc = _lib.oscar_get_status(self._h, ctypes.byref(code))
        if rc not in (OK, ERR_DEVICE_STATUS):
            raise OscarError(rc, "oscar_get_status")
        return code.value

    def pack_rotated(self, layer: int, kind: int, xrot, page_ids, rows, stream=None):
        pi = _dev_i32(page_ids, self.device)
        ro = _dev_i32(rows, self.device)
        _check(_lib.oscar_pack_rotated(self._h, layer, kind, _ptr(xrot), _ptr(pi), _ptr(ro), pi.numel(),
                                       _stream(stream)), "oscar_pack_rotated")

    def rotate(self, layer: int, kind: int, x, stream=None):
        import torch
        y = torch.empty(x.shape, dtype=torch.float32, device=self.device)
        _check(_lib.oscar_rotate(self._h, layer, kind, _ptr(x), _ptr(y), int(x.shape[0]), _stream(stream)),
               "oscar_rotate")
        return y

    def trace_ctas(self, buf=None):
        """Record per-CTA timelines of following tensor-core decode launches into ``buf`` (an int64 device
        tensor of 8 * n elements, n records); None stops recording."""
        n = 0 if buf is None else buf.numel() // 8
        _check(_lib.oscar_trace_ctas(self._h, _ptr(buf), n), "oscar_trace_ctas")

    def check_wait_timeout(self, stream=None):
        """Run the bounded-wait self-check: a device wait that nothing completes must give up (about 2 s)
        and set the TIMEOUT bit of the status word."""
        _check(_lib.oscar_check_wait_timeout(self._h, _stream(stream)), "oscar_check_wait_timeout")

    def trace_timeline(self, buf=None):
        """Record a timeline of every CTA of the following kernel launches into ``buf`` (an int64 device tensor
        of 4 + 4 * n elements, n records, buf[0] zeroed by the caller); None stops recording."""
        n = 0 if buf is None else (buf.numel() - 4) // 4
        _check(_lib.oscar_trace_timeline(self._h, _ptr(buf), n), "oscar_trace_timeline")

    def profile_begin(self, capacity: int):
        _check(_lib.oscar_profile_begin(self._h, capacity), "oscar_profile_begin")

    def profile_read(self) -> tuple[float, int]:
        ms, n = ctypes.c_double(), ctypes.c_int()
        _check(_lib.oscar_profile_read(self._h, ctypes.byref(ms), ctypes.byref(n)), "oscar_profile_read")
        return ms.value, n.value


def bf16_decode_workspace_bytes(max_batch: int, num_q_heads: int, max_splits: int) -> int:
    n = ctypes.c_size_t()
    _check(_lib.oscar_bf16_decode_workspace_bytes(max_batch, num_q_heads, max_splits, ctypes.byref(n)),
           "oscar_bf16_decode_workspace_bytes")
    return n.value


def bf16_decode(kv_pages, q, seq_lens, page_table, sm_scale: float, num_kv_heads: int, workspace, max_splits: int,
                out=None, out_dtype: int = OUT_BF16, lse=None, stream=None):
    """Decode over an all-BF16 paged cache kv_pages [num_pages, Hkv, 2, 64, 128] bf16."""
    import torch
    B, hq = int(q.shape[0]), int(q.shape[1])
    if out is None:
        out = torch.empty(q.shape, dtype=torch.float32 if out_dtype == OUT_FP32 else torch.bfloat16, device=q.device)
    sl = _dev_i32(seq_lens, q.device)
    pt = _dev_i32(page_table, q.device)
    _check(_lib.oscar_bf16_decode(B, hq, num_kv_heads, _ptr(kv_pages), int(kv_pages.shape[0]), _ptr(q), _ptr(sl),
                                  _ptr(pt), int(pt.shape[1]), float(sm_scale), _ptr(out), out_dtype, _ptr(lse),
                                  _ptr(workspace), workspace.numel() * workspace.element_size(), max_splits,
                                  _stream(stream)), "oscar_bf16_decode")
    return out


class RopePlan:
    """Rotary frequencies of a head's first rotary_dim channels (ROPE_* scaling) in the form rope() reads, on a
    device; inv_freq (float64, radians per position and pair) may be given instead of the base and its scaling.
    axes: for positions with several axes (time, height, width) the axis of every pair, for instance
    np.repeat([0, 1, 2], [16, 24, 24]); positions are then int32 [num_axes, N]."""

    def __init__(self, rotary_dim: int, base: float = 10000.0, scaling: int = ROPE_NONE, factor: float = 1.0,
                 original_length: float = 0.0, beta_fast: float = 32.0, beta_slow: float = 1.0, inv_freq=None,
                 scale: float | None = None, device="cuda", axes=None):
        import torch
        self.rotary_dim = int(rotary_dim)
        f = np.zeros(max(1, self.rotary_dim // 2), np.float64)
        s = ctypes.c_float(1.0)
        if inv_freq is None:
            _check(_lib.oscar_rope_frequencies(self.rotary_dim, base, scaling, factor, original_length, beta_fast,
                                               beta_slow, _ptr(f), ctypes.byref(s)), "oscar_rope_frequencies")
        else:
            f = np.ascontiguousarray(inv_freq, np.float64)
            if f.shape != (self.rotary_dim // 2,):
                raise OscarError(ERR_INVALID_ARG, "RopePlan: one frequency per pair")
        turns = np.zeros(f.shape, np.uint64)
        _check(_lib.oscar_rope_turns(_ptr(f), f.size, _ptr(turns)), "oscar_rope_turns")
        self.inv_freq, self.scale = f, float(s.value) if scale is None else float(scale)
        self.turns = torch.from_numpy(turns.view(np.int64)).to(device)
        self.axes, self.num_axes = None, 1
        if axes is not None:
            a = np.asarray(axes)
            if a.shape != f.shape or a.dtype.kind not in "iu" or a.min() < 0 or a.max() >= MAX_ROPE_AXES:
                raise OscarError(ERR_INVALID_ARG, "RopePlan: one axis per pair, 0 .. MAX_ROPE_AXES - 1")
            self.num_axes = int(a.max()) + 1
            self.axes = torch.from_numpy(a.astype(np.uint8)).to(device)

    def rotary(self, layout: int) -> Rotary:
        return Rotary(self.turns.data_ptr(), None if self.axes is None else self.axes.data_ptr(), self.num_axes,
                      self.rotary_dim, layout, self.scale)

    def positions(self, positions, dev: int, what: str):
        """(positions, tokens): int32 [N], or [num_axes, N] where the plan has axes."""
        pos = _in_i32(positions, dev)
        if self.turns.get_device() != dev or (self.axes is not None and (pos.dim() != 2 or pos.shape[0] != self.num_axes)):
            raise OscarError(ERR_INVALID_ARG, what)
        return pos, pos.numel() if self.axes is None else pos.shape[1]


def _rows_code(dtype, what: str) -> int:
    code = DTYPE_BF16 if dtype is _bf16 else DTYPE_FP32 if dtype is _f32 else DTYPE_FP16
    if code == DTYPE_FP16 and dtype is not _f16:
        raise OscarError(ERR_INVALID_ARG, what)
    return code


def _rows(pairs, dtype, n: int, dim: int, dev: int, what: str):
    """RopeTensors of (rows, results) pairs: rows [n, heads, dim] or None, results None for a new tensor."""
    args, outs = [], []
    for x, out in pairs:
        if x is None:
            args.append(RopeTensor())
            outs.append(None)
            continue
        shape = x.shape                            # asked for once: a tensor's attribute costs 0.1 us
        if x.dtype is not dtype or x.get_device() != dev or len(shape) != 3:
            raise OscarError(ERR_INVALID_ARG, what)
        tokens, heads, channels = shape
        if out is None:
            out = _empty(shape, dtype=dtype, device=dev)
        elif out.dtype is not dtype or out.get_device() != dev or out.shape != shape:
            raise OscarError(ERR_INVALID_ARG, what)
        (it, ih, ic), (ot, oh, oc) = x.stride(), out.stride()
        if tokens != n or channels != dim or (dim > 1 and (ic != 1 or oc != 1)):
            raise OscarError(ERR_INVALID_ARG, what)
        args.append(RopeTensor(x.data_ptr(), out.data_ptr(), it, ih, ot, oh, heads))
        outs.append(out)
    return args, outs


def rope(plan: RopePlan, q, k, positions, layout: int = ROPE_HALF, inverse: bool = False, q_out=None, k_out=None,
         stream=None):
    """Rotate q [N, Hq, D] and k [N, Hkv, D] (k may be None) by positions [N], or [num_axes, N] where the plan has axes;
    inverse gives the gradient. Token and head strides are free, a head's channels contiguous. Written to q_out, k_out
    (new tensors when not given; the inputs themselves for in place). Rows with a negative position (on any axis) are
    left as they are: new tensors hold them unset. Returns (q_out, k_out)."""
    if stream is not None:
        with _on(stream):
            return rope(plan, q, k, positions, layout, inverse, q_out, k_out)
    dev, st = _here(q)
    pos = _in_i32(positions, dev)
    dtype, shape, n = q.dtype, q.shape, pos.numel()
    if plan.axes is not None:
        pos, n = plan.positions(pos, dev, "oscar_rope_axes")
    code = DTYPE_BF16 if dtype is _bf16 else DTYPE_FP32 if dtype is _f32 else DTYPE_FP16
    if (code == DTYPE_FP16 and dtype is not _f16) or plan.turns.get_device() != dev or len(shape) != 3 or n >> 31:
        raise OscarError(ERR_INVALID_ARG, "oscar_rope")
    dim = shape[2]
    args, outs = _rows(((q, q_out), (k, k_out)), dtype, n, dim, dev, "oscar_rope")
    if plan.axes is None:
        _check(_lib.oscar_rope(args[0], args[1], n, dim, code, pos.data_ptr(), plan.turns.data_ptr(), plan.rotary_dim,
                               layout, plan.scale, inverse, st), "oscar_rope")
    else:
        _check(_lib.oscar_rope_axes(args[0], args[1], n, dim, code, pos.data_ptr(), plan.rotary(layout), inverse, st),
               "oscar_rope_axes")
    return outs[0], outs[1]


def _head_norm(q_weight, k_weight, eps: float, dtype, dim: int, dev: int, what: str) -> HeadNorm:
    for w in (q_weight, k_weight):
        if w is not None:
            _check_like(w, dtype, (dim,), dev, what)
    return HeadNorm(_ptr(q_weight), _ptr(k_weight), eps)


def norm_rope(plan: RopePlan, q, k, positions, q_weight=None, k_weight=None, eps: float = 1e-6, layout: int = ROPE_HALF,
              q_out=None, k_out=None, stream=None):
    """Root-mean-square norm of every head's row of q and k, times the weight [D] (of the rows' dtype; None: ones), then
    rope() of the result, in one pass. Arguments and results as for rope()."""
    if stream is not None:
        with _on(stream):
            return norm_rope(plan, q, k, positions, q_weight, k_weight, eps, layout, q_out, k_out)
    dev, st = _here(q)
    pos, n = plan.positions(positions, dev, "oscar_norm_rope")
    dtype, shape = q.dtype, q.shape
    code = _rows_code(dtype, "oscar_norm_rope")
    if len(shape) != 3 or n >> 31:
        raise OscarError(ERR_INVALID_ARG, "oscar_norm_rope")
    norm = _head_norm(q_weight, k_weight, eps, dtype, shape[2], dev, "oscar_norm_rope")
    args, outs = _rows(((q, q_out), (k, k_out)), dtype, n, shape[2], dev, "oscar_norm_rope")
    _check(_lib.oscar_norm_rope(args[0], args[1], n, shape[2], code, pos.data_ptr(), plan.rotary(layout), norm, st),
           "oscar_norm_rope")
    return outs[0], outs[1]


def norm_rope_backward(plan: RopePlan, q, k, positions, grad_q, grad_k, q_weight=None, k_weight=None, eps: float = 1e-6,
                       layout: int = ROPE_HALF, dq=None, dk=None, weight_grads: bool = True, workspace=None, stream=None):
    """Gradient of norm_rope() for the same q, k (k and grad_k may be None), positions and weights, from the gradients
    grad_q, grad_k by its results. Returns (dq, dk, dq_weight, dk_weight): dq, dk of the rows' dtype (they may be grad_q
    and grad_k, or q and k; rows with a negative position stay as they are), the weights' gradients float32 [D] (None
    without weight_grads; the weight of a k that is None gets zeros). workspace: a uint8 tensor of
    norm_rope_workspace_bytes(D), allocated per call when not given; calls that may overlap need one each."""
    if stream is not None:
        with _on(stream):
            return norm_rope_backward(plan, q, k, positions, grad_q, grad_k, q_weight, k_weight, eps, layout, dq, dk,
                                      weight_grads, workspace)
    what = "oscar_norm_rope_backward"
    dev, st = _here(q)
    pos, n = plan.positions(positions, dev, what)
    dtype, shape = q.dtype, q.shape
    code = _rows_code(dtype, what)
    if len(shape) != 3 or n >> 31 or grad_q is None or (k is None) != (grad_k is None):
        raise OscarError(ERR_INVALID_ARG, what)
    dim = shape[2]
    norm = _head_norm(q_weight, k_weight, eps, dtype, dim, dev, what)
    args, outs = _rows(((q, dq), (k, dk)), dtype, n, dim, dev, what)
    grads = []
    for x, g in ((q, grad_q), (k, grad_k)):
        if g is None:
            grads.append(RopeTensor())
            continue
        rows = x.shape                             # three numbers: _rows
        if g.dtype is not dtype or g.get_device() != dev or g.shape != rows:
            raise OscarError(ERR_INVALID_ARG, what)
        token, head, channel = g.stride()
        if channel != 1:
            raise OscarError(ERR_INVALID_ARG, what)
        grads.append(RopeTensor(g.data_ptr(), None, token, head, 0, 0, rows[1]))
    dqw = dkw = ws = None
    ws_bytes = 0
    if weight_grads:
        dqw, dkw = _empty(dim, dtype=_f32, device=dev), _empty(dim, dtype=_f32, device=dev)
        if workspace is None:
            ws_bytes = norm_rope_workspace_bytes(dim)
            ws = _empty(ws_bytes, dtype=_u8, device=dev)
        else:
            ws, ws_bytes = workspace, workspace.nbytes
            if ws.get_device() != dev or not ws.is_contiguous():
                raise OscarError(ERR_INVALID_ARG, what)
    _check(_lib.oscar_norm_rope_backward(args[0], args[1], grads[0], grads[1], n, dim, code, pos.data_ptr(),
                                         plan.rotary(layout), norm, None if dqw is None else dqw.data_ptr(),
                                         None if dkw is None else dkw.data_ptr(), None if ws is None else ws.data_ptr(),
                                         ws_bytes, st), what)
    return outs[0], outs[1], dqw, dkw


_norm_rope_workspace = {}                          # head_dim: bytes, which depend on nothing else


def norm_rope_workspace_bytes(head_dim: int) -> int:
    if head_dim not in _norm_rope_workspace:
        n = ctypes.c_size_t()
        _check(_lib.oscar_norm_rope_workspace_bytes(head_dim, ctypes.byref(n)), "oscar_norm_rope_workspace_bytes")
        _norm_rope_workspace[head_dim] = n.value
    return _norm_rope_workspace[head_dim]


def calibrate_codebook(x_rot, tau) -> np.ndarray:
    """Host Lloyd-Max calibration of one codebook from rotated float32 rows x_rot [N, 128] and clip
    thresholds tau [128]: returns the codebook bytes uint8 [4]."""
    x = np.ascontiguousarray(x_rot, dtype=np.float32)
    t = np.ascontiguousarray(tau, dtype=np.float32)
    out = np.zeros(4, np.uint8)
    _check(_lib.oscar_calibrate_codebook(_ptr(x), x.shape[0], _ptr(t), _ptr(out)), "oscar_calibrate_codebook")
    return out


def calibrate(Q, K, V, sm_scale: float, c_K: float = 0.96, c_V: float = 0.92):
    """Host calibration of one (layer, kv head): returns dict with U_K, U_V [128,128], tau_K, tau_V [128] float32
    and eig_K, eig_V [128] float64."""
    q = np.ascontiguousarray(Q, dtype=np.float32)
    k = np.ascontiguousarray(K, dtype=np.float32)
    v = np.ascontiguousarray(V, dtype=np.float32)
    out = {n: np.zeros((128, 128), np.float32) for n in ("U_K", "U_V")}
    out.update({n: np.zeros(128, np.float32) for n in ("tau_K", "tau_V")})
    out.update({n: np.zeros(128, np.float64) for n in ("eig_K", "eig_V")})
    _check(_lib.oscar_calibrate(_ptr(q), _ptr(k), _ptr(v), q.shape[0], float(sm_scale), float(c_K), float(c_V),
                                _ptr(out["U_K"]), _ptr(out["U_V"]), _ptr(out["tau_K"]), _ptr(out["tau_V"]),
                                _ptr(out["eig_K"]), _ptr(out["eig_V"])), "oscar_calibrate")
    return out


def decode_attention_noalloc(cfg: CacheConfig, pool, layer: int, q, seq_lens, hist_pt, bf16_pt, sm_scale: float,
                             out=None, out_dtype: int = OUT_BF16, lse=None, status=None, stream=None):
    """Decode attention through the allocation-free entry point, for callers that cannot allocate device
    memory (for instance inside CUDA graph capture): same result as OscarCache.decode_attention, with the
    cache given by its config and pool tensor, scratch in the library's fixed device array, and the call's
    status bits written to ``status`` (an int32 device tensor of one element) when given. Calls that may
    overlap on the GPU share that scratch and must not be issued concurrently."""
    import torch
    dev = pool.device
    sl = _dev_i32(seq_lens, dev)
    hp = _dev_i32(hist_pt, dev)
    bp = _dev_i32(bf16_pt, dev)
    if out is None:
        out = torch.empty(q.shape, dtype=torch.float32 if out_dtype == OUT_FP32 else torch.bfloat16, device=dev)
    lay = cfg.layout()
    _check(_lib.oscar_decode_attention_noalloc(ctypes.byref(lay), _ptr(pool), layer, sl.numel(), _ptr(q), _ptr(sl),
                                               _ptr(hp), hp.shape[1] if hp.dim() == 2 else 0, _ptr(bp),
                                               float(sm_scale), _ptr(out), out_dtype, _ptr(lse), _ptr(status),
                                               _stream(stream)), "oscar_decode_attention_noalloc")
    return out
