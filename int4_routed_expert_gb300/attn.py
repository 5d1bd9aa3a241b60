"""ctypes binding of include/moe_attn.h: rotary positions, the 8-bit paged cache and attention over it.

A decoder layer next to the MoE layer calls, per step:
    q, k = rope.apply(q, positions, k=k)         # Rope
    cache.write(k, v, batch)                      # KVCache: quantise into the pages
    out = cache.attend(q, batch)                  # attention over the cache, the new tokens included
``SeqBatch`` describes the step's tokens (device arrays and the host's bounds).  As in moe.py, torch supplies
device memory and streams only; every step runs in the library's kernels and there is no fallback.
Calls run on torch's current stream, or on ``stream``, whose memory their results are then; that the inputs are
ready there, and stay until it has run, is the caller's to see to, as with every other stream of torch.
"""
from __future__ import annotations

import ctypes as C
import math
from threading import get_ident

from . import moe
from .moe import MOE_BF16, MOE_F32, MOE_OK, MoeError


class moe_rope_tensor_t(C.Structure):
    _fields_ = [("x", C.c_void_p), ("y", C.c_void_p), ("n_heads", C.c_int), ("x_stride", C.c_int64),
                ("y_stride", C.c_int64)]


class moe_kv_config_t(C.Structure):
    _fields_ = [(n, C.c_int) for n in ("n_q_heads", "n_kv_heads", "head_dim", "page_size", "n_pages", "max_seqs",
                                       "max_tokens", "max_kv_len")]


class moe_kv_store_t(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("k", "v", "k_scale", "v_scale")]


class moe_kv_batch_t(C.Structure):
    _fields_ = [(n, C.c_int) for n in ("n_seqs", "n_tokens", "max_q_len", "max_kv_len", "table_stride")] + \
               [(n, C.c_void_p) for n in ("cu_q", "kv_len", "page_table")]


class moe_kv_mask_t(C.Structure):
    _fields_ = [("scale", C.c_float), ("causal", C.c_int), ("window", C.c_int), ("sinks", C.c_int)]


EXPORTED = ("moe_rope_create", "moe_rope_apply", "moe_rope_destroy", "moe_kv_create", "moe_kv_workspace_bytes",
            "moe_kv_last_error", "moe_kv_destroy", "moe_kv_write", "moe_kv_read", "moe_kv_attend",
            "moe_kv_device_status")

# bits of moe_kv_device_status
KV_WAIT_GAVE_UP, KV_BAD_BATCH, KV_NON_FINITE = 1, 2, 4

_lib = None
torch = None    # imported with the library: a call costs a few microseconds, and a module lookup is part of it
_codes = {}     # torch dtype -> moe_dtype_t
_raw_stream = None
_int32 = None


def _load() -> C.CDLL:
    global _lib, torch, _raw_stream, _int32
    if _lib is not None:
        return _lib
    import torch as _torch
    L = moe.load()
    vp, i32, i64 = C.c_void_p, C.c_int, C.c_int64
    sig = {
        "moe_rope_create": (i32, [i32, C.POINTER(C.c_double), C.c_float, i32, C.POINTER(vp)]),
        "moe_rope_apply": (i32, [vp, C.POINTER(moe_rope_tensor_t), C.POINTER(moe_rope_tensor_t), i32, i32, vp, i32, vp]),
        "moe_rope_destroy": (None, [vp]),
        "moe_kv_create": (i32, [C.POINTER(moe_kv_config_t), C.POINTER(moe_kv_store_t), C.POINTER(vp)]),
        "moe_kv_workspace_bytes": (C.c_size_t, [C.POINTER(moe_kv_config_t)]),
        "moe_kv_last_error": (C.c_char_p, [vp]),
        "moe_kv_destroy": (None, [vp]),
        "moe_kv_write": (i32, [vp, vp, i64, vp, i64, i32, C.POINTER(moe_kv_batch_t), vp]),
        "moe_kv_read": (i32, [vp, vp, vp, i32, C.POINTER(moe_kv_batch_t), vp]),
        "moe_kv_attend": (i32, [vp, vp, i64, vp, vp, C.POINTER(moe_kv_mask_t), C.POINTER(moe_kv_batch_t), vp]),
        "moe_kv_device_status": (i32, [vp, C.POINTER(C.c_int32)]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype, fn.argtypes = res, args
    torch = _torch
    _int32 = torch.int32
    _codes.update({torch.bfloat16: MOE_BF16, torch.float32: MOE_F32})
    # the stream's handle alone; torch.cuda.current_stream() builds an object, 3 us
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
        (lambda index: torch.cuda.current_stream(index).cuda_stream)
    _lib = L
    return L


def _dtype(t, name: str) -> int:
    code = _codes.get(t)
    if code is None:
        raise TypeError(f"{name} must be fp32 or bf16, got {t}")
    return code


def _stream(stream, index: int) -> int:
    return _raw_stream(index) if stream is None else stream.cuda_stream


def _results(shape, dtype, device, stream):
    """A result tensor in memory of the stream that writes it: memory of another one may still be in use there,
    and be given away there before the call's kernels have run."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _rows(x, name: str, heads: int, dim: int, device) -> int:
    """Checks a [tokens][heads][dim] (or [tokens][heads * dim]) CUDA tensor whose tokens may be strided and
    whose rows are whole; returns the elements between tokens."""
    shape, stride = x.shape, x.stride()
    if len(shape) == 3:
        ok = shape[1] == heads and shape[2] == dim and stride[2] == 1 and (heads == 1 or stride[1] == dim)
    else:
        ok = len(shape) == 2 and shape[1] == heads * dim and stride[1] == 1
    if not ok or x.device != device:
        raise ValueError(f"{name} must be [tokens, {heads}, {dim}] on {device} with contiguous rows, got "
                         f"{tuple(shape)} with strides {stride} on {x.device}")
    return stride[0] if shape[0] > 1 else heads * dim


def rope_frequencies(rot_dim: int, theta: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                     original_len: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0):
    """Radians per position of each of rot_dim / 2 pairs, and the amplitude of their sine and cosine.
      None      theta^(-2i / rot_dim)
      "linear"  divided by factor (position interpolation)
      "ntk"     theta raised to theta * factor^(rot_dim / (rot_dim - 2))
      "yarn"    pairs that make more than beta_fast turns over original_len keep their frequency, those below
                beta_slow are divided by factor, a ramp between; amplitude 0.1 ln(factor) + 1
    """
    if scaling not in (None, "linear", "ntk", "yarn"):
        raise ValueError(f"scaling must be None, 'linear', 'ntk' or 'yarn', got {scaling!r}")
    if not theta > 1 or not factor >= 1:
        raise ValueError("theta must be above 1 and factor at least 1")
    half = rot_dim // 2
    base = theta * factor ** (rot_dim / (rot_dim - 2)) if scaling == "ntk" else theta
    f = [base ** (-2.0 * i / rot_dim) for i in range(half)]
    if scaling == "linear":
        return [x / factor for x in f], 1.0
    if scaling != "yarn":
        return f, 1.0
    if original_len < 1:
        raise ValueError("yarn needs original_len")

    def pair_of(turns: float) -> float:
        return rot_dim * math.log(original_len / (turns * 2 * math.pi)) / (2 * math.log(theta))

    low, high = max(math.floor(pair_of(beta_fast)), 0), min(math.ceil(pair_of(beta_slow)), rot_dim - 1)
    ramp = [min(max((i - low) / max(high - low, 1e-3), 0.0), 1.0) for i in range(half)]
    return [x * (1 - r) + x / factor * r for x, r in zip(f, ramp)], 0.1 * math.log(factor) + 1.0


class Rope:
    """Rotary positions (moe_rope_*).  Frequencies by rope_frequencies, or given (radians per position)."""

    def __init__(self, rot_dim: int, theta: float = 10000.0, interleaved: bool = False, scaling: str | None = None,
                 factor: float = 1.0, original_len: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0,
                 inv_freq=None, amplitude: float | None = None):
        self.h = None
        self._layouts = {}
        if inv_freq is None:
            inv_freq, amp = rope_frequencies(rot_dim, theta, scaling, factor, original_len, beta_fast, beta_slow)
        else:
            inv_freq, amp = [float(x) for x in inv_freq], 1.0
        if len(inv_freq) != rot_dim // 2:
            raise ValueError(f"inv_freq must have {rot_dim // 2} entries, got {len(inv_freq)}")
        self.rot_dim, self.interleaved = rot_dim, interleaved
        self.inv_freq, self.amplitude = inv_freq, amp if amplitude is None else amplitude
        h = C.c_void_p()
        st = _load().moe_rope_create(rot_dim, (C.c_double * max(1, len(inv_freq)))(*inv_freq), self.amplitude,
                                     1 if interleaved else 0, C.byref(h))
        if st != MOE_OK:
            raise MoeError(st, moe.moe_last_error(None))
        self.h = h

    def apply(self, q, positions, k=None, q_out=None, k_out=None, stream=None):
        """Rotates q [tokens, heads, head_dim] (and k) at positions [tokens] int32; returns q's result, or
        (q's, k's) when k is given.  Tokens may be strided (parts of one projection); q_out is q rotates in
        place."""
        if q_out is None and k_out is None:
            # the checks of a layout (shapes, strides, types) once: a call is a few microseconds; the argument
            # structs are a thread's own
            key = (get_ident(), q.shape, q.stride(), q.dtype) if k is None else \
                (get_ident(), q.shape, q.stride(), q.dtype, k.shape, k.stride(), k.dtype)
            known = self._layouts.get(key)
            if known is None:
                known = self._layout(key, q, k)
            T, D, dt, tq, tk, contiguous = known
            dev = q.get_device()
            if dev < 0 or positions.dtype is not _int32 or positions.shape != (T,) or positions.get_device() != dev \
                    or not positions.is_contiguous() or (tk is not None and k.get_device() != dev):
                self._refuse(q, k, positions)
            if stream is not None:
                q_out = _results(q.shape, q.dtype, q.device, stream)
                k_out = None if tk is None else _results(k.shape, k.dtype, k.device, stream)
            elif contiguous:
                q_out = torch.empty_like(q)
                k_out = None if tk is None else torch.empty_like(k)
            else:
                q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
                k_out = None if tk is None else torch.empty(k.shape, dtype=k.dtype, device=k.device)
        else:
            known = self._layout(None, q, k)
            T, D, dt, tq, tk, _ = known
            dev = q.get_device()
            if dev < 0 or positions.dtype is not _int32 or positions.shape != (T,) or positions.get_device() != dev \
                    or not positions.is_contiguous() or (tk is not None and k.get_device() != dev):
                self._refuse(q, k, positions)
            if k is None and k_out is not None:
                raise ValueError("k_out needs k")
            q_out, tq.y_stride = self._out("q", q, q_out, stream)
            if tk is not None:
                k_out, tk.y_stride = self._out("k", k, k_out, stream)
        if T:
            tq.x, tq.y = q.data_ptr(), q_out.data_ptr()
            if tk is not None:
                tk.x, tk.y = k.data_ptr(), k_out.data_ptr()
            st = _lib.moe_rope_apply(self.h, tq, tk, D, dt, positions.data_ptr(), T,
                                     _raw_stream(dev) if stream is None else stream.cuda_stream)
            if st != MOE_OK:
                raise MoeError(st, moe.moe_last_error(None))
        return q_out if tk is None else (q_out, k_out)

    def _layout(self, key, q, k):
        """(tokens, head_dim, dtype, q's and k's argument structs, contiguous) of a checked layout."""
        dev, dtype = q.device, q.dtype
        if q.dim() != 3 or not q.is_cuda:
            raise ValueError(f"q must be a CUDA tensor [tokens, heads, head_dim], got {tuple(q.shape)} on {dev}")
        T, H, D = q.shape
        dt = _dtype(dtype, "q")
        tq = moe_rope_tensor_t(None, None, H, _rows(q, "q", H, D, dev), H * D)
        tk, contiguous = None, q.is_contiguous()
        if k is not None:
            if k.dim() != 3 or k.shape[0] != T or k.shape[2] != D or k.dtype != dtype:
                raise ValueError(f"k must be [{T}, heads, {D}] of {dtype}")
            tk = moe_rope_tensor_t(None, None, k.shape[1], _rows(k, "k", k.shape[1], D, dev), k.shape[1] * D)
            contiguous = contiguous and k.is_contiguous()
        known = (T, D, dt, tq, tk, contiguous)
        if key is not None:
            if len(self._layouts) >= 64:
                self._layouts.clear()
            self._layouts[key] = known
        return known

    @staticmethod
    def _refuse(q, k, positions):
        if not q.is_cuda:
            raise ValueError(f"q must be a CUDA tensor [tokens, heads, head_dim], got {tuple(q.shape)} on {q.device}")
        if k is not None and k.device != q.device:
            raise ValueError(f"k must be on {q.device}, got {k.device}")
        raise ValueError(f"positions must be a contiguous int32 tensor of {q.shape[0]} entries on {q.device}")

    @staticmethod
    def _out(name, x, y, stream):
        T, H, D = x.shape
        if y is None:
            return _results((T, H, D), x.dtype, x.device, stream), H * D
        if y.shape != x.shape or y.dtype != x.dtype:
            raise ValueError(f"{name}_out must be {(T, H, D)} of {x.dtype}")
        return y, _rows(y, name + "_out", H, D, x.device)

    def close(self):
        if self.h:
            _load().moe_rope_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class SeqBatch:
    """The tokens of one call: sequence b has kv_len[b] cached tokens, the last cu_q[b + 1] - cu_q[b] of them are
    the call's (rows cu_q[b] onwards), token t lies in page page_table[b][t // page_size].  The three int32
    tensors stay on the device and may change between calls (also between replays of a captured graph) within
    the host's bounds: n_tokens rows, max_q_len new and max_kv_len cached tokens of any sequence.  Rows that no
    sequence covers are not written: in results that a call makes itself they hold anything."""

    def __init__(self, cu_q, kv_len, page_table, n_tokens: int, max_q_len: int, max_kv_len: int):
        _load()
        for name, t, dims in (("cu_q", cu_q, 1), ("kv_len", kv_len, 1), ("page_table", page_table, 2)):
            if t.dtype != torch.int32 or t.dim() != dims or not t.is_contiguous() or t.device != cu_q.device:
                raise ValueError(f"{name} must be a contiguous {dims}-D int32 tensor on {cu_q.device}")
        n = kv_len.shape[0]
        if cu_q.shape[0] != n + 1 or page_table.shape[0] != n:
            raise ValueError(f"{n} sequences need cu_q of {n + 1} entries and page_table of {n} rows")
        self.cu_q, self.kv_len, self.page_table = cu_q, kv_len, page_table
        self.n_tokens, self.device, self.index = n_tokens, cu_q.device, cu_q.get_device()
        self.c = moe_kv_batch_t(n, n_tokens, max_q_len, max_kv_len, page_table.shape[1], cu_q.data_ptr(),
                                kv_len.data_ptr(), page_table.data_ptr())


class KVCache:
    """The 8-bit paged cache (moe_kv_*): wraps codes [pages, kv heads, page_size, head_dim] (torch.float8_e4m3fn
    or uint8) and scales [pages, kv heads] fp32 of keys and values; ``KVCache.empty`` allocates them."""

    def __init__(self, k_codes, v_codes, k_scale, v_scale, n_q_heads: int, max_seqs: int, max_tokens: int,
                 max_kv_len: int):
        self.h = None
        _load()
        if k_codes.dim() != 4:
            raise ValueError("codes must be [pages, kv heads, page_size, head_dim]")
        P, H, S, D = k_codes.shape
        for name, t in (("k_codes", k_codes), ("v_codes", v_codes)):
            if t.shape != k_codes.shape or t.dtype not in (torch.uint8, torch.float8_e4m3fn) or not t.is_contiguous() \
                    or not t.is_cuda or t.device != k_codes.device:
                raise ValueError(f"{name} must be a contiguous uint8 or float8_e4m3fn CUDA tensor {(P, H, S, D)}")
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if t.shape != (P, H) or t.dtype != torch.float32 or not t.is_contiguous() or t.device != k_codes.device:
                raise ValueError(f"{name} must be a contiguous fp32 tensor {(P, H)} on {k_codes.device}")
        self.k_codes, self.v_codes, self.k_scale, self.v_scale = k_codes, v_codes, k_scale, v_scale
        self.n_q_heads, self.n_kv_heads, self.head_dim, self.page_size = n_q_heads, H, D, S
        self.device = k_codes.device
        self._index = k_codes.get_device()
        self._row = {}  # checked layouts of the calls' tensors: (name, shape, stride) -> elements between tokens
        self.default_scale = D ** -0.5
        cfg = moe_kv_config_t(n_q_heads, H, D, S, P, max_seqs, max_tokens, max_kv_len)
        store = moe_kv_store_t(*(t.data_ptr() for t in (k_codes, v_codes, k_scale, v_scale)))
        h = C.c_void_p()
        with torch.cuda.device(self.device):
            st = _load().moe_kv_create(C.byref(cfg), C.byref(store), C.byref(h))
        if st != MOE_OK:
            raise MoeError(st, moe.moe_last_error(None))
        self.h = h

    @classmethod
    def empty(cls, n_pages: int, page_size: int, n_kv_heads: int, head_dim: int, n_q_heads: int, max_seqs: int,
              max_tokens: int, max_kv_len: int, device="cuda"):
        _load()
        shape = (n_pages, n_kv_heads, page_size, head_dim)
        codes = [torch.zeros(shape, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn) for _ in range(2)]
        scales = [torch.ones(shape[:2], dtype=torch.float32, device=device) for _ in range(2)]
        return cls(*codes, *scales, n_q_heads, max_seqs, max_tokens, max_kv_len)

    def _check(self, st):
        if st != MOE_OK:
            raise MoeError(st, (_lib.moe_kv_last_error(self.h) or b"").decode())

    def _tokens(self, x, name, heads, batch):
        key = (name, x.shape, x.stride())
        s = self._row.get(key)
        if s is None:
            s = _rows(x, name, heads, self.head_dim, self.device)
            if len(self._row) >= 64:
                self._row.clear()
            self._row[key] = s
        if x.shape[0] != batch.n_tokens or x.get_device() != self._index or batch.index != self._index:
            raise ValueError(f"{name} and the batch must have the same tokens on {self.device}, got {x.shape[0]} on "
                             f"{x.device} and {batch.n_tokens} on {batch.device}")
        return s

    def write(self, k, v, batch: SeqBatch, stream=None) -> None:
        """Quantises the batch's new keys and values [tokens, kv heads, head_dim] into their pages."""
        ks = self._tokens(k, "k", self.n_kv_heads, batch)
        vs = self._tokens(v, "v", self.n_kv_heads, batch)
        if k.dtype != v.dtype:
            raise TypeError("k and v must have one dtype")
        self._check(_lib.moe_kv_write(self.h, k.data_ptr(), ks, v.data_ptr(), vs, _dtype(k.dtype, "k"), batch.c,
                                      _stream(stream, self._index)))

    def read(self, batch: SeqBatch, dtype=None, k_out=None, v_out=None, stream=None):
        """The batch's new tokens as values: (keys, values) [tokens, kv heads, head_dim] of dtype (that of a result
        which is given; bf16 without one)."""
        shape, dev = (batch.n_tokens, self.n_kv_heads, self.head_dim), self.device
        if dtype is None:
            dtype = k_out.dtype if k_out is not None else v_out.dtype if v_out is not None else torch.bfloat16
        code = _dtype(dtype, "dtype")
        if batch.index != self._index:
            raise ValueError(f"the batch must be on {dev}, got {batch.device}")
        for name, t in (("k_out", k_out), ("v_out", v_out)) if k_out is not None or v_out is not None else ():
            if t is not None and (t.shape != shape or t.dtype != dtype or not t.is_contiguous() or t.device != dev):
                raise ValueError(f"{name} must be a contiguous {dtype} tensor {shape} on {dev}")
        if k_out is None:
            k_out = _results(shape, dtype, dev, stream)
        if v_out is None:
            v_out = _results(shape, dtype, dev, stream)
        self._check(_lib.moe_kv_read(self.h, k_out.data_ptr(), v_out.data_ptr(), code, batch.c, _stream(stream, self._index)))
        return k_out, v_out

    def attend(self, q, batch: SeqBatch, out=None, lse=None, scale: float | None = None, causal: bool = True,
               window: int = 0, sinks: int = 0, stream=None):
        """Attention of the batch's new tokens q [tokens, q heads, head_dim] bf16 over their sequences' cached
        tokens (write the new ones first).  window > 0: a token sees the last ``window`` tokens, itself
        included, and the first ``sinks`` ones.  Returns out [tokens, q heads, head_dim] bf16; lse, when given,
        is filled with the natural logarithms of the softmax denominators [tokens, q heads] fp32."""
        dev, H = self.device, self.n_q_heads
        qs = self._tokens(q, "q", H, batch)
        bf16 = torch.bfloat16
        if q.dtype != bf16:
            raise TypeError(f"q must be bf16, got {q.dtype}")
        shape = (batch.n_tokens, H, self.head_dim)
        if out is None:
            out = torch.empty_like(q) if stream is None and q.dim() == 3 and q.is_contiguous() else \
                _results(shape, bf16, dev, stream)
        elif out.numel() != shape[0] * shape[1] * shape[2] or out.dtype != bf16 or not out.is_contiguous() \
                or out.device != dev:
            raise ValueError(f"out must be a contiguous bf16 tensor {shape} on {dev}")
        if lse is not None and (lse.shape != shape[:2] or lse.dtype != torch.float32 or not lse.is_contiguous()
                                or lse.device != dev):
            raise ValueError(f"lse must be a contiguous fp32 tensor {shape[:2]} on {dev}")
        mask = moe_kv_mask_t(self.default_scale if scale is None else scale, 1 if causal else 0, window, sinks)
        self._check(_lib.moe_kv_attend(self.h, q.data_ptr(), qs, out.data_ptr(),
                                       lse.data_ptr() if lse is not None else None, mask, batch.c,
                                       _stream(stream, self._index)))
        return out

    def device_status(self) -> int:
        """Device error word (0 = fine; synchronous, clears it); raises MoeError when it is set."""
        f = C.c_int32(0)
        self._check(_load().moe_kv_device_status(self.h, C.byref(f)))
        return f.value

    def close(self):
        if self.h:
            _load().moe_kv_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
