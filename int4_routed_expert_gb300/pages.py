"""ctypes binding of include/moe_pages.h: the page pool, which knows which sequence has which pages of the cache.

A serving step with a pool calls, all of it on the device (so a graph may hold it):
    moves = pool.fork(parent, added)              # the step's sequences out of the last step's
    for each layer: cache.copy(moves)             # KVCache: pages that two sequences would write to
                    cache.write(k, v, batch)      # batch = pool.batch(n_tokens, max_q_len, max_kv_len)
                    out = cache.attend(q, batch)
``compact`` moves the pages in use to the front of the pool; its moves are copied in the same way.
"""
from __future__ import annotations

import ctypes as C

from . import attn, moe
from .attn import SeqBatch
from .moe import MOE_OK, MoeError


class moe_pages_config_t(C.Structure):
    _fields_ = [(n, C.c_int) for n in ("n_pages", "page_size", "n_slots", "table_stride")]


class moe_pages_store_t(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("table", "kv_len", "ref", "cu_q", "free_pages")]


EXPORTED = ("moe_pages_create", "moe_pages_workspace_bytes", "moe_pages_last_error", "moe_pages_destroy",
            "moe_pages_fork", "moe_pages_compact", "moe_pages_device_status")

# bits of moe_pages_device_status
PAGES_BAD_CALL, PAGES_EXHAUSTED = 2, 8

_lib = None
torch = None


def _load() -> C.CDLL:
    global _lib, torch
    if _lib is not None:
        return _lib
    L = attn._load()
    vp, i32 = C.c_void_p, C.c_int
    sig = {
        "moe_pages_create": (i32, [C.POINTER(moe_pages_config_t), C.POINTER(moe_pages_store_t), C.POINTER(vp)]),
        "moe_pages_workspace_bytes": (C.c_size_t, [C.POINTER(moe_pages_config_t)]),
        "moe_pages_last_error": (C.c_char_p, [vp]),
        "moe_pages_destroy": (None, [vp]),
        "moe_pages_fork": (i32, [vp, vp, vp, vp, vp, vp]),
        "moe_pages_compact": (i32, [vp, vp, vp]),
        "moe_pages_device_status": (i32, [vp, C.POINTER(C.c_int32)]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype, fn.argtypes = res, args
    torch = attn.torch
    _lib = L
    return L


class PagePool:
    """The page pool (moe_pages_*): wraps table [slots, width] (page ids, -1 for none), kv_len [slots] and ref [pages]
    (uses of each page), int32 CUDA tensors that it changes in place; ``PagePool.empty`` allocates them.  cu_q
    [slots + 1] and free [1] (free pages: counted here, then as of the last fork or compact) are its own results; so are
    the moves that fork and compact return, which the next call of the same kind writes over."""

    def __init__(self, table, kv_len, ref, page_size: int):
        self.h = None
        _load()
        for name, t, dims in (("table", table, 2), ("kv_len", kv_len, 1), ("ref", ref, 1)):
            if t.dtype != torch.int32 or t.dim() != dims or not t.is_contiguous() or not t.is_cuda or t.device != table.device:
                raise ValueError(f"{name} must be a contiguous {dims}-D int32 CUDA tensor on one device")
        n = table.shape[0]
        if kv_len.shape[0] != n:
            raise ValueError(f"{n} slots need kv_len of {n} entries, got {kv_len.shape[0]}")
        self.table, self.kv_len, self.ref, self.page_size = table, kv_len, ref, page_size
        self.n_slots, self.n_pages, self.device, self._index = n, ref.shape[0], table.device, table.get_device()
        i32 = dict(dtype=torch.int32, device=self.device)
        self.cu_q = torch.zeros(n + 1, **i32)
        self.free = (ref == 0).sum(dtype=torch.int32).view(1)
        self._forked = torch.full((n, 3), -1, **i32)
        self._compacted = torch.full((self.n_pages // 2, 3), -1, **i32)
        cfg = moe_pages_config_t(self.n_pages, page_size, n, table.shape[1])
        store = moe_pages_store_t(*(t.data_ptr() for t in (table, kv_len, ref, self.cu_q, self.free)))
        h = C.c_void_p()
        with torch.cuda.device(self.device):
            st = _lib.moe_pages_create(C.byref(cfg), C.byref(store), C.byref(h))
        if st != MOE_OK:
            raise MoeError(st, moe.moe_last_error(None))
        self.h = h

    @classmethod
    def empty(cls, n_pages: int, page_size: int, n_slots: int, max_kv_len: int, device="cuda"):
        _load()
        i32 = dict(dtype=torch.int32, device=device)
        return cls(torch.full((n_slots, -(-max_kv_len // page_size)), -1, **i32), torch.zeros(n_slots, **i32),
                   torch.zeros(n_pages, **i32), page_size)

    def _check(self, st):
        if st != MOE_OK:
            raise MoeError(st, (_lib.moe_pages_last_error(self.h) or b"").decode())

    def _slots(self, name, t):
        if t.dtype is not torch.int32 or t.shape != (self.n_slots,) or not t.is_contiguous() or t.get_device() != self._index:
            raise ValueError(f"{name} must be a contiguous int32 tensor of {self.n_slots} entries on {self.device}, got "
                             f"{t.dtype} {tuple(t.shape)} on {t.device}")
        return t.data_ptr()

    def fork(self, parent, added, keep=None, stream=None):
        """The next step's sequences: slot i goes on from the first keep[i] tokens (all, without keep) of slot
        parent[i] (-1: from none), with room for added[i] tokens; slots that none goes on from are freed.  int32
        tensors [slots].  Returns the pages to copy (``KVCache.copy``) [slots, 3]."""
        self._check(_lib.moe_pages_fork(self.h, self._slots("parent", parent), self._slots("added", added),
                                        None if keep is None else self._slots("keep", keep), self._forked.data_ptr(),
                                        attn._stream(stream, self._index)))
        return self._forked

    def compact(self, stream=None):
        """Moves the pages in use to the front of the pool; returns the pages to copy [pages // 2, 3]."""
        self._check(_lib.moe_pages_compact(self.h, self._compacted.data_ptr(), attn._stream(stream, self._index)))
        return self._compacted

    def batch(self, n_tokens: int, max_q_len: int, max_kv_len: int) -> SeqBatch:
        """The pool's sequences and the last fork's new tokens as a batch of the cache's calls, within the host's
        bounds.  It stays valid: later forks change the arrays that it looks at."""
        return SeqBatch(self.cu_q, self.kv_len, self.table, n_tokens, max_q_len, max_kv_len)

    def device_status(self) -> int:
        """Device error word (0 = fine; synchronous, clears it); raises MoeError when it is set."""
        f = C.c_int32(0)
        self._check(_lib.moe_pages_device_status(self.h, C.byref(f)))
        return f.value

    def close(self):
        if self.h:
            _load().moe_pages_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
