"""Attention over shared prefixes and rotary positions with several axes against the fake CUDA runtime of several devices
(fake_cuda.cpp): which device a call works on, what it refuses.  Only host code runs."""
from __future__ import annotations

import ctypes as C
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED, CAPACITY = -1, -2, -3


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    from int4_routed_expert_gb300 import attn as A
    from int4_routed_expert_gb300 import build as b
    out = tmp_path_factory.mktemp("fake") / "libfake_shared.so"
    subprocess.run([b._nvcc(), *b.ARCH, "-std=c++17", "-shared", "-Xcompiler", "-fPIC", "-Xlinker", "-Bsymbolic",
                    "--cudart", "shared", "--expt-relaxed-constexpr", "-I", b.INC,
                    *(os.path.join(b.CSRC, n) for n in ("attn_api.cu", "shared_api.cu", "rope_axes_api.cu")),
                    *(os.path.join(ROOT, "tests", n) for n in ("fake_cuda.cpp", "fake_shared.cpp")), "-o", str(out)], check=True)
    L = C.CDLL(str(out))
    vp, i32, i64 = C.c_void_p, C.c_int, C.c_int64
    L.fake_log.restype = L.fake_shared_log.restype = L.moe_kv_last_error.restype = L.moe_last_error.restype = C.c_char_p
    L.moe_kv_last_error.argtypes = L.moe_last_error.argtypes = [vp]
    L.moe_kv_create.argtypes = [vp, vp, C.POINTER(vp)]
    L.moe_kv_destroy.argtypes = L.moe_rope_destroy.argtypes = [vp]
    L.moe_kv_shared_workspace_bytes.argtypes = [vp] * 3
    L.moe_kv_shared_workspace_bytes.restype = C.c_size_t
    L.moe_kv_attend_shared.argtypes = [vp, vp, i64, vp, vp, vp, vp, vp, vp, C.c_size_t, vp]
    L.moe_rope_create_axes.argtypes = [i32, vp, C.c_float, i32, i32, vp, C.POINTER(vp)]
    L.moe_rope_apply_axes.argtypes = [vp, vp, vp, i32, i32, vp, i64, i32, vp]
    L.A = A
    return L


def at(device, offset=0):
    return ((device + 1) << 40) + offset


class Kv:
    """A handle on device 1, with a batch of three single tokens and a prefix of two of them there."""

    def __init__(self, lib):
        A = lib.A
        lib.fake_reset(1)
        self.lib, self.h = lib, C.c_void_p()
        cfg = A.moe_kv_config_t(8, 2, 64, 16, 10, 4, 64, 128)
        st = A.moe_kv_store_t(*(at(1, i << 20) for i in range(4)))
        assert lib.moe_kv_create(C.byref(cfg), C.byref(st), C.byref(self.h)) == 0
        lib.fake_make_current(0)
        lib.fake_clear_log()
        lib.fake_shared_log()
        self.batch = A.moe_kv_batch_t(3, 3, 1, 100, 8, *(at(1, (8 + i) << 20) for i in range(3)))
        self.prefix = A.moe_kv_prefix_t(1, 2, 90, 8, *(at(1, (12 + i) << 20) for i in range(3)))
        self.mask = A.moe_kv_mask_t(0.125, 1, 0, 0)

    def size(self):
        return self.lib.moe_kv_shared_workspace_bytes(self.h, C.byref(self.batch), C.byref(self.prefix))

    def call(self, q=at(1, 1 << 24), out=at(1, 1 << 25), lse=None, room=at(1, 1 << 26), size=4096, prefix=True):
        return self.lib.moe_kv_attend_shared(self.h, q, 512, out, lse, C.byref(self.mask), C.byref(self.batch),
                                             C.byref(self.prefix) if prefix else None, room, size, None)

    def message(self):
        return self.lib.moe_kv_last_error(self.h)


def test_calls_work_on_the_handle_s_device(lib):
    kv = Kv(lib)
    assert kv.size() == 4096 and kv.call() == 0
    assert lib.fake_shared_log() == b"shared@1 " and lib.fake_current() == 0
    kv.prefix.n_groups = 0  # the ordinary attention, without a workspace
    assert kv.call(room=None, size=0) == 0 and lib.fake_log() == b"few@1 " and kv.size() == 0
    kv.prefix.n_groups = 1
    kv.batch.n_tokens = 0
    assert kv.call() == 0 and lib.fake_shared_log() == b""
    lib.moe_kv_destroy(kv.h)


def test_refusals(lib):
    kv = Kv(lib)
    far = at(0, 1 << 24)
    for name, bad in (("q", far), ("out", far), ("lse", far), ("room", far), ("room", None), ("room", at(1, (1 << 26) + 8))):
        assert kv.call(**{name: bad}) == INVALID
    assert b"workspace" in kv.message()
    for field in ("cu_seq", "prefix_len", "page_table"):
        old = getattr(kv.prefix, field)
        for bad in (far, None, old + 4):
            setattr(kv.prefix, field, bad)
            assert kv.call() == INVALID and field.encode() in kv.message()
        setattr(kv.prefix, field, old)
    for field, bads in (("n_groups", (-1, 65536)), ("max_group_tokens", (0, -1)), ("max_prefix_len", (0, 129)), ("table_stride", (0,))):
        old = getattr(kv.prefix, field)
        for bad in bads:
            setattr(kv.prefix, field, bad)
            assert kv.call() == INVALID and kv.message() and kv.size() == 0
        setattr(kv.prefix, field, old)
    assert kv.call(prefix=False) == INVALID and kv.call(size=4095) == CAPACITY and b"4096" in kv.message()
    kv.mask.window = 50
    assert kv.call() == UNSUPPORTED and b"window" in kv.message()
    kv.mask.window = 100  # all that is cached
    assert kv.call() == 0 and lib.fake_shared_log() == b"shared@1 "
    kv.mask.causal = 0
    assert kv.call() == INVALID
    assert lib.moe_kv_attend_shared(None, None, 0, None, None, None, None, None, None, 0, None) == INVALID
    assert lib.fake_shared_log() == b"" and lib.fake_log() == b""
    for args in ((None, C.byref(kv.batch), C.byref(kv.prefix)), (kv.h, None, C.byref(kv.prefix)), (kv.h, C.byref(kv.batch), None)):
        assert lib.moe_kv_shared_workspace_bytes(*args) == 0
    kv.batch.n_seqs = 5
    assert kv.size() == 0
    lib.moe_kv_destroy(kv.h)


def test_rope_axes_work_on_their_tensors_device(lib):
    T = lib.A.moe_rope_tensor_t
    lib.fake_reset(0)
    lib.fake_shared_log()
    r = C.c_void_p()
    assert lib.moe_rope_create_axes(64, (C.c_double * 32)(*[0.5] * 32), 1.0, 0, 3, (C.c_int32 * 32)(*[0, 2] * 16), C.byref(r)) == 0

    def apply(q, y, k=None, pos=at(1), stride=5):
        tq, tk = T(q, y, 4, 256, 256), T(k, k, 2, 128, 128)
        return lib.moe_rope_apply_axes(r, C.byref(tq), C.byref(tk) if k else None, 64, 1, pos, stride, 5, None)

    assert apply(at(1, 1 << 24), at(1, 1 << 25), at(1, 1 << 26)) == 0
    assert lib.fake_shared_log() == b"axes@1 " and lib.fake_current() == 0
    for bad in (dict(y=at(0, 1 << 25)), dict(k=at(0, 1 << 26)), dict(pos=at(0)), dict(pos=None), dict(pos=at(1, 4)), dict(stride=4),
                dict(stride=-5), dict(stride=1 << 41)):
        assert apply(**{"q": at(1, 1 << 24), "y": at(1, 1 << 25), **bad}) == INVALID and lib.moe_last_error(None)
    assert lib.fake_shared_log() == b""
    lib.moe_rope_destroy(r)
