"""The attention-side entry points against a fake CUDA runtime of several devices (fake_cuda.cpp): which device a
call works on, what it refuses.  Only host code runs."""
from __future__ import annotations

import ctypes as C
import math
import os
import random
import subprocess
from fractions import Fraction

import pytest

from turns import TWO_PI

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID = -1
BF16 = 1


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    from int4_routed_expert_gb300 import attn as A
    from int4_routed_expert_gb300 import build as b
    out = tmp_path_factory.mktemp("fake") / "libfake.so"
    subprocess.run([b._nvcc(), *b.ARCH, "-std=c++17", "-shared", "-Xcompiler", "-fPIC", "-Xlinker", "-Bsymbolic",
                    "--cudart", "shared", "--expt-relaxed-constexpr", "-I", b.INC,
                    os.path.join(b.CSRC, "attn_api.cu"), os.path.join(ROOT, "tests", "fake_cuda.cpp"), "-o", str(out)],
                   check=True)
    L = C.CDLL(str(out))
    vp, i32, i64 = C.c_void_p, C.c_int, C.c_int64
    L.fake_log.restype = L.moe_kv_last_error.restype = L.moe_last_error.restype = C.c_char_p
    L.moe_kv_last_error.argtypes = L.moe_last_error.argtypes = [vp]
    L.moe_rope_create.argtypes = [i32, C.POINTER(C.c_double), C.c_float, i32, C.POINTER(vp)]
    L.moe_rope_apply.argtypes = [vp, vp, vp, i32, i32, vp, i32, vp]
    L.fake_rope_inc.restype = C.c_uint64
    L.moe_rope_destroy.argtypes = L.moe_kv_destroy.argtypes = [vp]
    L.moe_kv_create.argtypes = [vp, vp, C.POINTER(vp)]
    L.moe_kv_write.argtypes = [vp, vp, i64, vp, i64, i32, vp, vp]
    L.moe_kv_read.argtypes = [vp, vp, vp, i32, vp, vp]
    L.moe_kv_attend.argtypes = [vp, vp, i64, vp, vp, vp, vp, vp]
    L.moe_kv_device_status.argtypes = [vp, C.POINTER(C.c_int32)]
    L.A = A
    return L


def at(device, offset=0):
    """An address in the fake device's memory."""
    return ((device + 1) << 40) + offset


class Kv:
    """A handle on a device, with a batch of three single tokens there."""

    def __init__(self, lib, device, q_heads=8, max_tokens=64):
        A = lib.A
        lib.fake_reset(device)
        self.lib, self.h = lib, C.c_void_p()
        cfg = A.moe_kv_config_t(q_heads, 2, 64, 16, 10, 4, max_tokens, 128)
        st = A.moe_kv_store_t(*(at(device, i << 20) for i in range(4)))
        assert lib.moe_kv_create(C.byref(cfg), C.byref(st), C.byref(self.h)) == 0
        self.batch = A.moe_kv_batch_t(3, 3, 1, 100, 8, *(at(device, (8 + i) << 20) for i in range(3)))
        self.mask = A.moe_kv_mask_t(0.125, 1, 0, 0)
        self.device = device
        lib.fake_clear_log()

    def write(self, k=None, v=None, batch=None):
        b = C.byref(batch or self.batch)
        return self.lib.moe_kv_write(self.h, k or at(self.device, 1 << 24), 128, v or at(self.device, 1 << 25), 128,
                                     BF16, b, None)

    def read(self, k=None, v=None):
        return self.lib.moe_kv_read(self.h, k or at(self.device, 1 << 24), v or at(self.device, 1 << 25), BF16,
                                    C.byref(self.batch), None)

    def attend(self, q=None, out=None, lse=None, stride=512):
        return self.lib.moe_kv_attend(self.h, q or at(self.device, 1 << 24), stride, out or at(self.device, 1 << 25), lse,
                                      C.byref(self.mask), C.byref(self.batch), None)

    def log(self):
        text = self.lib.fake_log().decode().split()
        self.lib.fake_clear_log()
        return text


def test_calls_work_on_the_handle_s_device(lib):
    kv = Kv(lib, 1)
    lib.fake_make_current(0)
    for call, name in ((kv.write, "write"), (kv.read, "read"), (kv.attend, "few")):
        assert call() == 0
        assert kv.log() == [name + "@1"]
        assert lib.fake_current() == 0
    kv.batch.n_tokens = kv.batch.max_q_len = 50
    assert kv.attend() == 0 and kv.log() == ["tiles@1"] and lib.fake_current() == 0
    lib.fake_set_flags(1)
    flags = C.c_int32()
    assert lib.moe_kv_device_status(kv.h, C.byref(flags)) != 0 and flags.value == 1
    log = kv.log()
    assert log[:2] == ["sync@1", "memcpy@1"] and all(x.endswith("@1") for x in log) and lib.fake_current() == 0
    lib.moe_kv_destroy(kv.h)
    assert kv.log() == ["sync@1", "free@1"] and lib.fake_current() == 0


def test_tensors_of_another_device_are_refused(lib):
    kv = Kv(lib, 1)
    far = at(0, 1 << 24)
    for call in (lambda: kv.write(k=far), lambda: kv.write(v=far), lambda: kv.read(k=far), lambda: kv.read(v=far),
                 lambda: kv.attend(q=far), lambda: kv.attend(out=far), lambda: kv.attend(lse=far)):
        assert call() == INVALID and b"device" in lib.moe_kv_last_error(kv.h)
    for field in ("cu_q", "kv_len", "page_table"):
        old = getattr(kv.batch, field)
        setattr(kv.batch, field, far)
        assert kv.attend() == INVALID and field.encode() in lib.moe_kv_last_error(kv.h)
        setattr(kv.batch, field, old)
    assert kv.log() == []
    assert kv.attend(lse=at(1, 1 << 26)) == 0
    lib.moe_kv_destroy(kv.h)


def test_attend_refuses_more_rows_than_32_bits_number(lib):
    kv = Kv(lib, 0, q_heads=256, max_tokens=1 << 24)
    kv.batch.n_tokens = 1 << 23
    assert kv.attend(stride=256 * 64) == -2 and b"rows" in lib.moe_kv_last_error(kv.h) and kv.log() == []
    kv.batch.n_tokens -= 1
    assert kv.attend(stride=256 * 64) == 0 and len(kv.log()) == 1
    lib.moe_kv_destroy(kv.h)


@pytest.mark.parametrize("scale,status", [(2.3e38, 0), (2.4e38, INVALID), (-2.4e38, INVALID), (math.inf, INVALID),
                                          (math.nan, INVALID), (0.0, 0)])
def test_attend_refuses_scales_that_overflow(lib, scale, status):
    """The kernels take scale * log2 e, which is infinite in fp32 from 2.36e38 on: every result would be NaN."""
    kv = Kv(lib, 0)
    kv.mask.scale = scale
    assert kv.attend() == status and len(kv.log()) == (status == 0)
    lib.moe_kv_destroy(kv.h)


def _rows(lib, cfg):
    """Rows of partial results in a configuration's workspace: sums, a reference and a weight sum, a counter for 16."""
    L = lib.moe_kv_workspace_bytes
    L.restype = C.c_size_t
    rows, rest = divmod((L(C.byref(cfg)) - 256) * 4, (cfg.head_dim * 4 + 8) * 4 + 1)
    assert rest == 0 and rows % 32 == 0
    return rows


def test_workspace_holds_what_the_bounds_can_use(lib):
    """Room for a split of every tile of keys, up to each kernel's limits, for every call within the bounds; no more."""
    cfg = lib.A.moe_kv_config_t
    assert _rows(lib, cfg(48, 8, 128, 64, 100, 64, 8192, 131072)) == 1 << 18
    assert _rows(lib, cfg(8, 2, 64, 16, 10, 1, 1, 128)) == 64  # one token, one tile of keys
    assert _rows(lib, cfg(48, 8, 128, 64, 100, 1, 1, 4096)) == 8 * 32 * 32
    assert _rows(lib, cfg(4, 2, 64, 16, 64, 2, 64, 64)) == 2 * 2 * 256  # a tile of keys, 128 rows of 256
    r = random.Random(1)
    for _ in range(2000):
        hkv, g = r.choice((1, 2, 8, 256)), r.choice((1, 3, 16))
        seqs, tokens, kv = (int(2 ** r.uniform(0, b)) for b in (15.9, 24, 30))
        cap = _rows(lib, cfg(hkv * g, hkv, r.choice((64, 128)), 16, 10, seqs, tokens, kv))
        assert cap <= 1 << 18
        for _ in range(20):
            n, q = r.randint(1, seqs), r.randint(1, min(tokens, r.choice((1, 8, 100, tokens))))
            tiles = -(-r.randint(1, kv) // 128)
            if q * g <= 32:
                rows = 16 if q * g <= 16 else 32
                need = n * hkv * rows * min(tiles, 256, 4096 // rows)
            else:
                need = n * hkv * -(-q * g // 256) * 256 * min(tiles, 256)
            assert need <= cap or cap == 1 << 18


def test_rope_works_on_its_tensors_device(lib):
    T = lib.A.moe_rope_tensor_t
    lib.fake_reset(0)
    r = C.c_void_p()
    assert lib.moe_rope_create(64, (C.c_double * 32)(*[0.5] * 32), 1.0, 0, C.byref(r)) == 0

    def apply(q, y, k=None, pos=at(1)):
        tq, tk = T(q, y, 4, 256, 256), T(k, k, 2, 128, 128)
        return lib.moe_rope_apply(r, C.byref(tq), C.byref(tk) if k else None, 64, BF16, pos, 5, None)

    assert apply(at(1, 1 << 24), at(1, 1 << 25), at(1, 1 << 26)) == 0
    assert lib.fake_log() == b"rope@1 " and lib.fake_current() == 0
    lib.fake_clear_log()
    assert apply(at(1, 1 << 24), at(0, 1 << 25)) == INVALID and b"device" in lib.moe_last_error(None)
    assert apply(at(1, 1 << 24), at(1, 1 << 25), at(0, 1 << 26)) == INVALID
    assert apply(at(1, 1 << 24), at(1, 1 << 25), pos=at(0)) == INVALID
    assert lib.fake_log() == b""
    lib.moe_rope_destroy(r)


def test_rope_fractions_of_a_turn(lib):
    """The 64-bit fractions are off by at most a step of theirs, which every int32 position multiplies."""
    lib.fake_reset(0)
    r = random.Random(3)
    freq = [1.0, -1.0, 0.75, 2 * math.pi, 1e-30, 2.0 ** 37, -1e9] + \
        [r.choice((-1, 1)) * math.exp(r.uniform(-30, 3)) for _ in range(57)] + [r.uniform(0.5, 1.2) for _ in range(64)]
    h = C.c_void_p()
    assert lib.moe_rope_create(256, (C.c_double * 128)(*freq), 1.0, 0, C.byref(h)) == 0
    t = lib.A.moe_rope_tensor_t(at(0), at(0), 1, 256, 256)
    assert lib.moe_rope_apply(h, C.byref(t), None, 256, BF16, at(0, 1 << 20), 1, None) == 0
    for i, f in enumerate(freq):
        off = (lib.fake_rope_inc(i) - Fraction(f) / TWO_PI * 2 ** 64) % 2 ** 64
        assert min(off, 2 ** 64 - off) <= 1, f
    lib.moe_rope_destroy(h)
