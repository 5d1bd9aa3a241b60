"""Host-side checks of include/moe_attn.h and its binding: exports, C99, refusals before any launch, rotary
frequencies.  No kernel runs, so none of this needs a GPU."""
from __future__ import annotations

import ctypes as C
import math
import os
import re
import shutil
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED, CAPACITY, CUDA = -1, -2, -3, -4


@pytest.fixture(scope="module")
def lib():
    from int4_routed_expert_gb300 import build as b
    b.build()
    from int4_routed_expert_gb300 import attn
    return attn._load()


@pytest.fixture(scope="module")
def A():
    from int4_routed_expert_gb300 import attn
    return attn


def _message(lib):
    return (lib.moe_last_error(None) or b"").decode()


def test_declared_calls_are_bound_and_exported(lib, A):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "moe_attn.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(moe_[a-z_]+)\s*\(", text))
    assert names == set(A.EXPORTED)
    assert all(hasattr(lib, n) for n in names)


def test_header_is_strict_c99(lib, tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src, exe = tmp_path / "c.c", tmp_path / "c"
    src.write_text(r"""
#include "moe_attn.h"
int main(void) {
  double f[8] = {1, 0.5, 0.25, 0.1, 0.05, 0.01, 0.005, 0.001};
  moe_rope_t* r = 0;
  moe_kv_t* h = (moe_kv_t*)1;
  moe_kv_config_t cfg = {48, 8, 128, 64, 100, 4, 512, 4096}, bad = cfg;
  moe_kv_store_t st = {0, 0, 0, 0};
  moe_kv_mask_t mask = {0.1f, 1, 0, 0};
  moe_rope_tensor_t t = {0, 0, 4, 256, 256};
  bad.head_dim = 96;
  if (moe_rope_create(16, f, 1.0f, 0, &r) != MOE_OK || !r) return 1;
  if (moe_rope_apply(r, &t, 0, 64, MOE_BF16, 0, 0, 0) != MOE_OK) return 2; /* no tokens */
  moe_rope_destroy(r);
  moe_rope_destroy(0);
  if (moe_kv_workspace_bytes(&cfg) == 0 || moe_kv_workspace_bytes(&bad) != 0) return 3;
  if (moe_kv_create(&bad, &st, &h) != MOE_ERR_UNSUPPORTED || h) return 4;
  if (moe_kv_create(&cfg, &st, &h) != MOE_ERR_INVALID_ARG || h) return 5;
  if (moe_kv_attend(0, 0, 0, 0, 0, &mask, 0, 0) != MOE_ERR_INVALID_ARG) return 6;
  if (!moe_kv_last_error(0)[0]) return 7;
  moe_kv_destroy(0);
  return 0;
}
""")
    libdir = os.path.join(ROOT, "int4_routed_expert_gb300")
    subprocess.run([cc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"),
                    str(src), "-o", str(exe), "-L", libdir, "-lmoe", f"-Wl,-rpath,{libdir}"], check=True)
    assert subprocess.run([str(exe)], timeout=120).returncode == 0


@pytest.mark.parametrize("rot,freq,amp,status", [
    (8, [1.0] * 4, 1.0, UNSUPPORTED), (24, [1.0] * 12, 1.0, UNSUPPORTED), (272, [1.0] * 136, 1.0, UNSUPPORTED),
    (0, [1.0], 1.0, UNSUPPORTED), (16, None, 1.0, INVALID), (16, [1.0] * 7 + [math.inf], 1.0, INVALID),
    (16, [math.nan] * 8, 1.0, INVALID), (16, [1.0] * 8, math.nan, INVALID)])
def test_rope_create_refuses(lib, rot, freq, amp, status):
    h = C.c_void_p(1)
    arr = (C.c_double * len(freq))(*freq) if freq else None
    assert lib.moe_rope_create(rot, arr, amp, 0, C.byref(h)) == status and not h.value
    assert _message(lib)
    assert lib.moe_rope_create(rot, arr, amp, 0, None) == INVALID


def test_rope_apply_refuses(lib, A):
    r = A.Rope(32)
    T = A.moe_rope_tensor_t
    ok = T(0x10000, 0x20000, 2, 128, 128)

    def call(q, dim=64, dt=1, n=3, k=None, pos=0x1000, h=None):
        return lib.moe_rope_apply(r.h if h is None else h, C.byref(q) if q else None, C.byref(k) if k else None,
                                  dim, dt, pos, n, None)

    assert call(None) == INVALID
    assert lib.moe_rope_apply(None, C.byref(ok), None, 64, 1, 0x1000, 3, None) == INVALID
    assert call(ok, dim=72) == UNSUPPORTED and call(ok, dim=16) == UNSUPPORTED and call(ok, dim=272) == UNSUPPORTED
    assert call(ok, dt=2) == INVALID and call(ok, n=-1) == INVALID
    assert call(T(0x10000, 0x20000, 0, 128, 128)) == UNSUPPORTED
    for bad in (T(0x10000, 0x20000, 2, 120, 128), T(0x10000, 0x20000, 2, 128, 132), T(0x10000, 0x20000, 2, 64, 128)):
        assert call(bad) == INVALID and "stride" in _message(lib)
    assert call(T(None, 0x20000, 2, 128, 128)) == INVALID and "NULL" in _message(lib)
    assert call(T(0x10008, 0x20000, 2, 128, 128)) == INVALID and "aligned" in _message(lib)
    assert call(ok, k=T(0x10000, 0x20000, 2, 100, 128)) == INVALID
    assert call(ok, n=0) == 0  # nothing to do
    buf = C.create_string_buffer(4096)  # plain host memory
    at = (C.addressof(buf) + 15) // 16 * 16
    assert call(T(at, at, 2, 128, 128)) == INVALID


def _cfg(A, **kw):
    c = dict(n_q_heads=8, n_kv_heads=2, head_dim=64, page_size=16, n_pages=10, max_seqs=4, max_tokens=64, max_kv_len=128)
    c.update(kw)
    return A.moe_kv_config_t(**c)


@pytest.mark.parametrize("bad", [
    dict(n_kv_heads=0), dict(n_kv_heads=257, n_q_heads=257), dict(n_q_heads=7), dict(n_q_heads=0), dict(head_dim=96),
    dict(head_dim=256), dict(page_size=8), dict(page_size=48), dict(page_size=256), dict(n_pages=0), dict(max_seqs=0),
    dict(max_seqs=65536), dict(max_tokens=0), dict(max_kv_len=0), dict(max_kv_len=(1 << 30) + 1)])
def test_kv_create_refuses_geometry(lib, A, bad):
    h = C.c_void_p(1)
    st = A.moe_kv_store_t(0x10000, 0x20000, 0x30000, 0x40000)
    assert lib.moe_kv_create(C.byref(_cfg(A, **bad)), C.byref(st), C.byref(h)) == UNSUPPORTED and not h.value
    assert lib.moe_kv_workspace_bytes(C.byref(_cfg(A, **bad))) == 0 and _message(lib)


def test_kv_create_refuses_store(lib, A):
    h = C.c_void_p(1)
    assert lib.moe_kv_create(C.byref(_cfg(A)), None, C.byref(h)) == INVALID and not h.value
    for st in (A.moe_kv_store_t(None, 0x20000, 0x30000, 0x40000), A.moe_kv_store_t(0x10000, 0x20008, 0x30000, 0x40000)):
        assert lib.moe_kv_create(C.byref(_cfg(A)), C.byref(st), C.byref(h)) == INVALID
        assert "store array" in _message(lib)
    assert lib.moe_kv_create(C.byref(_cfg(A)), C.byref(st), None) == INVALID
    assert lib.moe_kv_workspace_bytes(C.byref(_cfg(A))) > 0
    if not torch.cuda.is_available():
        ok = A.moe_kv_store_t(0x10000, 0x20000, 0x30000, 0x40000)
        assert lib.moe_kv_create(C.byref(_cfg(A)), C.byref(ok), C.byref(h)) == CUDA and not h.value


def test_null_handles(lib, A):
    b, m = A.moe_kv_batch_t(), A.moe_kv_mask_t(1.0, 1, 0, 0)
    f = C.c_int32(7)
    assert lib.moe_kv_write(None, None, 0, None, 0, 1, C.byref(b), None) == INVALID
    assert lib.moe_kv_read(None, None, None, 1, C.byref(b), None) == INVALID
    assert lib.moe_kv_attend(None, None, 0, None, None, C.byref(m), C.byref(b), None) == INVALID
    assert lib.moe_kv_device_status(None, C.byref(f)) == INVALID and f.value == 7
    lib.moe_kv_destroy(None)
    lib.moe_rope_destroy(None)


def test_binding_refuses_tensors(A):
    x = torch.zeros(3, 4, 64)
    with pytest.raises(ValueError):
        A.Rope(32).apply(x, torch.zeros(3, dtype=torch.int32))  # host tensor
    with pytest.raises(ValueError):
        A.KVCache(torch.zeros(2, 1, 16, 64, dtype=torch.uint8), torch.zeros(2, 1, 16, 64, dtype=torch.uint8),
                  torch.zeros(2, 1), torch.zeros(2, 1), 1, 1, 1, 1)
    i = dict(dtype=torch.int32)
    with pytest.raises(ValueError):
        A.SeqBatch(torch.zeros(3, **i), torch.zeros(3, **i), torch.zeros(3, 2, **i), 1, 1, 1)  # cu_q too short
    with pytest.raises(ValueError):
        A.SeqBatch(torch.zeros(4), torch.zeros(3, **i), torch.zeros(3, 2, **i), 1, 1, 1)  # dtype
    cpu = torch.device("cpu")
    assert A._rows(torch.zeros(3, 4, 64), "x", 4, 64, cpu) == 256
    assert A._rows(torch.zeros(3, 12, 64)[:, 2:6], "x", 4, 64, cpu) == 768  # part of one projection
    assert A._rows(torch.zeros(3, 256), "x", 4, 64, cpu) == 256
    for bad in (torch.zeros(3, 64, 4).transpose(1, 2), torch.zeros(3, 4, 128)[..., ::2], torch.zeros(3, 5, 64),
                torch.zeros(3, 8, 64)[:, ::2], torch.zeros(3, 255)):
        with pytest.raises(ValueError):
            A._rows(bad, "x", 4, 64, cpu)


def test_rope_frequencies(A):
    f, amp = A.rope_frequencies(64, 10000.0)
    assert amp == 1.0 and len(f) == 32 and f[0] == 1.0
    assert f[8] == pytest.approx(10000.0 ** -0.25, rel=1e-14)
    lin, _ = A.rope_frequencies(64, 10000.0, "linear", 4.0)
    assert lin == [x / 4 for x in f]
    ntk, _ = A.rope_frequencies(64, 10000.0, "ntk", 4.0)
    # the slowest pair is slowed by factor, the fastest is kept
    assert ntk[0] == 1.0 and ntk[31] == pytest.approx(f[31] / 4, rel=1e-12)
    yarn, amp = A.rope_frequencies(64, 10000.0, "yarn", 16.0, 4096)
    assert amp == pytest.approx(0.1 * math.log(16) + 1)
    for x, y in zip(f, yarn):
        turns = 4096 * x / (2 * math.pi)
        if turns > 64:
            assert y == x
        if turns < 0.5:
            assert y == pytest.approx(x / 16)
        assert x / 16 <= y * (1 + 1e-12) and y <= x * (1 + 1e-12)
    for bad in (("cubic", 2.0, 0), ("yarn", 2.0, 0), ("linear", 0.5, 0)):
        with pytest.raises(ValueError):
            A.rope_frequencies(64, 10000.0, *bad)
    with pytest.raises(ValueError):
        A.Rope(32, inv_freq=[1.0] * 15)
