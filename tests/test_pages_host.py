"""Host side of include/moe_pages.h and of moe_kv_copy: exports, C99, refusals before any launch, the device that a
call works on (against the fake runtime of fake_cuda.cpp).  No kernel runs."""
from __future__ import annotations

import ctypes as C
import os
import re
import shutil
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED, CUDA = -1, -2, -4


@pytest.fixture(scope="module")
def G():
    from int4_routed_expert_gb300 import build as b
    b.build()
    from int4_routed_expert_gb300 import pages
    pages._load()
    return pages


def test_declared_calls_are_bound_and_exported(G):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "moe_pages.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(moe_[a-z_]+)\s*\(", text))
    assert names == set(G.EXPORTED)
    assert all(hasattr(G._lib, n) for n in names)


def test_header_is_strict_c99(G, tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src, exe = tmp_path / "c.c", tmp_path / "c"
    src.write_text(r"""
#include "moe_pages.h"
int main(void) {
  moe_pages_t* h = (moe_pages_t*)1;
  moe_pages_config_t cfg = {100, 64, 4, 32}, bad = cfg;
  moe_pages_store_t st = {0, 0, 0, 0, 0};
  moe_page_move_t mv = {0, 1, 64};
  int32_t f = 7;
  bad.page_size = 24;
  if (sizeof(mv) != 12) return 1;
  if (moe_pages_workspace_bytes(&cfg) == 0 || moe_pages_workspace_bytes(&bad) != 0) return 2;
  if (moe_pages_create(&bad, &st, &h) != MOE_ERR_UNSUPPORTED || h) return 3;
  if (moe_pages_create(&cfg, &st, &h) != MOE_ERR_INVALID_ARG || h) return 4;
  if (moe_pages_fork(0, 0, 0, 0, &mv, 0) != MOE_ERR_INVALID_ARG) return 5;
  if (moe_pages_compact(0, &mv, 0) != MOE_ERR_INVALID_ARG) return 6;
  if (moe_pages_device_status(0, &f) != MOE_ERR_INVALID_ARG || f != 7) return 7;
  if (moe_kv_copy(0, &mv, 1, 0) != MOE_ERR_INVALID_ARG) return 8;
  if (!moe_pages_last_error(0)[0]) return 9;
  moe_pages_destroy(0);
  return 0;
}
""")
    libdir = os.path.join(ROOT, "int4_routed_expert_gb300")
    subprocess.run([cc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"),
                    str(src), "-o", str(exe), "-L", libdir, "-lmoe", f"-Wl,-rpath,{libdir}"], check=True)
    assert subprocess.run([str(exe)], timeout=120).returncode == 0


@pytest.mark.parametrize("bad", [(0, 64, 4, 32), ((1 << 27) + 1, 64, 4, 32), (10, 8, 4, 32), (10, 48, 4, 32), (10, 256, 4, 32),
                                 (10, 64, 0, 32), (10, 64, 65536, 32), (10, 64, 4, 0), (10, 64, 4, (1 << 24) + 1),
                                 (10, 64, 17, 1 << 24)])
def test_create_refuses_geometry(G, bad):
    h = C.c_void_p(1)
    cfg, st = G.moe_pages_config_t(*bad), G.moe_pages_store_t(*range(0x10000, 0x60000, 0x10000))
    assert G._lib.moe_pages_create(C.byref(cfg), C.byref(st), C.byref(h)) == UNSUPPORTED and not h.value
    assert G._lib.moe_pages_workspace_bytes(C.byref(cfg)) == 0


def test_create_refuses_store(G):
    h = C.c_void_p(1)
    cfg = G.moe_pages_config_t(10, 64, 4, 32)
    assert G._lib.moe_pages_create(C.byref(cfg), None, C.byref(h)) == INVALID and not h.value
    good = list(range(0x10000, 0x60000, 0x10000))
    for i in range(5):
        for p in (None, good[i] + 4):
            st = G.moe_pages_store_t(*(p if j == i else x for j, x in enumerate(good)))
            assert G._lib.moe_pages_create(C.byref(cfg), C.byref(st), C.byref(h)) == INVALID
    assert G._lib.moe_pages_create(C.byref(cfg), C.byref(st), None) == INVALID
    if not torch.cuda.is_available():
        assert G._lib.moe_pages_create(C.byref(cfg), C.byref(G.moe_pages_store_t(*good)), C.byref(h)) == CUDA and not h.value
    with pytest.raises(ValueError):
        G.PagePool(torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(5, dtype=torch.int32), 16)


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    from int4_routed_expert_gb300 import attn as A
    from int4_routed_expert_gb300 import build as b
    from int4_routed_expert_gb300 import pages
    out = tmp_path_factory.mktemp("fake") / "libfake_pages.so"
    subprocess.run([b._nvcc(), *b.ARCH, "-std=c++17", "-shared", "-Xcompiler", "-fPIC", "-Xlinker", "-Bsymbolic",
                    "--cudart", "shared", "--expt-relaxed-constexpr", "-I", b.INC,
                    *(os.path.join(b.CSRC, n) for n in ("attn_api.cu", "pages_api.cu")),
                    *(os.path.join(ROOT, "tests", n) for n in ("fake_cuda.cpp", "fake_pages.cpp")), "-o", str(out)], check=True)
    L = C.CDLL(str(out))
    vp, i32 = C.c_void_p, C.c_int
    L.fake_log.restype = L.fake_pages_log.restype = L.moe_pages_last_error.restype = L.moe_kv_last_error.restype = C.c_char_p
    L.moe_pages_last_error.argtypes = L.moe_kv_last_error.argtypes = [vp]
    L.moe_pages_create.argtypes = L.moe_kv_create.argtypes = [vp, vp, C.POINTER(vp)]
    L.moe_pages_fork.argtypes = [vp] * 6
    L.moe_pages_compact.argtypes = [vp] * 3
    L.moe_pages_destroy.argtypes = L.moe_kv_destroy.argtypes = [vp]
    L.moe_pages_device_status.argtypes = [vp, C.POINTER(C.c_int32)]
    L.moe_kv_copy.argtypes = [vp, vp, i32, vp]
    L.A, L.G = A, pages
    return L


def at(device, offset=0):
    return ((device + 1) << 40) + offset


def test_calls_work_on_the_handle_s_device(lib):
    lib.fake_reset(1)
    h = C.c_void_p()
    cfg = lib.G.moe_pages_config_t(10, 64, 4, 32)
    far = lib.G.moe_pages_store_t(*(at(0 if i == 2 else 1, i << 20) for i in range(5)))
    assert lib.moe_pages_create(C.byref(cfg), C.byref(far), C.byref(h)) == INVALID and not h.value
    st = lib.G.moe_pages_store_t(*(at(1, i << 20) for i in range(5)))
    assert lib.moe_pages_create(C.byref(cfg), C.byref(st), C.byref(h)) == 0
    lib.fake_clear_log()
    lib.fake_make_current(0)
    a = [at(1, i << 21) for i in range(1, 5)]
    assert lib.moe_pages_fork(h, *a, None) == 0 and lib.moe_pages_fork(h, a[0], a[1], None, a[3], None) == 0
    assert lib.moe_pages_compact(h, a[0], None) == 0
    assert lib.fake_pages_log() == b"fork@1 fork@1 compact@1 " and lib.fake_current() == 0
    for i, name in enumerate((b"parent", b"added", b"keep", b"moves")):
        for bad in (at(0, 1 << 21), a[i] + 4, None if name != b"keep" else a[i] + 8):
            assert lib.moe_pages_fork(h, *(bad if j == i else x for j, x in enumerate(a)), None) == INVALID
            assert name in lib.moe_pages_last_error(h)
    assert lib.moe_pages_compact(h, None, None) == INVALID and lib.moe_pages_compact(h, at(0), None) == INVALID
    assert lib.fake_pages_log() == b"" and lib.fake_log() == b""
    flags = C.c_int32()
    lib.fake_set_flags(10)
    assert lib.moe_pages_device_status(h, C.byref(flags)) == CUDA and flags.value == 10
    assert b"free pages" in lib.moe_pages_last_error(h) and b"bounds" in lib.moe_pages_last_error(h)
    log = lib.fake_log().decode().split()
    assert log[:2] == ["sync@1", "memcpy@1"] and all(x.endswith("@1") for x in log) and lib.fake_current() == 0
    lib.fake_clear_log()
    lib.moe_pages_destroy(h)
    assert lib.fake_log() == b"sync@1 free@1 " and lib.fake_current() == 0


def test_copy_works_on_the_cache_s_device(lib):
    lib.fake_reset(2)
    h = C.c_void_p()
    cfg = lib.A.moe_kv_config_t(8, 2, 64, 16, 10, 4, 64, 128)
    st = lib.A.moe_kv_store_t(*(at(2, i << 20) for i in range(4)))
    assert lib.moe_kv_create(C.byref(cfg), C.byref(st), C.byref(h)) == 0
    lib.fake_make_current(0)
    assert lib.moe_kv_copy(h, at(2, 1 << 24), 5, None) == 0 and lib.fake_pages_log() == b"copy@2 " and lib.fake_current() == 0
    assert lib.moe_kv_copy(h, None, 0, None) == 0  # no moves
    assert lib.moe_kv_copy(h, at(2, 1 << 24), -1, None) == INVALID and lib.moe_kv_copy(None, at(2), 1, None) == INVALID
    for bad in (None, at(0), at(2, 4)):
        assert lib.moe_kv_copy(h, bad, 5, None) == INVALID and b"moves" in lib.moe_kv_last_error(h)
    assert lib.fake_pages_log() == b""
    lib.moe_kv_destroy(h)
