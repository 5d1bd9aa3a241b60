"""Host side of rotary positions with several axes: what is refused before any launch, the layouts of the axes."""
from __future__ import annotations

import ctypes as C

import pytest

INVALID, UNSUPPORTED = -1, -2


@pytest.fixture(scope="module")
def A():
    from int4_routed_expert_gb300 import build as b
    b.build()
    from int4_routed_expert_gb300 import attn
    attn._load()
    return attn


@pytest.mark.parametrize("n_axes,axis,status", [(0, [0] * 8, UNSUPPORTED), (5, [0] * 8, UNSUPPORTED), (2, None, INVALID),
                                                (2, [0] * 7 + [2], INVALID), (2, [-1] + [0] * 7, INVALID), (3, [0, 1, 2] * 2 + [0, 1], 0),
                                                (4, [3] * 8, 0)])
def test_create(A, n_axes, axis, status):
    h = C.c_void_p(1)
    f, a = (C.c_double * 8)(*[0.5] * 8), (C.c_int32 * 8)(*axis) if axis else None
    assert A._lib.moe_rope_create_axes(16, f, 1.0, 0, n_axes, a, C.byref(h)) == status and bool(h.value) == (status == 0)
    A._lib.moe_rope_destroy(h)
    assert A._lib.moe_rope_create_axes(16, f, 1.0, 0, n_axes, a, None) == INVALID
    assert A._lib.moe_rope_create_axes(24, f, 1.0, 0, n_axes, a, C.byref(h)) == UNSUPPORTED


def test_apply_refuses(A):
    r = A.Rope(32, axes=[0, 1] * 8)
    T = A.moe_rope_tensor_t
    ok = T(0x10000, 0x20000, 2, 128, 128)
    call = lambda q=ok, dim=64, dt=1, pos=0x1000, stride=3, n=3, h=r.h: A._lib.moe_rope_apply_axes(  # noqa: E731
        h, C.byref(q) if q else None, None, dim, dt, pos, stride, n, None)
    assert call(h=None) == INVALID and call(q=None) == INVALID and call(dim=72) == UNSUPPORTED and call(dt=2) == INVALID
    assert call(n=-1) == INVALID and call(q=T(0x10000, 0x20000, 2, 120, 128)) == INVALID
    assert call(n=0) == 0
    assert call() == INVALID  # addresses that the driver does not know
    assert A._lib.moe_rope_apply(r.h, C.byref(ok), None, 64, 1, 0x1000, 0, None) == INVALID
    assert "axes" in A.moe.moe_last_error(None)
    with pytest.raises(ValueError):
        A.Rope(32, axes=[0] * 15)
    with pytest.raises(A.MoeError):
        A.Rope(32, axes=[4] * 16)
    with pytest.raises(A.MoeError):
        A.Rope(32, axes=[-1] * 16)


def test_layouts(A):
    assert A.rope_axes(16, (2, 3, 3)) == [0, 0, 1, 1, 1, 2, 2, 2]
    assert A.rope_axes(16, (2, 3, 3), turns=True) == [0, 1, 2, 0, 1, 2, 1, 2]
    assert A.rope_axes(16, (0, 8), turns=True) == [1] * 8
    for bad in ((4, 3), (9, -1), ()):
        with pytest.raises(ValueError):
            A.rope_axes(16, bad)
