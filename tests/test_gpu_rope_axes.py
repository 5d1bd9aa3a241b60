"""Rotary positions with several axes against 64 bits."""
from __future__ import annotations

import random

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def m():
    from int4_routed_expert_gb300 import build as b
    b.build()
    import int4_routed_expert_gb300 as mod
    mod.load()
    return mod


def reference(x, pos, axes, freq, amp, interleaved):
    """Pair by pair, from the definition."""
    y = x.double().clone()
    for i, (a, f) in enumerate(zip(axes, freq)):
        angle = pos[a].double() * f
        c, s = amp * torch.cos(angle)[:, None], amp * torch.sin(angle)[:, None]
        u, v = (2 * i, 2 * i + 1) if interleaved else (i, i + len(freq))
        p, q = x[..., u].double(), x[..., v].double()
        y[..., u], y[..., v] = p * c - q * s, p * s + q * c
    return y


def close(y, x, ref, amp):
    """A turn's sine and cosine are off by at most 4 ulp, the two products and their sum by one each: 2^-21 of the
    pair's magnitude, and half a step of the type (bf16 2^-8, fp32 2^-24 of the result)."""
    half = 2.0 ** -8 if x.dtype == torch.bfloat16 else 2.0 ** -24
    tol = half * ref.abs() + 2.0 ** -21 * amp * 1.5 * x.double().abs().amax(-1, keepdim=True) + 1e-37
    assert ((y.double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,heads,kv,dim,rot,n_axes", [(1, 1, 1, 64, 64, 3), (3, 5, 2, 128, 32, 2), (257, 6, 1, 128, 128, 3),
                                                       (33, 3, 0, 256, 256, 4), (17, 2, 1, 96, 16, 1), (2051, 2, 1, 64, 64, 3)])
def test_axes(m, T, heads, kv, dim, rot, n_axes, interleaved, dtype):
    g = torch.Generator(DEV)
    g.manual_seed(T + dim)
    r = random.Random(rot)
    axes = [r.randrange(n_axes) for _ in range(rot // 2 - n_axes)] + list(range(n_axes))
    rope = m.Rope(rot, theta=1e6, interleaved=interleaved, scaling="yarn", factor=8.0, original_len=4096, axes=axes)
    pos = torch.randint(-5, 1 << 20, (n_axes, T + 8), device=DEV, generator=g).int()
    pos[:, 0] = 2 ** 31 - 1
    pos[-1, 0] = -2 ** 31
    at = pos[:, :T]  # rows further apart than their tokens
    q = torch.randn(T, heads, dim, device=DEV, generator=g).to(dtype)
    k = torch.randn(T, kv, dim, device=DEV, generator=g).to(dtype) if kv else None
    out = rope.apply(q, at, k=k)
    again = rope.apply(q, at.contiguous(), k=k)
    for x, y, z in ((q, out, again),) if not kv else ((q, out[0], again[0]), (k, out[1], again[1])):
        close(y, x, reference(x, at, axes, rope.inv_freq, rope.amplitude, interleaved), rope.amplitude)
        assert torch.equal(y[..., rot:], x[..., rot:]) and torch.equal(y, z)
    rope.apply(q, at, k=k, q_out=q, k_out=k)  # in place
    assert torch.equal(q, out[0] if kv else out)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_alike_positions_are_plain_ones(m, dtype):
    """Text: every axis has the same position, and the result is that of one axis, bit for bit."""
    q = torch.randn(300, 6, 64, device=DEV).to(dtype)
    pos = (torch.arange(300, device=DEV) * 977).int()
    plain = m.Rope(64, theta=1e6).apply(q, pos)
    for axes in (m.rope_axes(64, (8, 12, 12)), m.rope_axes(64, (8, 12, 12), turns=True), m.rope_axes(64, (16, 16))):
        assert torch.equal(m.Rope(64, theta=1e6, axes=axes).apply(q, pos.expand(max(axes) + 1, -1).contiguous()), plain)
    assert torch.equal(m.Rope(64, theta=1e6, axes=[0] * 32).apply(q, pos[None]), plain)


def test_a_captured_call_follows_its_positions(m):
    q = torch.randn(40, 4, 64, device=DEV).bfloat16()
    axes = m.rope_axes(64, (8, 12, 12))
    rope = m.Rope(64, axes=axes)
    pos = torch.zeros(3, 40, dtype=torch.int32, device=DEV)
    out = torch.empty_like(q)
    rope.apply(q, pos, q_out=out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rope.apply(q, pos, q_out=out)
    pos.copy_(torch.randint(0, 5000, (3, 40), device=DEV))
    g.replay()
    close(out, q, reference(q, pos, axes, rope.inv_freq, 1.0, False), 1.0)


def test_refusals(m):
    rope = m.Rope(64, axes=m.rope_axes(64, (8, 12, 12)))
    q = torch.zeros(4, 2, 64, device=DEV)
    pos = torch.zeros(3, 4, dtype=torch.int32, device=DEV)
    for bad in (pos.long(), pos[:2], pos[0], pos[:, :3], pos.T.contiguous().T, pos.cpu(), torch.zeros(3, 8, device=DEV).int()[:, ::2],
                pos[0].expand(3, 4)):
        with pytest.raises(ValueError):
            rope.apply(q, bad)
    with pytest.raises(ValueError):
        m.Rope(64).apply(q, pos)
    assert rope.apply(q[:0], pos[:, :0].contiguous()).shape == (0, 2, 64)
