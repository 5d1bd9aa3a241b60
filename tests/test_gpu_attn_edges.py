"""The attention-side operators where their inputs are unusual: far positions, scales that no write makes, rows that
no sequence covers, other streams."""
from __future__ import annotations

import math
import random
from fractions import Fraction

import pytest
import torch

import attn_ref as R
from turns import TWO_PI

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def m():
    from int4_routed_expert_gb300 import build as b
    b.build()
    import int4_routed_expert_gb300 as mod
    mod.load()
    return mod


def test_rope_angles_at_far_positions(m):
    """Rotating (1, 0) gives the cosine and the sine themselves.  Off by at most 2 ulp of the library's function
    (2^-23) and half an ulp of the step by the derivatives (2^-25); the angle's 2^-32 turns are 2^-29."""
    r = random.Random(5)
    freq = [1.0] + [r.uniform(0.5, 1.2) for _ in range(95)] + [math.exp(r.uniform(-16, 0)) for _ in range(32)]
    pos = [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 12345, 2 ** 30 + 7, -1999999999, 4000037, 131071, 1000, 1, 0]
    rope = m.Rope(256, inv_freq=freq, amplitude=1.0)
    x = torch.zeros(len(pos), 1, 256, device=DEV)
    x[..., :128] = 1
    y = rope.apply(x, torch.tensor(pos, dtype=torch.int32, device=DEV)).double().cpu()
    for t, p in enumerate(pos):
        angle = [float(p * Fraction(f) % TWO_PI) for f in freq]
        want = torch.tensor([math.cos(a) for a in angle] + [math.sin(a) for a in angle], dtype=torch.float64)
        assert float((y[t, 0] - want).abs().max()) <= 2.0 ** -23 + 2.0 ** -25 + 2.0 ** -29


def batch(m, lens, news, page, dim, hkv, hq, seed=0):
    """(Batch, cache with normal codes, queries) of sequences."""
    g = torch.Generator(DEV)
    g.manual_seed(seed)
    bt = R.Batch(lens, news, page, DEV, seed=seed)
    shape = (bt.n_pages, hkv, page, dim)
    codes = [torch.randn(*shape, device=DEV, generator=g).to(R.F8) for _ in range(2)]
    scales = [torch.exp2(torch.randint(-6, 3, shape[:2], device=DEV, generator=g).float()) for _ in range(2)]
    c = m.KVCache(*codes, *scales, n_q_heads=hq, max_seqs=len(lens), max_tokens=bt.cu[-1], max_kv_len=max(lens))
    return bt, c, torch.randn(bt.cu[-1], hq, dim, device=DEV, generator=g).bfloat16()


def owner(t):
    """The stream whose memory a tensor's is."""
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("not the allocator's")


def test_results_belong_to_the_stream_that_writes_them(m):
    """Memory of the current stream may still be in use there, or be given away there, while `stream` writes."""
    bt, c, q = batch(m, [90, 40], [3, 2], 16, 64, 2, 4)
    k = q[:, :2].contiguous()
    pos = torch.arange(5, dtype=torch.int32, device=DEV)
    rope = m.Rope(64)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    results = [rope.apply(q, pos, stream=s), *rope.apply(q, pos, k=k, stream=s), *rope.apply(q[..., :], pos, k=q[:, 1:3], stream=s),
               rope.apply(q, pos, k=k, q_out=torch.empty_like(q), stream=s)[1], *c.read(bt.b, stream=s),
               c.attend(q, bt.b, stream=s), c.attend(torch.cat((q, q), 1)[:, :4], bt.b, stream=s)]
    s.synchronize()
    assert [owner(t) for t in results] == [s.cuda_stream] * len(results)
    assert owner(c.attend(q, bt.b)) == owner(q) != s.cuda_stream


def test_read_takes_the_type_of_a_given_result(m):
    bt, c, _ = batch(m, [90, 40], [90, 40], 16, 64, 2, 4)
    want = c.read(bt.b, dtype=torch.float32)
    for name in ("k_out", "v_out"):
        given = torch.empty_like(want[0])
        got = c.read(bt.b, **{name: given})
        assert got[name == "v_out"] is given
        assert all(y.dtype == torch.float32 and torch.equal(y, x) for x, y in zip(want, got))
    with pytest.raises(ValueError):
        c.read(bt.b, k_out=torch.empty_like(want[0]), v_out=torch.empty_like(want[0]).bfloat16())
