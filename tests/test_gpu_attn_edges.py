"""The attention-side operators where their inputs are unusual: far positions, scales that no write makes, rows that
no sequence covers, other streams."""
from __future__ import annotations

import importlib.util
import math
import os
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
    c = m.KVCache(*codes, *scales, n_q_heads=hq, max_seqs=len(lens), max_tokens=max(bt.cu[-1], sum(lens)),
                  max_kv_len=max(lens))
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


@pytest.mark.parametrize("new", [1, 70])
@pytest.mark.parametrize("dim", [64, 128])
def test_attend_and_read_agree_about_small_scales(m, new, dim):
    """Value scales at and below 2^-64, zero among them, on some pages and on all of them: attend's result is the
    softmax of what read returns, to attend's own tolerance and the 448 * 2^-64 that such a value may be off by."""
    bt, c, q = batch(m, [300, 90], [new, 1], 16, dim, 2, 8, seed=1)
    small = [2.0 ** -64, 2.0 ** -65, 2.0 ** -80, 2.0 ** -126, 2.0 ** -140, 0.0]
    lse = torch.empty(q.shape[:2], device=DEV)
    for whole in (False, True):
        for p in range(bt.n_pages):
            if whole or p % 2:
                c.v_scale[p] = small[p // 2 % 6]
        out = c.attend(q, bt.b, lse=lse)
        o, ref_lse, tol = R.attend(q, c.k_codes, c.v_codes, c.k_scale, c.v_scale, bt, dim ** -0.5)
        assert ((out.double() - o).abs() <= tol + 448 * 2.0 ** -64).all()
        assert ((lse.double() - ref_lse).abs() <= 2.0 ** -16 * (1 + ref_lse.abs())).all()
        assert c.device_status() == 0
    every = R.Batch([300, 90], [300, 90], 16, DEV, seed=1)
    assert every.table == bt.table
    values = c.read(every.b, dtype=torch.float32)[1].double()
    assert float(values.abs().max()) <= 448 * 2.0 ** -64


@pytest.mark.parametrize("new", [1, 70])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -1.0])
def test_attend_says_that_it_met_a_bad_scale(m, new, bad):
    bt, c, q = batch(m, [300, 90], [new, 1], 16, 64, 2, 8, seed=2)
    want = c.attend(q, bt.b)
    for scales in (c.k_scale, c.v_scale):
        keep = scales.clone()
        unused = next(p for p in range(bt.n_pages) if all(p not in row for row in bt.table))
        scales[unused] = bad
        assert torch.equal(c.attend(q, bt.b), want) and c.device_status() == 0
        scales[bt.table[0][3], 1] = bad
        out = c.attend(q, bt.b)
        with pytest.raises(m.MoeError, match="scale"):
            c.device_status()
        assert torch.equal(out[:, :4], want[:, :4]) and torch.equal(out[bt.cu[1]:], want[bt.cu[1]:])
        scales.copy_(keep)
    assert torch.equal(c.attend(q, bt.b), want) and c.device_status() == 0


@pytest.mark.parametrize("new", [1, 40])
def test_rows_that_no_sequence_covers_keep_what_they_held(m, new):
    """A graph may be replayed with fewer tokens than it was captured for, and a sequence may break its bounds."""
    bt, c, q = batch(m, [200, 90, 60], [new, new, new], 16, 64, 2, 8, seed=3)
    want, values = c.attend(q, bt.b), c.read(bt.b)
    assert c.device_status() == 0

    def run():
        out = torch.full_like(q, 7)
        lse = torch.full(q.shape[:2], 7.0, device=DEV)
        read = [torch.full_like(x, 7) for x in values]
        c.attend(q, bt.b, out=out, lse=lse)
        c.read(bt.b, k_out=read[0], v_out=read[1])
        return out, lse, *read

    bt.b.cu_q[3] = bt.cu[2]  # the last sequence has no tokens now
    bt.b.kv_len[2] = 0
    for x, y in zip(run(), (want, None, *values)):
        assert (x[2 * new:] == 7).all() and (y is None or torch.equal(x[:2 * new], y[:2 * new]))
    assert c.device_status() == 0
    bt.b.cu_q[3], bt.b.kv_len[2], bt.b.kv_len[1] = bt.cu[3], 60, -1
    for x, y in zip(run(), (want, None, *values)):
        assert (x[new:2 * new] == 7).all()
        assert y is None or (torch.equal(x[:new], y[:new]) and torch.equal(x[2 * new:], y[2 * new:]))
    with pytest.raises(m.MoeError, match="bounds"):
        c.device_status()


@pytest.mark.parametrize("new", [5, 60])
def test_rows_below_position_zero(m, new):
    """More new tokens than cached ones: nothing to see for the first rows under the causal mask, all without."""
    bt, c, q = batch(m, [3, 0], [new, 2], 16, 64, 1, 2, seed=4)
    q[1:new] = q[0]  # the rows then differ by what they see alone
    lse = torch.empty(q.shape[:2], device=DEV)
    out = c.attend(q, bt.b, lse=lse)
    assert not out[:new - 3].any() and lse[:new - 3].isneginf().all() and lse[new - 3:new].isfinite().all()
    whole = c.attend(q, bt.b, lse=lse, causal=False)
    assert torch.equal(whole[:new], out[new - 1:new].expand(new, 2, 64)) and lse[:new].isfinite().all()
    assert not whole[new:].any() and lse[new:].isneginf().all() and c.device_status() == 0


def test_the_example_does_not_hide_what_is_not_finite(m, monkeypatch):
    """Its difference is NaN where a result is, for both sequences and for the second alone."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decoder_step.py")
    spec = importlib.util.spec_from_file_location("decoder_step", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    step = ex.DecoderLayer.step
    for bad in (slice(None), slice(1, 2)):
        def broken(self, x, news):
            y = step(self, x, news)
            if news == [1, 1]:
                y[bad] = math.nan
            return y

        monkeypatch.setattr(ex.DecoderLayer, "step", broken)
        assert math.isnan(ex.main())
