"""Rotary positions, the 8-bit paged cache and attention over it against 64-bit references."""
from __future__ import annotations

import math

import pytest
import torch

import attn_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def m():
    from int4_routed_expert_gb300 import build as b
    b.build()
    import int4_routed_expert_gb300 as mod
    mod.load()
    return mod


def gen(seed):
    g = torch.Generator(DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, device=DEV, generator=g).to(dtype)


# ------------------------------------------------------------------- rope --

def rope_close(y, x, ref, amp):
    """fp32: a turn's sine and cosine are off by at most 4 ulp (the library's bound for sincospi with the phase's
    half step), the two products and their sum by one each: 2^-21 of the pair's magnitude.  bf16 adds half a
    step, 2^-8 of the result."""
    half = 2.0 ** -8 if x.dtype == torch.bfloat16 else 2.0 ** -24
    tol = half * ref.abs() + 2.0 ** -21 * amp * 1.5 * x.double().abs().amax(-1, keepdim=True) + 1e-37
    assert ((y.double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,heads,kv,dim,rot", [(1, 1, 1, 64, 64), (3, 5, 2, 128, 32), (257, 6, 1, 128, 128),
                                                (33, 3, 0, 256, 256), (17, 2, 1, 96, 16)])
def test_rope(m, T, heads, kv, dim, rot, interleaved, dtype):
    g = gen(T + dim)
    r = m.Rope(rot, theta=1e6, interleaved=interleaved, scaling="yarn", factor=8.0, original_len=4096)
    pos = torch.randint(-5, 1 << 20, (T,), device=DEV, generator=g).int()
    pos[0] = 2 ** 31 - 1
    q = randn(g, T, heads, dim, dtype=dtype)
    k = randn(g, T, kv, dim, dtype=dtype) if kv else None
    out = r.apply(q, pos, k=k)
    for x, y in ((q, out[0] if kv else out),) + (((k, out[1]),) if kv else ()):
        rope_close(y, x, R.rope(x, pos, r.inv_freq, r.amplitude, interleaved), r.amplitude)
        assert torch.equal(y[..., rot:], x[..., rot:])


def test_rope_strided_and_in_place(m):
    g = gen(5)
    T, D = 37, 64
    qkv = randn(g, T, (6 + 2 + 2) * D, dtype=torch.bfloat16)
    keep = qkv.clone()
    q, k = qkv[:, :6 * D].unflatten(1, (6, D)), qkv[:, 6 * D:8 * D].unflatten(1, (2, D))
    pos = torch.arange(T, device=DEV, dtype=torch.int32) * 1000
    r = m.Rope(D)
    q0, k0 = r.apply(q, pos, k=k)
    r.apply(q, pos, k=k, q_out=q, k_out=k)
    assert torch.equal(q, q0) and torch.equal(k, k0)
    assert torch.equal(qkv[:, 8 * D:], keep[:, 8 * D:])
    rope_close(q0, keep[:, :6 * D].unflatten(1, (6, D)),
               R.rope(keep[:, :6 * D].unflatten(1, (6, D)), pos, r.inv_freq, 1.0, False), 1.0)
    assert r.apply(q[:0], pos[:0]).shape == (0, 6, D)


def test_rope_refuses(m):
    r = m.Rope(64)
    q = torch.zeros(4, 2, 64, device=DEV)
    pos = torch.zeros(4, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError):
        r.apply(q, pos.long())
    with pytest.raises(ValueError):
        r.apply(q, pos[:3])
    with pytest.raises(TypeError):
        r.apply(q.half(), pos)
    with pytest.raises(ValueError):
        r.apply(q, pos, k=q.bfloat16())
    with pytest.raises(m.MoeError):
        r.apply(torch.zeros(4, 2, 48, device=DEV), pos)  # narrower than rot_dim


# ------------------------------------------------------------------ cache --

def make_cache(m, g, bt, hq, hkv, dim, scales=None, fill="random", n_tokens=None):
    """A cache whose pages hold random codes (no NaN), stale ones behind every sequence's end included."""
    shape = (bt.n_pages, hkv, bt.page, dim)
    codes = []
    for _ in range(2):
        c = torch.randint(0, 127, shape, device=DEV, generator=g, dtype=torch.uint8)  # 0x7f is NaN
        c |= torch.randint(0, 2, shape, device=DEV, generator=g, dtype=torch.uint8) << 7
        if fill == "normal":
            c = randn(g, *shape).to(F8).view(torch.uint8)
        codes.append(c)
    sc = scales or [torch.exp2(torch.randint(-6, 3, shape[:2], device=DEV, generator=g).float()) for _ in range(2)]
    return m.KVCache(*codes, *sc, n_q_heads=hq, max_seqs=max(len(bt.lens), 1), max_tokens=max(bt.cu[-1], 1),
                     max_kv_len=max(max(bt.lens), 1))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("page,dim", [(16, 64), (32, 128), (64, 64), (128, 128)])
def test_write_and_read(m, page, dim, dtype):
    g = gen(page)
    hkv = 3
    lens, news = [1, page, page + 1, 3 * page + 5, 5, 0, 2, 700, 64], [1, page, 1, 2 * page, 5, 0, 4, 411, 0]
    bt = R.Batch(lens, news, page, DEV, seed=1, slack=2)
    c = make_cache(m, g, bt, hkv, hkv, dim)
    T = bt.cu[-1]
    k = randn(g, T, hkv, dim) * torch.exp2(torch.randint(-12, 12, (T, hkv, 1), device=DEV, generator=g).float())
    v = randn(g, T, hkv, dim) * 1e-3
    v[3] = 0
    k, v = k.to(dtype), v.to(dtype)
    want = [R.write(x, c0, s0, bt) for x, c0, s0 in ((k, c.k_codes, c.k_scale), (v, c.v_codes, c.v_scale))]
    c.write(k, v, bt.b)
    for (wc, ws), gc, gs in zip(want, (c.k_codes, c.v_codes), (c.k_scale, c.v_scale)):
        assert torch.equal(gs.double(), ws)
        assert torch.equal(gc.view(F8).double(), wc)
    assert c.device_status() == 0
    for out_dtype in (torch.bfloat16, torch.float32):
        got = c.read(bt.b, dtype=out_dtype)
        for y, x, codes, scales in ((got[0], k, c.k_codes, c.k_scale), (got[1], v, c.v_codes, c.v_scale)):
            rows = set()
            for row, b, t in bt.places():
                rows.add(row)
                p = bt.table[b][t // page]
                ref = codes.view(F8)[p, :, t % page].double() * scales[p].double()[:, None]
                assert torch.equal(y[row].double(), ref)  # a code times a power of two: exact in either type
            for row in set(range(T)) - rows:
                assert not y[row].any()  # a position below 0


def test_write_one_token_at_a_time(m):
    """Growing a sequence token by token gives each block the scale of its largest value so far, and every code
    within half a step (and the re-encodings' underflow) of its value."""
    g = gen(9)
    page, dim, n = 16, 64, 37
    x = randn(g, n, 1, dim) * torch.exp2(torch.arange(n, device=DEV).float() % 7)[:, None, None]
    bt = R.Batch([n], [n], page, DEV)
    c = make_cache(m, g, bt, 1, 1, dim)
    table = bt.b.page_table
    for i in range(n):
        i32 = dict(dtype=torch.int32, device=DEV)
        b = m.SeqBatch(torch.tensor([0, 1], **i32), torch.tensor([i + 1], **i32), table, 1, 1, i + 1)
        c.write(x[i:i + 1], x[i:i + 1], b)
    got = c.read(bt.b, dtype=torch.float32)[0].double()
    for p in range(-(-n // page)):
        rows = x[p * page:(p + 1) * page].double()
        s = R.pow2_scale(float(rows.abs().max()))
        assert float(c.k_scale[bt.table[0][p], 0]) == s
        # half a step, at most one more per re-encoding of a subnormal (steps of 2^-9 of a scale), 6 growths
        tol = 2.0 ** -4 * rows.abs() + 7 * s * 2.0 ** -10
        assert ((got[p * page:(p + 1) * page] - rows).abs() <= tol).all()


def test_write_non_finite(m):
    g = gen(4)
    bt = R.Batch([20], [20], 16, DEV)
    c = make_cache(m, g, bt, 1, 1, 64)
    k, v = randn(g, 20, 1, 64), randn(g, 20, 1, 64)
    k[2, 0, 5], k[3, 0, 6], v[17, 0, 0] = math.nan, -math.inf, math.inf
    want = R.write(k, c.k_codes, c.k_scale, bt), R.write(v, c.v_codes, c.v_scale, bt)
    c.write(k, v, bt.b)
    assert torch.equal(c.k_codes.view(F8).double(), want[0][0]) and torch.equal(c.v_codes.view(F8).double(), want[1][0])
    assert torch.equal(c.k_scale.double(), want[0][1]) and torch.equal(c.v_scale.double(), want[1][1])
    with pytest.raises(m.MoeError, match="NaN or infinity"):
        c.device_status()
    assert c.device_status() == 0
    # rows of zeros and of the smallest and largest magnitudes
    k[:] = 0
    v[:10], v[10:] = 1e-38, 3e38
    c.write(k, v, bt.b)
    r = c.read(bt.b, dtype=torch.float32)
    assert not r[0].any() and (c.k_scale[bt.table[0][0]] == 2.0 ** -64).all()
    assert ((r[1][10:].double() - v[10:].double()).abs() <= 2.0 ** -4 * v[10:].double()).all()
    assert c.device_status() == 0


# -------------------------------------------------------------- attention --

def check(c, bt, q, scale=None, **kw):
    lse = torch.empty(q.shape[:2], device=DEV)
    out = c.attend(q, bt.b, lse=lse, scale=scale, **kw)
    o, l, tol = R.attend(q, c.k_codes, c.v_codes, c.k_scale, c.v_scale, bt,
                         q.shape[-1] ** -0.5 if scale is None else scale, **kw)
    err = (out.double() - o).abs()
    assert (err <= tol).all(), f"error {float((err / tol).max()):.3g} of its bound"
    fin = torch.isfinite(l)
    assert torch.equal(torch.isfinite(lse), fin)
    # the logits' own error moves lse by as much; 2^-16 for it, logarithms and sums
    assert ((lse.double() - l).abs()[fin] <= 2.0 ** -16 * (1 + l.abs()[fin])).all()
    assert c.device_status() == 0
    return out


SHAPES = [  # lens, new, heads, kv heads, dim, page
    ([1], [1], 1, 1, 64, 16),
    ([2, 1], [1, 1], 4, 2, 128, 16),
    ([33, 0, 777], [1, 1, 1], 6, 1, 128, 64),
    ([5000], [1], 8, 2, 64, 32),
    ([3001, 40], [1, 1], 24, 2, 128, 128),
    ([130, 9], [4, 3], 12, 1, 128, 16),
    ([2049], [8], 16, 4, 64, 64),
    ([17], [17], 7, 7, 128, 32),
    ([300, 1, 45], [300, 1, 12], 6, 2, 128, 64),
    ([1000], [129], 8, 1, 64, 16),
    ([777, 513], [300, 513], 12, 2, 128, 128),
    ([3], [5], 2, 1, 64, 16),  # more new tokens than cached ones
    ([600, 700, 0, 64], [64, 128, 3, 64], 4, 1, 128, 32),
]


@pytest.mark.parametrize("lens,news,hq,hkv,dim,page", SHAPES)
@pytest.mark.parametrize("mask", [dict(), dict(causal=False), dict(window=40, sinks=3), dict(window=1), dict(window=128, sinks=130)])
def test_attend(m, lens, news, hq, hkv, dim, page, mask):
    g = gen(len(lens) + hq + dim)
    bt = R.Batch(lens, news, page, DEV, seed=3)
    c = make_cache(m, g, bt, hq, hkv, dim, fill="normal")
    check(c, bt, randn(g, bt.cu[-1], hq, dim, dtype=torch.bfloat16), **mask)


@pytest.mark.parametrize("new", [1, 150])
def test_attend_wild_scales(m, new):
    """Blocks whose scales differ by 2^40, and any positive scale, not only powers of two: the blocks with small
    values dominate some rows, so their weights must not underflow."""
    g = gen(11)
    hq, hkv, dim, page = 4, 1, 128, 16
    bt = R.Batch([500], [new], page, DEV)
    shape = (bt.n_pages, hkv)
    ks = 0.02 * torch.rand(shape, device=DEV, generator=g) + 0.001
    vs = torch.exp2(40 * torch.rand(shape, device=DEV, generator=g) - 20)
    c = make_cache(m, g, bt, hq, hkv, dim, scales=[ks, vs])
    check(c, bt, randn(g, new, hq, dim, dtype=torch.bfloat16) * 0.1)


@pytest.mark.parametrize("new", [1, 200])
def test_attend_query_ranges(m, new):
    """Rows of very small and very large queries, zero rows, a NaN row: a row never touches another."""
    g = gen(12)
    hq, hkv, dim = 8, 2, 64
    bt = R.Batch([400], [new], 16, DEV)
    c = make_cache(m, g, bt, hq, hkv, dim, fill="normal")
    q = randn(g, new, hq, dim)
    q[:, 0] *= 1e-30
    q[:, 1] = 0
    q[:, 2] *= 100
    q[:, 3, ::2] *= 1e-6
    q = q.bfloat16()
    out = check(c, bt, q)
    q[:, 5, 7] = math.nan
    q[:, 6, 9] = math.inf
    again = c.attend(q, bt.b)
    assert again[:, 5:7].isnan().all()
    keep = [0, 1, 2, 3, 4, 7]
    assert torch.equal(again[:, keep], out[:, keep])


@pytest.mark.parametrize("new,window", [(1, 0), (3, 0), (1, 50), (200, 0), (200, 50)])
def test_attend_ignores_what_no_row_sees(m, new, window):
    """NaN codes and NaN scales behind a sequence's end, before its window and in unused pages change nothing."""
    g = gen(13)
    hq, hkv, dim, page, length = 6, 2, 128, 16, 389
    bt = R.Batch([length], [new], page, DEV, spare=4)
    c = make_cache(m, g, bt, hq, hkv, dim, fill="normal")
    q = randn(g, new, hq, dim, dtype=torch.bfloat16)
    kw = dict(window=window, sinks=2) if window else {}
    out = check(c, bt, q, **kw)
    used = bt.table[0]
    low = length - new - window + 1 if window else 0  # the first token in some row's window
    for codes, scales in ((c.k_codes, c.k_scale), (c.v_codes, c.v_scale)):
        codes[used[-1], :, length % page:] = 0x7f
        for p in range(bt.n_pages):
            at = used.index(p) if p in used else -1
            if at < 0 or (window and at > 0 and (at + 1) * page <= low // 64 * 64):
                codes[p] = 0x7f
                scales[p] = math.nan
    assert torch.equal(c.attend(q, bt.b, **kw), out)


def test_attend_strides_and_streams(m):
    """Queries as part of a projection's rows, on a stream of their own; the same call gives the same bits."""
    g = gen(14)
    hq, hkv, dim = 6, 2, 64
    bt = R.Batch([900, 300], [5, 130], 32, DEV)
    c = make_cache(m, g, bt, hq, hkv, dim, fill="normal")
    qkv = randn(g, bt.cu[-1], (hq + 2 * hkv) * dim, dtype=torch.bfloat16)
    q = qkv[:, :hq * dim].unflatten(1, (hq, dim))
    want = check(c, bt, q.contiguous())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a = c.attend(q, bt.b)
        b = c.attend(q, bt.b)
    s.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want)


def test_attend_far_pages(m):
    """Pages whose bytes lie beyond 2^32: offsets are 64-bit."""
    hq, hkv, dim, page = 8, 8, 128, 64
    pool = 2 ** 32 // (hkv * dim * page) + 40
    if torch.cuda.mem_get_info()[0] < 6 * 2 ** 32:
        pytest.skip("not enough free memory")
    g = gen(15)
    bt = R.Batch([200, 777], [1, 300], page, DEV, base=pool - 25, pool=pool)
    codes = [torch.zeros(pool, hkv, page, dim, dtype=torch.uint8, device=DEV) for _ in range(2)]
    scales = [torch.ones(pool, hkv, device=DEV) for _ in range(2)]
    c = m.KVCache(*codes, *scales, n_q_heads=hq, max_seqs=2, max_tokens=1200, max_kv_len=777)
    whole = R.Batch([200, 777], [200, 777], page, DEV, base=pool - 25, pool=pool)
    assert whole.table == bt.table
    k, v = randn(g, 977, hkv, dim, dtype=torch.bfloat16), randn(g, 977, hkv, dim, dtype=torch.bfloat16)
    c.write(k, v, whole.b)
    assert not codes[0][:pool - 26].any()
    got = c.read(whole.b)
    assert ((got[0].double() - k.double()).abs() <= 2.0 ** -4 * k.double().abs() + 2.0 ** -8).all()
    q = randn(g, bt.cu[-1], hq, dim, dtype=torch.bfloat16)
    check(c, bt, q)


@pytest.mark.parametrize("new", [1, 140])
def test_graph_replays_with_other_lengths(m, new):
    """A captured step replays with other lengths, pages and contents within the host's bounds."""
    g = gen(16)
    hq, hkv, dim, page = 8, 2, 64, 16
    big = R.Batch([700, 650], [new, new], page, DEV, seed=1)
    c = make_cache(m, g, big, hq, hkv, dim, fill="normal")
    q, k, v = (randn(g, 2 * new, h, dim, dtype=torch.bfloat16) for h in (hq, hkv, hkv))
    pos = torch.zeros(2 * new, dtype=torch.int32, device=DEV)
    r = m.Rope(dim)
    out = torch.empty(2 * new, hq, dim, dtype=torch.bfloat16, device=DEV)

    def step():
        q2, k2 = r.apply(q, pos, k=k)
        c.write(k2, v, big.b)
        c.attend(q2, big.b, out=out)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for lens in ([700, 650], [300, new], [new + 1, 512]):
        bt = R.Batch(lens, [new, new], page, DEV, seed=2, pool=big.n_pages)
        t = torch.full_like(big.b.page_table, -1)
        t[:, :bt.b.page_table.shape[1]] = bt.b.page_table
        big.b.page_table.copy_(t)
        big.b.kv_len.copy_(bt.b.kv_len)
        pos.copy_(torch.cat([torch.arange(n - new, n, device=DEV) for n in lens]).int())
        q.copy_(randn(g, *q.shape))
        k.copy_(randn(g, *k.shape))
        want = R.write(r.apply(k, pos), c.k_codes, c.k_scale, bt)
        graph.replay()
        torch.cuda.synchronize()
        q2 = r.apply(q, pos)
        o, _, tol = R.attend(q2, c.k_codes, c.v_codes, c.k_scale, c.v_scale, bt, dim ** -0.5)
        assert ((out.double() - o).abs() <= tol).all()
        assert torch.equal(c.k_codes.view(F8).double(), want[0]) and torch.equal(c.k_scale.double(), want[1])
    assert c.device_status() == 0


def test_bad_batches_are_flagged(m):
    """Device arrays that break the bounds: nothing out of bounds is touched, the other sequences are computed,
    the status word says so."""
    g = gen(17)
    hq, hkv, dim, page = 4, 2, 64, 16
    good = R.Batch([100, 80, 60], [1, 1, 1], page, DEV)
    c = make_cache(m, g, good, hq, hkv, dim, fill="normal")
    q = randn(g, 3, hq, dim, dtype=torch.bfloat16)
    want = c.attend(q, good.b)
    k = randn(g, 3, hkv, dim, dtype=torch.bfloat16)
    for field, index, value in (("page_table", (1, 2), good.n_pages), ("page_table", (1, 2), -7),
                                ("kv_len", (1,), 101), ("kv_len", (1,), -1), ("kv_len", (1,), 2 ** 31 - 1),
                                ("cu_q", (2,), 7), ("cu_q", (2,), -3)):
        t = getattr(good.b, field)
        old = int(t[index])
        t[index] = value
        out = c.attend(q, good.b)
        with pytest.raises(m.MoeError, match="bounds"):
            c.device_status()
        assert torch.equal(out[0], want[0])
        if field != "cu_q":
            assert torch.equal(out[2], want[2])
        if field != "page_table":  # (the page written is another one there)
            state = (c.k_codes, c.v_codes, c.k_scale, c.v_scale)
            before = [x.clone() for x in state]
            c.write(k, k, good.b)
            c.read(good.b)
            with pytest.raises(m.MoeError, match="bounds"):
                c.device_status()
            for now, then in zip(state, before):
                now.copy_(then)
        t[index] = old
    assert torch.equal(c.attend(q, good.b)[1], want[1])


def test_refusals(m):
    g = gen(18)
    bt = R.Batch([100], [4], 16, DEV)
    c = make_cache(m, g, bt, 4, 2, 64)
    q = randn(g, 4, 4, 64, dtype=torch.bfloat16)
    for bad in (q.float(), q.half()):
        with pytest.raises(TypeError):
            c.attend(bad, bt.b)
    for bad in (q[:3], q[:, :3], q.cpu(), q.transpose(0, 1), q[..., :32]):
        with pytest.raises(ValueError):
            c.attend(bad, bt.b)
    with pytest.raises(ValueError):
        c.attend(q, bt.b, out=torch.empty(4, 4, 64, device=DEV))
    with pytest.raises(ValueError):
        c.attend(q, bt.b, lse=torch.empty(4, 3, device=DEV))
    for kw in (dict(window=-1), dict(window=5, sinks=-1), dict(causal=False, window=5), dict(causal=False, sinks=5),
               dict(scale=math.nan), dict(scale=math.inf)):
        with pytest.raises(m.MoeError):
            c.attend(q, bt.b, **kw)
    k = q[:, :2]
    with pytest.raises(TypeError):
        c.write(k.contiguous(), k.float().contiguous(), bt.b)
    with pytest.raises(ValueError):
        c.write(q, q, bt.b)  # the query's heads
    i32 = dict(dtype=torch.int32, device=DEV)
    over = m.SeqBatch(torch.tensor([0, 5], **i32), torch.tensor([100], **i32), bt.b.page_table, 5, 5, 100)
    with pytest.raises(m.MoeError, match="exceeds"):
        c.attend(randn(g, 5, 4, 64, dtype=torch.bfloat16), over)
    st = torch.zeros(2, 2, 16, 64, dtype=torch.uint8, device=DEV)
    with pytest.raises(ValueError):
        m.KVCache(st, st, torch.ones(2, 1, device=DEV), torch.ones(2, 2, device=DEV), 2, 1, 1, 1)
    # nothing to do
    empty = m.SeqBatch(torch.zeros(1, **i32), torch.zeros(0, **i32), torch.zeros(0, 1, **i32), 0, 0, 0)
    assert c.attend(q[:0], empty).shape == (0, 4, 64)


def test_no_allocation_after_create(m):
    """Calls with outputs given allocate nothing on the device."""
    g = gen(19)
    bt = R.Batch([500, 40], [1, 1], 16, DEV)
    c = make_cache(m, g, bt, 4, 2, 64)
    q = randn(g, 2, 4, 64, dtype=torch.bfloat16)
    out = torch.empty_like(q)
    c.attend(q, bt.b, out=out)
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    for _ in range(5):
        c.attend(q, bt.b, out=out)
    torch.cuda.synchronize()
    assert torch.cuda.mem_get_info()[0] == free


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("scale", [0.0, -0.11, 1.7])
def test_attend_scales(m, new, scale):
    """Softmax scales of zero (every visible key counts alike), negative and large."""
    g = gen(20)
    bt = R.Batch([300, 77], [new, new], 32, DEV)
    c = make_cache(m, g, bt, 8, 2, 64, fill="normal")
    check(c, bt, randn(g, 2 * new, 8, 64, dtype=torch.bfloat16), scale=scale)


@pytest.mark.parametrize("new,hq,hkv", [(1, 8, 8), (1, 24, 1), (2, 24, 1), (3, 64, 4), (40, 40, 5)])
def test_attend_is_repeatable(m, new, hq, hkv):
    """Many splits, joined in their order whatever the order of arrival: the same bits every time."""
    g = gen(21)
    bt = R.Batch([20000, 4097], [new, new], 64, DEV)
    c = make_cache(m, g, bt, hq, hkv, 128, fill="normal")
    q = randn(g, 2 * new, hq, 128, dtype=torch.bfloat16)
    want = check(c, bt, q)
    for _ in range(20):
        assert torch.equal(c.attend(q, bt.b), want)


@pytest.mark.parametrize("new,hq,hkv", [(1, 16, 16), (5, 64, 8), (20, 64, 8)])
def test_attend_many_sequences(m, new, hq, hkv):
    """More row tiles than the workspace holds partial results for: every row tile ends in its own CTA."""
    g = gen(22)
    n = 1100 if new == 1 else 160
    bt = R.Batch([1 + 7 * i % 61 for i in range(n)], [new] * n, 16, DEV)
    c = make_cache(m, g, bt, hq, hkv, 64, fill="normal")
    check(c, bt, randn(g, bt.cu[-1], hq, 64, dtype=torch.bfloat16))


def test_decoder_step_example():
    """Token by token and as a prompt: the cache's blocks differ only in the scales they had on the way (codes
    rounded once more below 2^-6 of a scale), so the layers agree far inside e4m3's half step of 2^-4."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decoder_step.py")
    spec = importlib.util.spec_from_file_location("decoder_step", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    assert ex.main() < 2.0 ** -4
