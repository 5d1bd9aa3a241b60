"""Attention of sequences that share prefixes, against 64 bits; and a step of forked sequences as it is used."""
from __future__ import annotations

import math
import random

import pytest
import torch

import attn_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
I32 = dict(dtype=torch.int32, device=DEV)
NAN = 0x7f


FAR = 1 << 17


@pytest.fixture(params=["near", "far"], autouse=True)
def bounds(request, monkeypatch):
    """The host's bounds as the lengths are, or far above them: short calls are one launch over all keys in the first
    case and launches over parts of them in the second."""
    monkeypatch.setattr(Case, "far", request.param == "far")


@pytest.fixture(scope="module")
def m():
    from int4_routed_expert_gb300 import build as b
    b.build()
    import int4_routed_expert_gb300 as mod
    mod.load()
    return mod


def t(x):
    return torch.tensor(x, **I32)


class Case:
    """Groups of sequences [(prefix length, [(tokens behind the prefix, new tokens), ...]), ...]; a length below 0 is
    that of a sequence which does not take part.  Sequences before the first group and behind the last one: `lone`."""

    far = False

    def __init__(self, m, groups, dim, hkv, hq, page, seed=0, lone=(), junk=True):
        self.m, self.page, self.dim, self.scale = m, page, dim, dim ** -0.5
        g = torch.Generator(DEV)
        g.manual_seed(seed)
        lens, news, self.prefix, cu = [], [], [], [len(lone)]
        for n in lone:
            lens.append(n), news.append(min(n, 2)), self.prefix.append(0)
        for p, seqs in groups:
            for more, new in seqs:
                lens.append(p + more if more >= 0 else -1 - more), news.append(new)
                self.prefix.append(p if lens[-1] - new >= p else 0)
            cu.append(len(lens))
        for n in lone:
            lens.append(n), news.append(1), self.prefix.append(0)
        self.bt = bt = R.Batch(lens, news, page, DEV, seed=seed, spare=sum(-(-p // page) for p, _ in groups) + 3)
        used = {x for row in bt.table for x in row}
        spare = [x for x in range(bt.n_pages) if x not in used]
        width = max([1] + [-(-p // page) for p, _ in groups])
        self.rows, at = [], 0
        for p, _ in groups:
            n = -(-p // page)
            self.rows.append(spare[at:at + n] + [-1] * (width - n))
            at += n
        shape = (bt.n_pages, hkv, page, dim)
        codes = [torch.randn(*shape, device=DEV, generator=g).to(R.F8).view(torch.uint8) for _ in range(2)]
        scales = [torch.exp2(torch.randint(-6, 3, shape[:2], device=DEV, generator=g).float()) for _ in range(2)]
        if junk:  # what no row may see: behind a prefix's end and before a sequence's own tokens
            table = [list(r) for r in bt.table]
            for c in codes:
                for (p, _), row in zip(groups, self.rows):
                    if p % page:
                        c[row[p // page], :, p % page:] = NAN
                for b, p in enumerate(self.prefix):
                    if p % page and lens[b] > p:
                        c[bt.table[b][p // page], :, :p % page] = NAN
            for b, p in enumerate(self.prefix):
                for i in range(p // page):
                    table[b][i] = (-1, bt.n_pages + 5, -2 ** 31)[i % 3]
            bt.b.page_table.copy_(t(table))
        most = max(max(lens), max(p for p, _ in groups), 1)
        if self.far:
            most = FAR
            bt.b = m.SeqBatch(bt.b.cu_q, bt.b.kv_len, bt.b.page_table, bt.cu[-1], max(max(news), 1), FAR)
        self.c = m.KVCache(*codes, *scales, n_q_heads=hq, max_seqs=len(lens), max_tokens=max(bt.cu[-1], 1),
                           max_kv_len=most)
        self.q = (1.5 * torch.randn(bt.cu[-1], hq, dim, device=DEV, generator=g)).bfloat16()
        tokens = [bt.cu[b] - bt.cu[a] for a, b in zip(cu, cu[1:])]
        self.cu_seq, self.lens = cu, [p for p, _ in groups]
        self.share = m.SharedPrefix(t(cu), t(self.lens), t(self.rows).view(len(groups), width), max(max(tokens), 1),
                                    FAR if self.far else max(max(self.lens), 1))

    def want(self, monkeypatch, causal=True):
        whole, bt = R.tokens, self.bt

        class Row:
            page = self.page

        def spliced(codes, scales, bt, b, length):
            x = whole(codes, scales, bt, b, length)
            p = self.prefix[b]
            if p:
                of = Row()
                of.table = [self.rows[max(g for g, s in enumerate(self.cu_seq[:-1]) if s <= b)]]
                x[:, :p] = whole(codes, scales, of, 0, p)
            return x

        with monkeypatch.context() as mp:
            mp.setattr(R, "tokens", spliced)
            return R.attend(self.q, self.c.k_codes, self.c.v_codes, self.c.k_scale, self.c.v_scale, bt, self.scale,
                            causal=causal)

    def check(self, monkeypatch, causal=True):
        lse = torch.empty(self.q.shape[:2], device=DEV)
        out = self.c.attend(self.q, self.bt.b, lse=lse, causal=causal, prefix=self.share)
        o, ref_lse, tol = self.want(monkeypatch, causal)
        err = (out.double() - o).abs()
        assert (err <= tol).all(), f"error {float((err / tol).max()):.3g} of its bound"
        fin = ref_lse.isfinite()
        assert torch.equal(fin, lse.isfinite()) and (lse[~fin] == -math.inf).all()
        # as a weight's sum: fp32 products of 2^-22 of the logits' magnitude a step, and the logarithm
        x = self.q.double().abs().amax() * self.c.k_scale.max().double() * 448 * self.dim * self.scale
        assert ((lse.double() - ref_lse)[fin].abs() <= 2.0 ** -16 * (1 + ref_lse[fin].abs()) + self.dim * 2.0 ** -22 * x).all()
        assert self.c.device_status() == 0
        again = self.c.attend(self.q, self.bt.b, causal=causal, prefix=self.share)
        assert torch.equal(out, again)
        return out


def ragged(r, n, most, new):
    return [(k := r.randint(1, new), (k + r.randint(0, most), k))[1] for _ in range(n)]


GROUPS = {
    "tokens": [(300, [(1, 1), (7, 1), (130, 1)])],
    "tile": [(256, [(1, 1), (128, 1), (129, 1), (2, 1)])],
    "short": [(5, [(1, 1), (40, 1)]), (1, [(1, 1), (1, 1)])],
    "verify": [(517, [(4, 4), (9, 4), (300, 4)]), (129, [(4, 4)] * 5)],
    "mixed": [(700, [(1, 1), (33, 17), (90, 90)]), (64, [(200, 130), (3, 2)])],
    "idle": [(300, [(-1, 1), (5, 1), (-1, 3), (0, 0)]), (90, [(-91, 1), (-31, 2), (4, 2)])],
    "none": [(0, [(50, 1), (200, 3)]), (40, [(1, 1)]), (0, [(-1, 0)])],
    "empty": [(64, []), (64, [(3, 1)]), (200, []), (30, [(2, 1), (1, 1)])],
}


@pytest.mark.parametrize("name", GROUPS)
@pytest.mark.parametrize("dim,hkv,hq,page", [(64, 1, 1, 16), (128, 2, 12, 64), (64, 2, 32, 32), (128, 1, 7, 128)])
def test_groups(m, monkeypatch, name, dim, hkv, hq, page):
    Case(m, GROUPS[name], dim, hkv, hq, page, seed=len(name)).check(monkeypatch)


def test_the_bounds_choose_the_launches(m):
    """One launch, which needs no workspace, and launches over parts of the keys."""
    k = Case(m, GROUPS["verify"], 64, 2, 8, 16)
    k.c.attend(k.q, k.bt.b, prefix=k.share)
    (size,) = k.c._shared.values()
    assert (size > 0) == Case.far


@pytest.mark.parametrize("name", ["tokens", "mixed", "idle"])
def test_without_the_causal_mask(m, monkeypatch, name):
    """All of a sequence's tokens, rows below position 0 included (which the reference has with a length of theirs)."""
    groups = [(p, [s for s in seqs if s != (-1, 1) and s != (-1, 3)]) for p, seqs in GROUPS[name]]
    Case(m, groups, 64, 2, 8, 16, seed=3).check(monkeypatch, causal=False)


@pytest.mark.parametrize("dim,hkv,hq,page,new", [(128, 4, 32, 64, 1), (64, 2, 16, 16, 1), (128, 2, 16, 32, 3),
                                                 (64, 1, 6, 128, 40), (128, 8, 8, 64, 1)])
def test_many(m, monkeypatch, dim, hkv, hq, page, new):
    """Rows of a group from one product's to several tiles', keys split over CTAs."""
    r = random.Random(dim + new)
    groups = [(5000, ragged(r, 40, 500, new)), (700, ragged(r, 3, 2000, new)), (3333, ragged(r, 21, 100, new))]
    Case(m, groups, dim, hkv, hq, page, seed=new, lone=(40, 1000)).check(monkeypatch)


def test_as_many_groups_as_sequences(m, monkeypatch):
    """The search for a sequence's group goes through several steps of 32."""
    r = random.Random(7)
    groups = [(r.randint(0, 40), ragged(r, r.randint(0, 2), 20, 1)) for _ in range(1300)]
    Case(m, groups, 64, 1, 2, 16, seed=1, lone=(3,)).check(monkeypatch)


@pytest.mark.parametrize("groups,dim,hq,new", [(33, 64, 8, 20), (32, 64, 8, 20), (40, 128, 6, 25), (5, 128, 8, 70)])
def test_groups_of_many_rows(m, monkeypatch, groups, dim, hq, new):
    """Row tiles of several groups, some of them empty or without a prefix, one CTA's work after the other's."""
    r = random.Random(groups)
    some = [(r.choice((0, 40, 128, 700, r.randint(1, 400))), ragged(r, r.choice((0, 1, 2, 3)), 50, new)) for _ in range(groups - 2)]
    Case(m, [(0, []), *some, (300, [(new, new)] * 9)], dim, 1, hq, 16, seed=2).check(monkeypatch)


def test_agrees_with_attention_of_each(m):
    """Tables that name the prefix's pages themselves: both calls see the same tokens."""
    r = random.Random(2)
    k = Case(m, [(640, ragged(r, 9, 100, 2)), (320, ragged(r, 4, 100, 2))], 128, 2, 8, 64, seed=5, junk=False)
    table = [list(x) for x in k.bt.table]
    for b, p in enumerate(k.prefix):
        g = max(g for g, s in enumerate(k.cu_seq[:-1]) if s <= b)
        table[b][:p // 64] = k.rows[g][:p // 64]
    k.bt.b.page_table.copy_(t(table))
    one, other = k.c.attend(k.q, k.bt.b, prefix=k.share).double(), k.c.attend(k.q, k.bt.b).double()
    # half a step of bf16 each, and the weights' half steps of f16
    spread = k.c.v_scale.max().double() * 448
    assert ((one - other).abs() <= 2.0 ** -7 * other.abs() + 2.0 ** -10 * spread).all()


def test_wild_scales(m, monkeypatch):
    """Values of the prefix and of the own tokens 2^40 apart, either way, and logits that leave one of them nothing."""
    for up in (40, -40):
        k = Case(m, [(300, [(70, 2), (5, 1), (130, 3)])], 64, 1, 4, 16, seed=9)
        mine = torch.tensor([x for x in k.rows[0] if x >= 0], device=DEV)
        k.c.v_scale[mine] *= 2.0 ** up
        k.check(monkeypatch)
        k.c.k_scale[mine] *= 64
        k.check(monkeypatch)


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_a_query_that_is_not_finite_stays_in_its_row(m, new, bad):
    k = Case(m, [(300, [(new, new), (new + 50, new), (new, new)])], 64, 2, 8, 16, seed=11)
    want = k.c.attend(k.q, k.bt.b, prefix=k.share)
    k.q[new, 3, 17] = bad
    out = k.c.attend(k.q, k.bt.b, prefix=k.share)
    assert out[new, 3].isnan().all()
    out[new, 3] = want[new, 3]
    assert torch.equal(out, want)


@pytest.mark.parametrize("dim,new", [(64, 1), (128, 1), (64, 9), (128, 30)])
def test_far_pages(m, monkeypatch, dim, new):
    """Pages whose codes lie beyond 2^31 bytes, of the prefix and of the sequences."""
    k = Case(m, [(200, [(new + 3, new), (new, new), (new + 140, new)])], dim, 8, 8, 128, seed=13, junk=False)
    far = (1 << 32) // (8 * 128 * dim) + 17  # pages behind 4 GB
    codes = [torch.zeros(far + k.bt.n_pages, 8, 128, dim, dtype=torch.uint8, device=DEV) for _ in range(2)]
    scales = [torch.ones(far + k.bt.n_pages, 8, device=DEV) for _ in range(2)]
    for big, small in zip(codes + scales, (k.c.k_codes, k.c.v_codes, k.c.k_scale, k.c.v_scale)):
        big[far:] = small
    want = k.c.attend(k.q, k.bt.b, prefix=k.share)
    c = m.KVCache(*codes, *scales, n_q_heads=8, max_seqs=3, max_tokens=k.bt.cu[-1], max_kv_len=FAR)
    for table in (k.bt.b.page_table, k.share.page_table):
        table += far
    assert torch.equal(c.attend(k.q, k.bt.b, prefix=k.share), want) and c.device_status() == 0


@pytest.mark.parametrize("new", [1, 40])
def test_strided_queries_and_given_results(m, new):
    k = Case(m, [(300, [(new, new), (new + 50, new)])], 64, 2, 8, 16, seed=4)
    want = k.c.attend(k.q, k.bt.b, prefix=k.share)
    wide = torch.zeros(k.q.shape[0], 12, 64, device=DEV).bfloat16()
    wide[:, 2:10] = k.q
    out = torch.full_like(k.q, 7)
    assert k.c.attend(wide[:, 2:10], k.bt.b, out=out, prefix=k.share) is out and torch.equal(out, want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = k.c.attend(k.q, k.bt.b, prefix=k.share, stream=s)
    s.synchronize()
    assert torch.equal(other, want)
    for x in torch.cuda.memory_snapshot():
        if x["address"] <= other.data_ptr() < x["address"] + x["total_size"]:
            assert x["stream"] == s.cuda_stream


def test_a_captured_call_follows_its_arrays(m, monkeypatch):
    """Two graphs of one cache, replayed in turn with other lengths and groups, have memory of their own."""
    a = Case(m, [(300, [(5, 1), (60, 1), (7, 1), (130, 1)])], 64, 2, 16, 16, seed=6, junk=False)
    outs, graphs = [torch.empty_like(a.q) for _ in range(2)], []
    a.c.attend(a.q, a.bt.b, prefix=a.share)
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            a.c.attend(a.q, a.bt.b, out=o, prefix=a.share)
        graphs.append(g)
    for lens, prefix in (([290, 300, 299, 301], 289), ([17, 300, 16, 301], 16), ([305, 360, 307, 430], 300)):
        a.bt.lens[:] = lens
        a.bt.b.kv_len.copy_(t(lens))
        a.share.prefix_len.fill_(prefix)
        a.prefix = [prefix if n - 1 >= prefix else 0 for n in lens]
        o, _, tol = a.want(monkeypatch)
        for out, g in zip(outs, graphs):
            g.replay()
            assert ((out.double() - o).abs() <= tol).all()
    assert a.c.device_status() == 0


@pytest.mark.parametrize("new", [1, 40])
def test_what_breaks_its_bounds_is_left_out(m, new):
    """Groups and lengths that break their bounds set the status bit; other groups' rows are what they were."""
    k = Case(m, [(300, [(new, new), (new + 5, new)]), (200, [(new, new), (new + 3, new)])], 64, 2, 8, 16, seed=8, junk=False)
    want = k.c.attend(k.q, k.bt.b, prefix=k.share)
    half = k.bt.cu[2]
    assert k.c.device_status() == 0
    for tensor, i, bad in ((k.share.prefix_len, 1, k.share.bounds[2] + 1), (k.share.prefix_len, 1, -1), (k.share.prefix_len, 1, 2 ** 31 - 1),
                           (k.share.cu_seq, 2, 5), (k.share.cu_seq, 2, 2 ** 31 - 1), (k.share.cu_seq, 2, 1),
                           (k.share.cu_seq, 2, -2 ** 31),
                           (k.share.page_table.view(-1), 19, k.bt.n_pages), (k.share.page_table.view(-1), 19, -1)):
        keep = tensor[i].item()
        tensor[i] = bad
        out = k.c.attend(k.q, k.bt.b, prefix=k.share)
        with pytest.raises(m.MoeError, match="bounds"):
            k.c.device_status()
        assert torch.equal(out[:half], want[:half])
        tensor[i] = keep
    for bad in (-3, 2 ** 31 - 1):  # the first group's begin: then no sequence before the second has one
        k.share.cu_seq[0] = bad
        k.c.attend(k.q, k.bt.b, prefix=k.share)
        with pytest.raises(m.MoeError, match="bounds"):
            k.c.device_status()
        k.share.cu_seq[0] = 0
    k.bt.b.cu_q[2] = half + 10 ** 6
    k.c.attend(k.q, k.bt.b, prefix=k.share)
    with pytest.raises(m.MoeError, match="bounds"):
        k.c.device_status()
    k.bt.b.cu_q[2] = half
    assert torch.equal(k.c.attend(k.q, k.bt.b, prefix=k.share), want) and k.c.device_status() == 0


@pytest.mark.parametrize("new", [1, 40])
def test_rows_that_no_sequence_covers_keep_what_they_held(m, new):
    k = Case(m, [(300, [(new, new), (new + 5, new), (new, new)])], 64, 2, 8, 16, seed=8, junk=False)
    want = k.c.attend(k.q, k.bt.b, prefix=k.share)
    k.bt.b.cu_q[3] = k.bt.cu[2]  # the last sequence has no tokens now
    out, lse = torch.full_like(k.q, 7), torch.full(k.q.shape[:2], 7.0, device=DEV)
    k.c.attend(k.q, k.bt.b, out=out, lse=lse, prefix=k.share)
    end = k.bt.cu[2]
    assert (out[end:] == 7).all() and (lse[end:] == 7).all() and torch.equal(out[:end], want[:end])
    assert k.c.device_status() == 0


def test_refusals(m):
    k = Case(m, [(300, [(5, 1), (60, 1)])], 64, 2, 8, 16, junk=False)
    assert torch.equal(k.c.attend(k.q, k.bt.b, prefix=k.share, window=10 ** 6), k.c.attend(k.q, k.bt.b, prefix=k.share))
    with pytest.raises(m.MoeError, match="window"):
        k.c.attend(k.q, k.bt.b, prefix=k.share, window=100)
    rows = k.share.page_table

    def prefix(cu=(0, 2), lens=(300,), table=rows, group=2, most=k.share.bounds[2]):
        return m.SharedPrefix(t(list(cu)), t(list(lens)), table, group, most)

    assert torch.equal(k.c.attend(k.q, k.bt.b, prefix=prefix(group=99)), k.c.attend(k.q, k.bt.b, prefix=k.share))
    for bad in (prefix(group=0), prefix(most=0), prefix(most=10 ** 6)):
        with pytest.raises(m.MoeError):
            k.c.attend(k.q, k.bt.b, prefix=bad)
    for args in ((t([0]), t([300]), rows, 2, 300), (t([0, 2]), t([300]).long(), rows, 2, 300), (t([0, 2]), t([300]), rows[0], 2, 300),
                 (t([0, 2]), t([300]).cpu(), rows, 2, 300), (t([0, 2]), t([300]), rows.expand(2, -1).contiguous(), 2, 300)):
        with pytest.raises(ValueError):
            m.SharedPrefix(*args)
    none = m.SharedPrefix(t([0]), t([]).view(0), rows[:0], 1, 1)
    assert torch.equal(k.c.attend(k.q, k.bt.b, prefix=none), k.c.attend(k.q, k.bt.b))
    assert k.c.device_status() == 0


# ------------------------------------------------------------------ as it is used

@pytest.mark.parametrize("dim,page,captured", [(64, 16, False), (128, 64, True)])
def test_a_step_of_forked_sequences(m, dim, page, captured):
    """A prompt, forked into answers that go on, branch, end and begin anew, through pool, cache and attention: each
    token's result is that of a cache of its own into which the sequence's tokens were written one by one alike."""
    hkv, hq, slots, steps, prompt = 2, 8, 6, 12, 5 * page + 11
    g = torch.Generator(DEV)
    g.manual_seed(dim)
    r = random.Random(dim)
    pages = slots * (prompt // page + 4)
    most = FAR if Case.far else prompt + 4 * page
    pool = m.PagePool.empty(pages, page, slots, prompt + 4 * page, device=DEV)
    cache = m.KVCache.empty(pages, page, hkv, dim, n_q_heads=hq, max_seqs=slots, max_tokens=prompt + 4 * page,
                            max_kv_len=most, device=DEV)

    def randn(n, h):
        return torch.randn(n, h, dim, device=DEV, generator=g).bfloat16()

    # the prompt, in slot 0
    cache.copy(pool.fork(t([-1] * slots), t([prompt] + [0] * (slots - 1))))
    k0, v0 = randn(prompt, hkv), randn(prompt, hkv)
    cache.write(k0, v0, pool.batch(prompt, prompt, prompt))
    # its whole pages are kept for all answers, whatever becomes of slot 0
    shared = prompt // page * page
    prefix_table = pool.table[:1, :shared // page].clone()
    pool.ref[prefix_table[0].long()] += 1
    share = m.SharedPrefix(t([0, slots]), t([shared]), prefix_table, slots, most if Case.far else shared)

    parent, added, keep = (torch.zeros(slots, **I32) for _ in range(3))
    q, k, v = randn(slots, hq), randn(slots, hkv), randn(slots, hkv)
    out = torch.zeros_like(q)
    batch = pool.batch(slots, 1, most)

    def step():
        moves = pool.fork(parent, added, keep=keep)
        cache.copy(moves)
        cache.write(k, v, batch)
        cache.attend(q, batch, out=out, prefix=share)

    graph = None
    tokens = [[(k0[i], v0[i]) for i in range(prompt)]] + [[] for _ in range(slots - 1)]
    for n in range(steps):
        p = [0] * slots if n == 0 else [r.choice((i, i, r.randrange(slots))) for i in range(slots)]
        kept = [len(tokens[x]) - (r.randrange(3) if n > 2 and len(tokens[x]) > prompt + 3 else 0) for x in p]
        if n == 7:  # a slot that ends, and one that begins anew from the kept prompt's tokens
            p[2], kept[2] = -1, 0
        news = [0 if x < 0 or (n == 4 and i == 3) else 1 for i, x in enumerate(p)]
        parent.copy_(t(p)), added.copy_(t(news)), keep.copy_(t(kept))
        for x in (q, k, v):
            x.copy_(randn(slots, x.shape[1]))
        if captured and n == 3:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        graph.replay() if graph else step()
        assert pool.device_status() == 0 and cache.device_status() == 0
        tokens = [list(tokens[x][:c]) if x >= 0 else [] for x, c in zip(p, kept)]
        row = 0
        for i in range(slots):
            if news[i]:
                tokens[i].append((k[row].clone(), v[row].clone()))
                row += 1
        assert pool.kv_len.tolist() == [len(x) for x in tokens] and pool.cu_q[-1].item() == row
        # slot 0's tokens, whatever pages they came by: off by half a step of e4m3 or, where values are small, of its
        # subnormals, 2^-10 of a scale; a scale is below 2^1 / 448 of the largest value that its page has held
        n0 = len(tokens[0])
        whole = m.SeqBatch(t([0, n0]), pool.kv_len[:1].contiguous(), pool.table[:1].contiguous(), n0, n0, n0)
        for got, j in zip(cache.read(whole, dtype=torch.float32), (0, 1)):
            want = torch.stack([x[j] for x in tokens[0]]).double()
            assert ((got.double() - want).abs() <= 2.0 ** -4 * want.abs() + 2.0 ** -9 * 8 / 448).all()
        # attention over what the cache holds, sequence by sequence in 64 bits
        row = 0
        for i in range(slots):
            if not news[i]:
                continue
            L = len(tokens[i])
            at = pool.table[i, :-(-L // page)].long()
            kk, vv = ((c.view(R.F8)[at].double() * s[at].double()[..., None, None]).transpose(0, 1).flatten(1, 2)[:, :L]
                      for c, s in ((cache.k_codes, cache.k_scale), (cache.v_codes, cache.v_scale)))
            x = q[row].double().view(hkv, hq // hkv, dim)
            w = torch.softmax(x @ kk.transpose(1, 2) * dim ** -0.5, -1)
            want = (w @ vv).view(hq, dim)
            spread = (w @ vv.abs()).view(hq, dim)
            # half a step of bf16; half a step of f16 on a weight (2^-11) and what its logit is off: 2 D 2^-22 times
            # a sum of magnitudes below 16
            assert ((out[row].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -9 * spread + 1e-6).all()
            row += 1
