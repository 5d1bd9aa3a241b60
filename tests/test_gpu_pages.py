"""The page pool and the copying of pages against their definitions (whole numbers and bytes: equal)."""
from __future__ import annotations

import random

import pytest
import torch

import pages_ref as P

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
I32 = dict(dtype=torch.int32, device=DEV)


@pytest.fixture(scope="module")
def m():
    from int4_routed_expert_gb300 import build as b
    b.build()
    import int4_routed_expert_gb300 as mod
    mod.load()
    return mod


def t(x):
    return torch.tensor(x, **I32)


def same(pool, ref):
    assert torch.equal(pool.table, t(ref.table()).view(pool.table.shape))
    assert pool.kv_len.tolist() == ref.lens and pool.ref.tolist() == ref.ref


def empty(m, pages, page, slots, width):
    pool = m.PagePool.empty(pages, page, slots, width * page, device=DEV)
    return pool, P.Pool([[] for _ in range(slots)], [0] * slots, [0] * pages, page, width)


def fork(m, pool, ref, parent, added, keep=None):
    """Both; returns the status bits."""
    free = pool.free.item()
    want, moves, cu = ref.fork(parent, added, keep)
    got = pool.fork(t(parent), t(added), keep=None if keep is None else t(keep))
    assert got.tolist() == [list(x) for x in moves]
    assert pool.cu_q.tolist() == cu
    same(pool, ref)
    assert pool.free.item() == (free if want else sum(u == 0 for u in ref.ref))
    if want:
        with pytest.raises(m.MoeError, match="free pages" if want == 8 else "bounds"):
            pool.device_status()
    assert pool.device_status() == 0
    return want


@pytest.mark.parametrize("pages,page,slots,width,steps", [
    (40, 16, 1, 30, 25), (60, 16, 5, 12, 60), (300, 32, 33, 17, 40), (2000, 64, 40, 61, 30), (9001, 16, 700, 41, 12),
    (40000, 128, 2000, 15, 8), (12000, 16, 9000, 3, 6), (30000, 16, 20000, 2, 5), (150001, 16, 40, 9000, 7), (300000, 64, 300, 2500, 7),
    (524288, 16, 20, 30000, 5), (524289, 16, 20, 30000, 5)])
def test_fork_steps(m, pages, page, slots, width, steps):
    """Random steps: sequences go on, are cut back, forked at different points, ended, begun; some steps are refused."""
    r = random.Random(slots)
    pool, ref = empty(m, pages, page, slots, width)
    seen = set()
    for step in range(steps):
        parent = [r.choice((i, i, i, r.randrange(slots), r.randrange(min(slots, 3)), -1)) for i in range(slots)]
        most = 2 * pages // slots * page if step % 3 == 0 else page // 2 + 1
        added = [r.choice((0, 1, r.randint(0, most))) for _ in range(slots)]
        keep = None
        if step % 2:
            keep = [r.choice((-1, 0, ref.lens[max(p, 0)], ref.lens[max(p, 0)] - r.randint(0, 5), r.randint(0, width * page),
                              2 ** 31 - 1)) for p in parent]
            if step % 4 == 1:  # lengths and points that end with a page
                keep = [max(k, 0) // page * page if k < 2 ** 31 - 1 else k for k in keep]
        kept = [0 if p < 0 else ref.lens[p] if keep is None else min(max(k, 0), ref.lens[p])
                for p, k in zip(parent, keep or parent)]
        if step % 5:  # (else too long for the table now and then)
            added = [min(a, width * page - k) for a, k in zip(added, kept)]
        seen.add(fork(m, pool, ref, parent, added, keep))
    assert 0 in seen


def test_fork_of_one_page_by_all(m):
    """Who copies a page that is not full: all writers but the lowest, all where another keeps it, none alone."""
    pool, ref = empty(m, 64, 16, 6, 4)
    assert fork(m, pool, ref, [-1] * 6, [21, 0, 0, 0, 0, 0]) == 0
    assert fork(m, pool, ref, [0] * 6, [1] * 6) == 0  # slot 0 stays, five copies
    assert (pool.ref[pool.table[:, 0].long()] == 6).all() and pool.free.item() == 64 - 7
    assert fork(m, pool, ref, [3] * 6, [1, 0, 1, 1, 0, 2]) == 0  # two do not write: four copies
    assert fork(m, pool, ref, list(range(6)), [0, 1, 0, 0, 1, 0]) == 0  # now they do
    assert fork(m, pool, ref, [2, 2, 2, 2, 2, 2], [1] * 6, [22, 20, 18, 17, 16, 3]) == 0  # at different points
    assert fork(m, pool, ref, [5, 4, 3, 2, 1, 0], [0] * 6) == 0  # a permutation: nothing to copy
    assert fork(m, pool, ref, [-1] * 6, [0] * 6) == 0
    assert pool.free.item() == 64 and (pool.table == -1).all()


@pytest.mark.parametrize("slots,width", [(5, 6), (2000, 40)])
def test_keep_may_be_the_lengths_themselves(m, slots, width):
    """keep=pool.kv_len (a slot keeps at most as many tokens as it had): the lengths are read before they change."""
    r = random.Random(slots)
    pool, ref = empty(m, slots * width, 16, slots, width)
    assert fork(m, pool, ref, [-1] * slots, [r.randint(0, 40) for _ in range(slots)]) == 0
    for _ in range(3):
        parent, added = [r.randrange(slots) for _ in range(slots)], [r.randint(0, 3) for _ in range(slots)]
        assert ref.fork(parent, added, list(ref.lens))[0] == 0
        pool.fork(t(parent), t(added), keep=pool.kv_len)
        same(pool, ref)
    assert pool.device_status() == 0


def test_a_captured_fork_follows_its_arrays(m):
    pool, ref = empty(m, 3000, 16, 300, 40)
    parent, added, keep = (torch.zeros(300, **I32) for _ in range(3))
    parent.fill_(-1)
    pool.fork(parent, added, keep=keep)
    assert ref.fork([-1] * 300, [0] * 300)[0] == 0
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moves = pool.fork(parent, added, keep=keep)
        compacted = pool.compact()
    r = random.Random(1)
    for step in range(12):
        p = [r.choice((i, r.randrange(300), -1)) if step else -1 for i in range(300)]
        a = [r.randint(0, 60 if step % 4 == 0 else 2) for _ in range(300)]
        if step == 7:
            a[200] = -1  # refused: the graph's compaction runs all the same
        k = [r.randint(0, 640 - x) for x in a]
        parent.copy_(t(p)), added.copy_(t(a)), keep.copy_(t(k))
        g.replay()
        want, wanted, cu = ref.fork(p, a, k)
        assert (want == 0) == (step != 7)
        assert moves.tolist() == [list(x) for x in wanted] and pool.cu_q.tolist() == cu
        assert compacted.tolist() == [list(x) for x in ref.compact()]
        same(pool, ref)
        if want:
            with pytest.raises(m.MoeError):
                pool.device_status()
    assert pool.device_status() == 0


def test_kept_pages(m):
    """A page that the caller counts once more stays when its sequence ends, and is copied by its only writer."""
    pool, ref = empty(m, 32, 16, 2, 4)
    assert fork(m, pool, ref, [-1, -1], [20, 0]) == 0
    held = pool.table[0, :2].tolist()
    for x in held:
        pool.ref[x] += 1
        ref.ref[x] += 1
    assert fork(m, pool, ref, [0, -1], [1, 0]) == 0 and ref.rows[0][1] != held[1]
    assert fork(m, pool, ref, [-1, -1], [0, 33]) == 0
    assert all(ref.ref[x] == 1 for x in held) and not set(held) & set(ref.rows[1])


@pytest.mark.parametrize("slots", [6, 3000])
def test_fork_refuses_on_the_device(m, slots):
    """What breaks its bounds, whatever it is, changes nothing and reads nothing outside; the rest of a step has no
    tokens then."""
    pool, ref = empty(m, 8 * slots, 16, slots, 8)
    go_on, none = list(range(slots)), [0] * slots
    assert fork(m, pool, ref, [-1] * slots, [20] * slots) == 0

    def but(x, i, v):
        x = list(x)
        x[i] = v
        return x

    for i in (0, slots - 1):
        for parent, added in ((but(go_on, i, slots), none), (but(go_on, i, -2), none), (but(go_on, i, 2 ** 31 - 1), none),
                              (but(go_on, i, -2 ** 31), none), (go_on, but(none, i, -1)), (go_on, but(none, i, -2 ** 31)),
                              (go_on, but(none, i, 2 ** 31 - 1)), (go_on, but(none, i, 8 * 16 - 19))):
            assert fork(m, pool, ref, parent, added) == 2
    assert fork(m, pool, ref, go_on, [100] * slots) == 0 and pool.free.item() == 0  # 8 pages each: all of them
    tight, tight_ref = empty(m, 8 * slots - 1, 16, slots, 8)
    assert fork(m, tight, tight_ref, [-1] * slots, [20] * slots) == 0
    assert fork(m, tight, tight_ref, go_on, [100] * slots) == 8
    assert fork(m, tight, tight_ref, but(go_on, 1, -1), [100] * slots) == 0  # (slot 1 has 7 pages)
    # state that no fork makes
    for tensor, i, bad in ((pool.kv_len, 1, -5), (pool.kv_len, 1, 8 * 16 + 1), (pool.kv_len, 1, 2 ** 31 - 1),
                           (pool.table.view(-1), 8, 8 * slots), (pool.table.view(-1), 8, -7), (pool.table.view(-1), 15, 2 ** 31 - 1)):
        keep = tensor[i].item()
        tensor[i] = bad
        before = pool.table.clone(), pool.kv_len.clone(), pool.ref.clone()
        moves = pool.fork(t([1] * slots), t([1] * slots))
        assert (moves == -1).all() and (pool.cu_q == 0).all()
        assert all(torch.equal(x, y) for x, y in zip(before, (pool.table, pool.kv_len, pool.ref)))
        with pytest.raises(m.MoeError, match="bounds"):
            pool.device_status()
        tensor[i] = keep
    assert fork(m, pool, ref, [1] * slots, [1] * slots) == 0


@pytest.mark.parametrize("pages,page,slots,width,used", [(1, 16, 1, 1, 1), (2, 16, 1, 2, 1), (33, 32, 3, 10, 20), (1000, 16, 7, 80, 300),
                                                         (8200, 64, 5, 900, 4000), (50001, 16, 300, 200, 30000),
                                                         (300000, 16, 40, 6000, 100000), (700001, 16, 40, 6000, 150000)])
def test_compact(m, pages, page, slots, width, used):
    r = random.Random(pages)
    for fill in ("anywhere", "behind", "before", "none"):
        ids = {"anywhere": r.sample(range(pages), used), "behind": list(range(pages - used, pages)),
               "before": list(range(used)), "none": []}[fill]
        r.shuffle(ids)
        rows, uses = [], [0] * pages
        for i in range(slots):
            n = min(len(ids), r.randint(0, min(width, 2 * used // slots + 1)))
            rows.append(ids[:n])
            ids = ids[n // 2:]  # half of them are the next one's too
            for x in rows[-1]:
                uses[x] += 1
        for x in ids[:3]:
            uses[x] += 1  # kept, and in no table
        lens = [max(0, len(x) * page - r.randrange(page)) for x in rows]
        ref = P.Pool(rows, lens, uses, page, width)
        pool = m.PagePool(t(ref.table()).view(slots, width), t(lens), t(uses), page)
        for _ in range(2):  # a second time nothing moves
            moves = ref.compact()
            got = pool.compact()
            assert torch.equal(got, t(moves).view(-1, 3))
            same(pool, ref)
            assert pool.free.item() == sum(u == 0 for u in ref.ref) and pool.device_status() == 0


@pytest.mark.parametrize("bad", [4000, -1, 2 ** 31 - 1, 399])
def test_compact_leaves_bad_entries(m, bad):
    """Entries outside of the pool, and of pages that are free."""
    uses = [0] * 400
    for x in (5, 300, 301):
        uses[x] = 1
    pool = m.PagePool(t([[5, bad, 300], [301, -1, -1]]), t([40, 10]), t(uses), 16)
    pool.compact()
    assert pool.table.tolist() == [[0, bad, 1], [2, -1, -1]] and pool.ref.tolist()[:4] == [1, 1, 1, 0]
    with pytest.raises(m.MoeError, match="bounds"):
        pool.device_status()


def cache(m, pages, heads, page, dim, seed=0):
    g = torch.Generator(DEV)
    g.manual_seed(seed)
    codes = [torch.randint(0, 256, (pages, heads, page, dim), device=DEV, generator=g, dtype=torch.uint8) for _ in range(2)]
    scales = [torch.rand(pages, heads, device=DEV, generator=g) for _ in range(2)]
    return m.KVCache(*codes, *scales, n_q_heads=heads, max_seqs=4, max_tokens=64, max_kv_len=64)


@pytest.mark.parametrize("heads,page,dim", [(1, 16, 64), (3, 16, 64), (8, 64, 128), (5, 128, 64), (2, 32, 128), (256, 16, 64)])
@pytest.mark.parametrize("n", [1, 7, 900])
def test_copy(m, heads, page, dim, n):
    """Codes (NaN ones too) and scales bit for bit; tokens from none to all; moves that are none in between."""
    r = random.Random(n)
    pages = 2 * n + 5
    c = cache(m, pages, heads, page, dim)
    ids = r.sample(range(pages), 2 * n)
    moves = [(a, b, r.choice((page, 0, 1, page - 1, r.randint(0, page)))) for a, b in zip(ids[:n], ids[n:])]
    want = [x.clone() for x in (c.k_codes, c.v_codes, c.k_scale, c.v_scale)]
    for a, b, k in moves:
        for x in want[:2]:
            x[b, :, :k] = x[a, :, :k]
        for x in want[2:]:
            x[b] = x[a]
    spread = []
    for x in moves:
        spread += [x] + [(-1, r.randrange(-3, pages), r.randrange(page))] * r.choice((0, 0, 1, 40))
    c.copy(t(spread))
    assert all(torch.equal(x, y) for x, y in zip(want, (c.k_codes, c.v_codes, c.k_scale, c.v_scale)))
    c.copy(t(spread)[:0])
    c.copy(t([(-1, -1, -1)] * 1000))
    c.copy(t([(ids[0], ids[0], page)]))  # onto itself
    assert all(torch.equal(x, y) for x, y in zip(want, (c.k_codes, c.v_codes, c.k_scale, c.v_scale)))
    assert c.device_status() == 0


def test_copy_far_pages(m):
    """Offsets beyond 2^31 bytes, either way."""
    pages, page = 40001, 128
    codes = [torch.empty(pages, 8, page, 128, dtype=torch.uint8, device=DEV) for _ in range(2)]  # 5 GB each
    scales = [torch.empty(pages, 8, device=DEV) for _ in range(2)]
    c = m.KVCache(*codes, *scales, n_q_heads=8, max_seqs=1, max_tokens=1, max_kv_len=1)
    ends = [0, 1, 16384, pages - 2, pages - 1]
    for x in codes + scales:
        for i in ends:
            x[i] = torch.randint(0, 256, x.shape[1:], device=DEV).to(x.dtype)
    want = [[x[i].clone() for i in ends] for x in codes + scales]
    c.copy(t([(pages - 1, 1, page), (0, pages - 2, page), (16384, 20000, 5)]))
    for x, (a, _, mid, _, z) in zip(codes + scales, want):
        assert torch.equal(x[1], z) and torch.equal(x[pages - 2], a) and torch.equal(x[pages - 1], z) and torch.equal(x[0], a)
        part = slice(None) if x.dim() == 2 else (slice(None), slice(0, 5))
        assert torch.equal(x[20000][part], mid[part])
    assert c.device_status() == 0


@pytest.mark.parametrize("bad", [(20, 1, 16), (2, 20, 16), (2, -1, 16), (2, 2 ** 31 - 1, 1), (2 ** 31 - 1, 1, 1), (2, 3, 17), (2, 3, -1)])
def test_copy_leaves_bad_moves_out(m, bad):
    c = cache(m, 20, 2, 16, 64)
    want = [x.clone() for x in (c.k_codes, c.v_codes, c.k_scale, c.v_scale)]
    for x in want:
        x[9] = x[4]
    c.copy(t([bad, (4, 9, 16)]))
    assert all(torch.equal(x, y) for x, y in zip(want, (c.k_codes, c.v_codes, c.k_scale, c.v_scale)))
    with pytest.raises(m.MoeError, match="bounds"):
        c.device_status()


def test_binding_refuses(m):
    pool, _ = empty(m, 20, 16, 4, 3)
    ok = t([0, 1, 2, 3])
    for bad in (ok[:3], ok.long(), torch.zeros(8, **I32)[::2], ok.cpu(), ok.view(2, 2)):
        for call in (lambda: pool.fork(bad, ok), lambda: pool.fork(ok, bad), lambda: pool.fork(ok, ok, keep=bad)):
            with pytest.raises(ValueError):
                call()
    c = cache(m, 20, 2, 16, 64)
    for bad in (torch.zeros(3, 3, dtype=torch.int64, device=DEV), torch.zeros(3, 4, **I32), torch.zeros(9, **I32),
                torch.zeros(3, 6, **I32)[:, ::2], torch.zeros(3, 3, dtype=torch.int32)):
        with pytest.raises(ValueError):
            c.copy(bad)
    for args in ((t([[0]]), t([0, 0]), t([0]), 16), (t([0]), t([0]), t([0]), 16), (t([[0]]).long(), t([0]), t([0]), 16),
                 (t([[0]]).cpu(), t([0]), t([0]), 16)):
        with pytest.raises(ValueError):
            m.PagePool(*args)
    with pytest.raises(m.MoeError):
        m.PagePool(t([[0]]), t([0]), t([0]), 24)
