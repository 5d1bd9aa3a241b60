"""The page pool where one slot alone has what breaks its bounds, and where the caller made the state."""
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


@pytest.mark.parametrize("slots,width", [(3, 7), (40, 600), (900, 40)])
@pytest.mark.parametrize("cut", [0, 1])
def test_a_bad_entry_of_a_slot_that_goes_on(m, slots, width, cut):
    """Kept page ids outside of the pool are refused in a slot that goes on too, wherever they stand; what the call drops
    may be anything."""
    page, r = 16, random.Random(slots)
    pages = slots * width
    pool = m.PagePool.empty(pages, page, slots, width * page, device=DEV)
    ref = P.Pool([[] for _ in range(slots)], [0] * slots, [0] * pages, page, width)
    lens = [page * r.randint(2, width - 1) for _ in range(slots)]
    lens[-1] = page * (width - 1)

    def fork(parent, added, keep):
        want, moves, cu = ref.fork(parent, added, keep)
        got = pool.fork(t(parent), t(added), keep=t(keep))
        assert got.tolist() == [list(x) for x in moves] and pool.cu_q.tolist() == cu and want == 0
        assert torch.equal(pool.table, t(ref.table()).view(slots, width)) and pool.ref.tolist() == ref.ref
        assert pool.kv_len.tolist() == ref.lens and pool.device_status() == 0

    fork([-1] * slots, lens, [0] * slots)
    go_on, added = list(range(slots)), [r.randint(0, 1) for _ in range(slots)]
    keep = [n - cut * page for n in lens]  # whole pages: no slot writes into one that it keeps
    for slot in (0, slots - 1):
        kept = lens[slot] // page - cut
        for at in sorted({0, kept // 2, kept - 1} & set(range(kept))):
            good = pool.table[slot, at].item()
            for bad in (pages, -1, -2 ** 31, 2 ** 31 - 1):
                pool.table[slot, at] = bad
                before = [x.clone() for x in (pool.table, pool.kv_len, pool.ref, pool.free)]
                moves = pool.fork(t(go_on), t(added), keep=t(keep))
                assert (moves == -1).all() and (pool.cu_q == 0).all()
                assert all(torch.equal(x, y) for x, y in zip(before, (pool.table, pool.kv_len, pool.ref, pool.free)))
                with pytest.raises(m.MoeError, match="bounds"):
                    pool.device_status()
            pool.table[slot, at] = good
    fork(go_on, added, keep)


@pytest.mark.parametrize("uses", [[0], [3], [0, 1, 0, -1, 2, 0], [1, 0] * 3000])
def test_free_pages_of_a_pool_that_no_call_has_changed(m, uses):
    """The count is right before the first call, and stays when that one is refused."""
    pool = m.PagePool(t([[-1, -1], [-1, -1]]), t([0, 0]), t(uses), 16)
    free = uses.count(0)
    assert pool.free.shape == (1,) and pool.free.dtype == torch.int32 and pool.free.item() == free
    pool.fork(t([-1, 2]), t([1, 0]))
    with pytest.raises(m.MoeError, match="bounds"):
        pool.device_status()
    assert pool.free.item() == free
    if free:
        pool.fork(t([-1, -1]), t([1, 0]))
        assert pool.free.item() == free - 1 and pool.device_status() == 0
    pool = m.PagePool.empty(len(uses), 16, 3, 100, device=DEV)
    assert pool.free.item() == len(uses) and pool.table.shape == (3, 7)
    parent, added, side = t([-1, -1, -1]), t([1, 0, 0]), torch.cuda.Stream()
    pool = m.PagePool.empty(len(uses), 16, 3, 100, device=DEV)
    pool.fork(parent, added, stream=side)  # on another stream, straight behind
    torch.cuda.synchronize()
    assert pool.free.item() == len(uses) - 1


def test_copy_of_the_longest_list(m):
    """2^31 - 1 moves (26 GB), most of which are none: the first, some in between and the last are made."""
    n = 2 ** 31 - 1
    codes = [torch.randint(0, 256, (16, 2, 16, 64), device=DEV, dtype=torch.uint8) for _ in range(2)]
    scales = [torch.rand(16, 2, device=DEV) for _ in range(2)]
    c = m.KVCache(*codes, *scales, n_q_heads=2, max_seqs=1, max_tokens=1, max_kv_len=1)
    want = [x.clone() for x in codes + scales]
    moves = torch.full((n, 3), -1, **I32)
    for i, (at, tokens) in enumerate(((0, 16), (38911, 16), (38912, 3), (2 ** 30 + 5, 16), (n - 38913, 16), (n - 2, 16), (n - 1, 9))):
        moves[at] = t([i, 15 - i, tokens])
        for x in want[:2]:
            x[15 - i, :, :tokens] = x[i, :, :tokens]
        for x in want[2:]:
            x[15 - i] = x[i]
    c.copy(moves)
    assert c.device_status() == 0
    assert all(torch.equal(x, y) for x, y in zip(want, codes + scales))
    del moves
    torch.cuda.empty_cache()
