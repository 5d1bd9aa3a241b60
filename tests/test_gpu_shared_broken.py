"""Attention over shared prefixes where one offset on the device breaks its bounds: what does not need that offset is
what it was."""
from __future__ import annotations

import random

import pytest
import torch

from test_gpu_shared import Case, bounds, m, ragged, t  # noqa: F401  (fixtures: both ways that the host's bounds choose)

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def case(mod, n_groups, new):
    r = random.Random(n_groups + new)
    sizes = [r.choice((1, 2, 4)) for _ in range(n_groups)]
    groups = [(r.choice((40, 128, 200, 333)), ragged(r, n, 50, new)) for n in sizes]
    return Case(mod, groups, 64, 1, 4, 16, seed=new, lone=(9, 30))


def check(mod, k, want, out, left_out, keep):
    """Rows of the sequences in `left_out` may hold anything (`keep`: hold what they held), all others are as before."""
    with pytest.raises(mod.MoeError, match="bounds"):
        k.c.device_status()
    of = torch.tensor([b for b, n in enumerate(k.bt.news) for _ in range(n)], device=DEV)  # rows' sequences
    free = torch.isin(of, torch.tensor(sorted(left_out), device=DEV))
    same = (out == want).flatten(1).all(1)
    assert (same | free).all(), f"sequences {of[~(same | free)].unique().tolist()}"
    if keep:
        assert (out[free] == 7).all()


@pytest.mark.parametrize("n_groups,new", [(3, 1), (5, 40), (32, 1), (33, 1), (40, 9), (1100, 1)])
def test_a_group_s_offset(m, n_groups, new):  # noqa: F811
    k = case(m, n_groups, new)
    want = k.c.attend(k.q, k.bt.b, prefix=k.share)
    assert k.c.device_status() == 0
    for i in sorted({0, 1, n_groups // 2, n_groups - 1, n_groups}):
        good = k.cu_seq[i]
        for bad in (-5, -2 ** 31, len(k.bt.lens) + 1, 2 ** 31 - 1):
            k.share.cu_seq[i] = bad
            out = torch.full_like(k.q, 7)
            k.c.attend(k.q, k.bt.b, out=out, prefix=k.share)
            first, last = k.cu_seq[max(i - 1, 0)], k.cu_seq[min(i + 1, n_groups)]
            check(m, k, want, out, range(first, last), False)
        k.share.cu_seq[i] = good
    assert torch.equal(k.c.attend(k.q, k.bt.b, prefix=k.share), want) and k.c.device_status() == 0


@pytest.mark.parametrize("n_groups,new", [(1, 1), (3, 1), (5, 40), (33, 1), (40, 9), (1100, 1)])
def test_a_sequence_s_offset(m, n_groups, new):  # noqa: F811
    """Within a group: at its ends it is the group's offset as well, whose rows are not valid then."""
    k = case(m, n_groups, new)
    n = len(k.bt.lens)
    want = k.c.attend(k.q, k.bt.b, prefix=k.share)
    ends = set(k.cu_seq)
    inner = [i for i in range(n + 1) if i not in ends]
    r = random.Random(n)
    for i in sorted({inner[0], inner[-1], *(r.choice(inner) for _ in range(4))}):
        good = k.bt.cu[i]
        for bad in (-5, -2 ** 31, k.bt.cu[-1] + 1, 2 ** 31 - 1):
            k.bt.b.cu_q[i] = bad
            out = torch.full_like(k.q, 7)
            k.c.attend(k.q, k.bt.b, out=out, prefix=k.share)
            check(m, k, want, out, {i - 1, i}, True)
        k.bt.b.cu_q[i] = good
    for i in sorted(ends - {0, n}):
        if i % 3 and n_groups > 5:
            continue
        good = k.bt.cu[i]
        g = [x for x in range(n_groups) if i in (k.cu_seq[x], k.cu_seq[x + 1])]
        k.bt.b.cu_q[i] = -1
        out = torch.full_like(k.q, 7)
        k.c.attend(k.q, k.bt.b, out=out, prefix=k.share)
        check(m, k, want, out, {i - 1, i, *range(k.cu_seq[min(g)], k.cu_seq[max(g) + 1])}, False)
        k.bt.b.cu_q[i] = good
    assert torch.equal(k.c.attend(k.q, k.bt.b, prefix=k.share), want) and k.c.device_status() == 0
