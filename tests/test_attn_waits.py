"""The attention kernels' tensor memory accesses and bounded waits, read from their sources.  Neither a missing wait
nor a wait that gives up shows in a result on the GPU, so the order is checked where it is written."""
from __future__ import annotations

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "int4_routed_expert_gb300", "csrc")
KERNELS = ("attn_tiles.cu", "attn_few.cu")


def code(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


def columns(expr, width, x, text):
    """(base, columns) of an address `base + a whole number`, the columns None where it is not one; `x` is the
    half of the keys, k... a constant of the source."""
    base, _, rest = expr.partition("+")
    known = {n: int(v) for n, v in re.findall(r"constexpr int (k\w+) = (\d+);", text)}
    try:
        at = int(eval(rest or "0", {"__builtins__": {}}, {**known, "x": x}))
    except NameError:
        return base.strip(), None
    return base.strip(), set(range(at, at + width))


@pytest.mark.parametrize("name", KERNELS)
def test_stores_keep_off_columns_whose_load_is_under_way(name):
    """tcgen05.ld and tcgen05.st are asynchronous, and only a wait::ld puts a later store behind a load: between
    a load and its wait, stores go to other columns."""
    text = code(name)
    calls = re.finditer(r"tmem_(ld32|ld16f|ld16|st16|wait_ld)\w*\(([^,;]*)[,)]", text)
    under_way, stores = [], 0
    for c in calls:
        what, arg = c.group(1), c.group(2)
        if what.startswith("ld"):
            under_way.append((arg, 32 if what == "ld32" else 16))
        elif what == "wait_ld":
            under_way.clear()
        else:
            stores += 1
            for load, width in under_way:
                for x in (0, 1):
                    a, mine = columns(arg, 16, x, text)
                    b, theirs = columns(load, width, x, text)
                    assert a != b or (mine is not None and theirs is not None and not mine & theirs), \
                        f"{name}: store to [{arg}] (x = {x}) while [{load}] is being read"
    assert stores >= 1


def test_products_read_the_weights_where_they_are_stored():
    text = code("attn_tiles.cu")
    assert re.search(r"tmem_st16\(ts \+ kPAt \+ 16 \* x, u\)", text)
    assert re.search(r"pt = tmem \+ i \* 128 \+ kPAt\b", text)
    # the second 64 keys' weights: as far on as their thread's columns
    assert re.search(r"ts = tmem \+ i \* 128 \+ lanes \+ half \* 64\b", text) and "mma_o(ot, pt + 64," in text


@pytest.mark.parametrize("name", KERNELS)
def test_a_lane_that_gave_up_does_not_part_from_its_warp(name):
    """A bounded wait can give up in one lane and succeed in its neighbour.  Where the outcome decides whether a
    warp goes on to something that all its lanes have to reach, the warp has agreed on it before: else the lanes
    that go on wait for the others without limit."""
    text = code(name)
    softmax = text[text.index("float* red =" if name == "attn_few.cu" else "const RowSees sees ="):]
    collective = r"tmem_ld|tmem_st|__\w+_sync\(|named_sync|break;"
    found = 0
    for c in re.finditer(r"\bif \(", softmax):
        end, depth = c.end(), 1
        while depth:
            depth += {"(": 1, ")": -1}.get(softmax[end], 0)
            end += 1
        condition, rest = softmax[c.end():end - 1], softmax[end:].lstrip()
        body = rest[:rest.index("}" if rest[0] == "{" else ";") + 1]
        if not re.search(r"\bok\b", condition) or not re.search(collective, body):
            continue
        found += 1
        last = re.findall(r"\bok = ([^;]*);", softmax[:c.start()])[-1]
        agreed = condition + last  # (a vote in the condition is an agreement itself)
        assert "__all_sync(" in agreed or "named_vote(" in agreed, f"{name}: [if ({condition})] after [ok = {last}]"
    assert found >= 3
