"""What the plans of attention over shared prefixes promise, for sizes that no test runs (CPU: host code alone)."""
from __future__ import annotations

import ctypes as C
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
KEYS, ROWS = 128, 256  # of a tile of keys, of a row tile of dealt out work


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    from int4_routed_expert_gb300 import build as b
    out = tmp_path_factory.mktemp("plan") / "libshared_plan.so"
    subprocess.run([b._nvcc(), *b.ARCH, "-std=c++17", "-shared", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr", "-I", b.INC,
                    os.path.join(ROOT, "tests", "shared_plan.cu"), "-o", str(out)], check=True)
    lib = C.CDLL(str(out))
    lib.shared_plan.restype = C.c_ulonglong

    def of(seqs, tokens, max_q, max_kv, kv_heads, dim, g, groups, group_tokens, prefix, n_sm=152):
        p = (C.c_int * 6)()
        sizes = (seqs, tokens, max_q, max_kv, kv_heads, dim, g, groups, group_tokens, prefix)
        size = lib.shared_plan((C.c_int * 10)(*sizes), n_sm, p)
        return dict(zip(("one", "ctas", "row_tiles", "splits", "parts", "own_splits"), p)), size

    return of


def test_dealt_out_units_fit_32_bits_whatever_the_arrays_hold(plan):
    """The device numbers (row tile, kv head, tile of keys) in 32 bits. Offsets that do not ascend make groups of the same
    sequences, each within its bounds: all of max_group_tokens rows and max_prefix_len keys, in every one of the groups."""
    r, dealt = random.Random(1), 0
    sizes = [(32, 1 << 18, 1 << 18, 131072, 8, 128, 8, 32, 1 << 18, 131072),
             (64, 1 << 20, 1 << 20, 1 << 20, 8, 128, 8, 31, 1 << 20, 1 << 20)]
    for _ in range(3000):
        kv_heads, g = r.choice((1, 2, 4, 8, 64)), r.choice((1, 2, 4, 8, 12))
        tokens = int(2 ** r.uniform(8, 24))
        if tokens * kv_heads * g > 2 ** 31 - 1:
            continue
        kv = int(2 ** r.uniform(7, 30))
        sizes.append((r.randint(1, 64), tokens, r.randint(1, tokens), kv, kv_heads, r.choice((64, 128)), g, r.randint(1, 32),
                      r.randint(1, tokens), r.randint(max(1, kv // 2), kv)))
    for s in sizes:
        p, _ = plan(*s)
        if p["ctas"] and not p["one"]:
            dealt += 1
            kv_heads, g, groups, tokens, prefix = s[4], s[6], s[7], s[8], s[9]
            units = groups * -(-tokens * g // ROWS) * kv_heads * -(-prefix // KEYS)
            assert units + max(units // p["ctas"] + 1, -(-prefix // KEYS)) < 2 ** 31, (s, p)
    assert dealt > 300


def test_the_workspace_stays_below_what_the_header_says(plan):
    r, most = random.Random(2), 0.0
    sizes = [(64, 64, 1, 17884, 8, 128, 8, 1, 64, 16384), (4, 16384, 4096, 34096, 8, 128, 8, 1, 16384, 30000),
             (42, 218, 7, 3485842, 256, 128, 16, 1, 87, 2644173)]
    for _ in range(3000):
        kv_heads, g = r.choice((1, 2, 4, 8, 64, 256)), r.choice((1, 2, 4, 8, 12, 16))
        tokens = int(2 ** r.uniform(0, 24))
        if tokens * kv_heads * g > 2 ** 31 - 1:
            continue
        kv, seqs = int(2 ** r.uniform(0, 30)), r.randint(1, min(r.choice((64, 65535)), tokens))
        sizes.append((seqs, tokens, r.choice((1, tokens, r.randint(1, tokens))), kv, kv_heads, r.choice((64, 128)), g,
                      r.choice((1, 1, 2, 5, 32, 33, seqs)), r.randint(1, tokens), r.randint(1, kv)))
    for s in sizes:
        p, size = plan(*s)
        bound = max(4 * s[1] * s[4] * s[6], 1 << 21) * (4 * s[5] + 8) + 1024
        assert size <= bound and (size == 0) == bool(p["one"]), (s, p, size)
        most = max(most, size / bound)
    assert most > 0.9
    assert [plan(*s)[1] >> 20 for s in sizes[:2]] == [12, 1560]  # MiB, of the sizes that the header gives
