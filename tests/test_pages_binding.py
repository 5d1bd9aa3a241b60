"""KVCache.copy's binding where sizes pass 32 bits (CPU: no kernel runs)."""
from __future__ import annotations

from types import SimpleNamespace

import pytest
import torch


def test_a_list_longer_than_the_call_takes_is_refused(monkeypatch):
    """The library counts moves in 32 bits: a longer list would have been cut to its length modulo 2^32."""
    from int4_routed_expert_gb300 import attn as A
    A._load()
    seen = []
    monkeypatch.setattr(A, "_lib", SimpleNamespace(moe_kv_copy=lambda h, moves, n, stream: seen.append(n) or 0))
    monkeypatch.setattr(A, "_raw_stream", lambda index: 0)
    c = object.__new__(A.KVCache)
    c.h, c.device, c._index = None, torch.device("cpu"), -1
    for n in (2 ** 31, 2 ** 32, 2 ** 32 + 5):
        with pytest.raises(ValueError, match="2\\^31"):
            c.copy(torch.empty(n, 3, dtype=torch.int32, device="meta"))
    c.copy(torch.empty(2 ** 31 - 1, 3, dtype=torch.int32, device="meta"))
    c.copy(torch.empty(0, 3, dtype=torch.int32))
    assert seen == [2 ** 31 - 1, 0]
