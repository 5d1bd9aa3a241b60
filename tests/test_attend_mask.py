"""The mask that KVCache.attend hands to the library: what the call and the cache say at the time of the call, whatever
calls were before.  CPU: the library's entry is a stand-in that notes its arguments."""
from __future__ import annotations

from types import SimpleNamespace

import numpy as np
import pytest
import torch


@pytest.fixture
def calls(monkeypatch):
    """attend of a cache on the CPU, and the masks that it passed on."""
    from int4_routed_expert_gb300 import attn as A
    A._load()
    seen = []

    def attend(h, q, q_stride, out, lse, mask, batch, stream):
        seen.append((mask.scale, mask.causal, mask.window, mask.sinks))
        return 0

    monkeypatch.setattr(A, "_lib", SimpleNamespace(moe_kv_attend=attend))
    monkeypatch.setattr(A, "_raw_stream", lambda index: 0)
    c = object.__new__(A.KVCache)
    c.h, c.n_q_heads, c.n_kv_heads, c.head_dim, c.page_size = None, 2, 1, 64, 16
    c.device, c._index, c._row, c._mask, c._shared, c.default_scale = torch.device("cpu"), -1, {}, {}, {}, 0.125
    batch = SimpleNamespace(n_tokens=3, index=-1, c=None)
    q = torch.zeros(3, 2, 64, dtype=torch.bfloat16)

    def call(**kw):
        c.attend(q, batch, **kw)
        return seen[-1]

    return c, call


def test_the_default_scale_is_the_cache_s_of_the_time(calls):
    c, call = calls
    assert call() == (0.125, 1, 0, 0)
    c.default_scale = 0.25
    assert call() == (0.25, 1, 0, 0) and call(causal=False) == (0.25, 0, 0, 0)
    c.default_scale = 0.125
    assert call() == (0.125, 1, 0, 0)


@pytest.mark.parametrize("make", [lambda x: torch.tensor(x), lambda x: np.array(x), lambda x: np.array(x, np.float32)])
def test_a_scale_that_changes_in_place(calls, make):
    _, call = calls
    scale = make(0.5)
    assert call(scale=scale)[0] == 0.5
    scale *= 2
    assert call(scale=scale)[0] == 1.0 and call(scale=1)[0] == 1.0 and call(scale=0.5)[0] == 0.5


def test_masks_of_all_kinds(calls):
    _, call = calls
    for causal in (True, 1, 0, False, np.bool_(True), torch.tensor(False)):
        for window, sinks in ((0, 0), (7, 2), (8, 2), (np.int64(8), np.int32(3))):
            for scale in (None, 0.125, 0.5):
                assert call(scale=scale, causal=causal, window=window, sinks=sinks) == \
                    (0.125 if scale is None else scale, int(bool(causal)), window, sinks)
    for bad in (dict(window=8.0), dict(sinks=2.5), dict(window="8"), dict(sinks=None)):  # also after an equal whole number
        with pytest.raises(TypeError):
            call(**bad)


def test_many_masks(calls):
    c, call = calls
    for i in range(300):
        assert call(scale=i / 8)[0] == i / 8 and call(window=i)[2] == i
    assert len(c._mask) <= 64
