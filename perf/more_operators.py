"""Workloads of the sequence operators of a serving step: pages of the cache forked, freed, compacted and copied,
attention for sequences that share a prefix, rotary positions with several axes.

A program that answers many questions about one document, image or video, or searches with several beams, calls them
around the operators of ``operators.py``: ``PagePool.fork`` makes the next step's sequences out of the last step's
(shared pages, room for the new tokens, ended sequences freed) and says which pages have to be copied, ``KVCache.copy``
copies them in each layer's cache, ``Rope.apply`` rotates the step's queries and keys, with a position for each axis
where tokens are patches, ``KVCache.attend`` with a ``SharedPrefix`` reads what the sequences share once for all of
them, and ``PagePool.compact`` moves the pages in use to the front of the pool when its memory is wanted elsewhere.

Every case has a plain form in elementary torch operations (``own`` False) and the package's calls (``own`` True).
The layouts are those of the package:
  cache codes  [pages][kv heads][page][dim] float8_e4m3fn, one fp32 scale per (page, kv head), for keys and values
  a pool       table [slots][width] page ids (-1: none), kv_len [slots], ref [pages] uses of each page, all int32
  moves        [n][3] int32: source page, destination page, tokens; a negative source is no move
  a prefix     group g holds sequences cu_seq[g] .. cu_seq[g + 1] - 1, whose first prefix_len[g] tokens lie in
               page_table[g]
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

DEV = "cuda:0"
F8 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases

def _rope(name, tokens, heads, kv_heads, dim, rot, axes, order, restart, interleaved, dtype, max_pos):
    return {"name": name, "op": "rope", "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "dim": dim, "rot": rot,
            "axes": axes, "order": order, "restart": restart, "interleaved": interleaved, "dtype": dtype, "max_pos": max_pos}


def _copy(name, moves, pages, whole, kv_heads, dim, page):
    return {"name": name, "op": "copy", "moves": moves, "pages": pages, "whole": whole, "kv_heads": kv_heads, "dim": dim,
            "page": page}


def _fork(name, slots, kv, page, forked, ended, drafts, new):
    return {"name": name, "op": "fork", "slots": slots, "kv": kv, "page": page, "forked": forked, "ended": ended,
            "drafts": drafts, "new": new}


def _compact(name, slots, kv, page, used):
    return {"name": name, "op": "compact", "slots": slots, "kv": kv, "page": page, "used": used}


def _shared(name, groups, seqs, new, prefix, suffix, heads, kv_heads, dim, page):
    return {"name": name, "op": "shared", "groups": groups, "seqs": seqs, "new": new, "prefix": prefix, "suffix": suffix,
            "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page}


def listed():
    return [
        # a decoding step after an image: a few tokens in fp32 activations, three axes that take turns: latency
        _rope("rope_axes_step", 9, 48, 8, 128, 128, 3, "turns", False, False, "f32", 131072),
        # a video's patches with text before them: blocks of pairs for time, height and width
        _rope("rope_axes_video", 8192, 48, 8, 128, 128, 3, "blocks", False, False, "bf16", 131072),
        # what a step of 24 forks copies in one layer: half-filled pages
        _copy("copy_forks", 24, 700, False, 8, 128, 64),
        # a compaction's pages in one layer
        _copy("copy_compaction", 1501, 4000, True, 8, 128, 64),
        # a step of a beam search: every beam continues one of the last step's, a token each
        _fork("fork_beams", 16, 1500, 64, 0.6, 0.0, 0, 1),
        # a serving step of many sequences: rejected drafts, forks, ended sequences, new prompts in their place
        _fork("fork_serving", 777, 40000, 32, 0.1, 0.06, 4, 4),
        # a small pool after its sequences have come and gone
        _compact("compact_small", 16, 3000, 64, 0.5),
        # a large one
        _compact("compact_large", 400, 50000, 32, 0.7),
        # three answers to one short prompt: the smallest call
        _shared("shared_short", 1, 3, 1, 1000, 40, 48, 8, 128, 64),
        # a decoding step of 64 answers about one document, an idle slot among them
        _shared("shared_batch", 1, 64, 1, 16384, 1500, 64, 8, 128, 64),
        # speculative verify of 4 tokens, three documents with several readers each
        _shared("shared_verify", 3, 37, 4, 66001, 777, 48, 4, 128, 128),
        # the prompts of 12 questions about one document, heads of 64
        _shared("shared_questions", 1, 12, 601, 24001, 650, 32, 2, 64, 32),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rope", "copy", "fork", "compact", "shared", "shared", "shared"))
    dim = rng.choice((64, 128))
    kv_heads = rng.choice((1, 2, 4, 8))
    page = rng.choice((16, 32, 64, 128))
    if op == "rope":
        heads = kv_heads * rng.choice((1, 2, 3, 4, 6, 8))
        c = _rope("", _log_int(rng, 1, 8192), heads, kv_heads, dim, rng.choice((dim // 2, dim)), rng.choice((2, 3, 4)),
                  rng.choice(("blocks", "turns")), rng.random() < 0.5, rng.random() < 0.5, rng.choice(("bf16", "f32")),
                  _log_int(rng, 2048, 1 << 20))
    elif op == "copy":
        bytes_ = 2 * kv_heads * page * dim
        moves = _log_int(rng, 1, min(20000, (190 << 20) // bytes_))
        c = _copy("", moves, int(2 * moves * rng.uniform(1.0, 1.5)) + 1, rng.random() < 0.5, kv_heads, dim, page)
    elif op in ("fork", "compact"):
        slots = _log_int(rng, 1, 800)
        kv = _log_int(rng, 20, min(131072, (1 << 18) * page // slots))
        if op == "fork":
            c = _fork("", slots, kv, page, rng.choice((0.0, 0.1, 0.7)), rng.choice((0.0, 0.1)), rng.choice((0, 0, 4)),
                      rng.choice((1, 1, 5, 300)))
        else:
            c = _compact("", slots, kv, page, rng.uniform(0.3, 0.95))
    else:
        heads = kv_heads * rng.choice((1, 2, 3, 4, 6, 7, 8, 12))
        groups = rng.choice((1, 1, 2, 5))
        seqs = _log_int(rng, 2, 64)
        kind = rng.choice(("token", "token", "verify", "chunk"))
        new = 1 if kind == "token" else rng.randint(2, 8) if kind == "verify" else _log_int(rng, 9, 6000 // seqs)
        seqs = max(seqs, groups)
        most = int(1.5e11 / (heads * dim * seqs * new))
        c = _shared("", groups, seqs, new, _log_int(rng, 50, max(100, min(131072 // groups, most))),
                    _log_int(rng, 1, 2000) + new, heads, kv_heads, dim, page)
    del c["name"]
    return c


# ---------------------------------------------- lengths and pools, by the case alone

def _members(case):
    """A shared case's (sequences of each group, prefix lengths, lengths, new tokens); an idle slot has length 0."""
    r = random.Random(case["seqs"] * 1000003 + case["prefix"])
    cuts = sorted(r.sample(range(1, case["seqs"]), case["groups"] - 1))
    cu = [0, *cuts, case["seqs"]]
    prefix = [case["prefix"]] + [max(1, int(case["prefix"] * r.uniform(0.1, 1.0))) for _ in range(case["groups"] - 1)]
    kv, new = [], []
    for g in range(case["groups"]):
        for i in range(cu[g], cu[g + 1]):
            u = r.uniform(0.05, 1.0) if i else 1.0
            n = case["new"] if case["new"] <= 8 else max(1, int(case["new"] * u))
            kv.append(prefix[g] + max(n, int(case["suffix"] * u)))
            new.append(n)
    if case["seqs"] >= 32:
        kv[-1] = 0  # a slot that has no sequence now: its rows see nothing
    return cu, prefix, kv, new


def _pool(case, seed):
    """A fork or compact case's pool in numpy: table, lengths, uses, and a fork's parents, kept and new tokens.

    Families of up to four slots share the first half of their pages; pages lie anywhere in the pool."""
    size = random.Random(case["slots"] * 1000003 + case["kv"])  # what the sizes hang on
    g = np.random.default_rng(seed)
    n, page = case["slots"], case["page"]
    kv = np.array([case["kv"]] + [max(1, int(case["kv"] * size.uniform(0.02, 1.0))) for _ in range(n - 1)], np.int64)
    if n >= 16:
        kv[n // 2] = 0  # an empty slot
    have = -(-kv // page)
    prompt = 400 + 3 * case.get("new", 0)
    width = -(-(case["kv"] + (prompt if case["op"] == "fork" else 0)) // page)
    lead = np.arange(n) // 4 * 4
    half = np.minimum(kv, kv[lead]) // (2 * page)  # whole pages that a slot shares with its family's first
    half[lead == np.arange(n)] = 0
    mine = have - half
    off = np.cumsum(mine) - mine
    total = int(mine.sum())
    out = {"table": np.full((n, width), -1, np.int32), "kv_len": kv.astype(np.int32)}
    parent = keep = new = None
    pages = int(total / case["used"]) + 1 if case["op"] == "compact" else 0
    if case["op"] == "fork":
        parent, new = np.arange(n), np.full(n, case["new"])
        keep = np.full(n, 1 << 30)
        for i in range(n):
            u = size.random()
            if u < case["ended"]:  # a new prompt in the place of an ended sequence, or nothing
                parent[i], new[i] = -1, size.choice((0, size.randint(1, prompt)))
            elif u < case["ended"] + case["forked"]:
                parent[i] = size.randrange(n)
            if parent[i] >= 0 and case["drafts"]:
                keep[i] = max(0, kv[parent[i]] - size.randint(0, case["drafts"]))
        keep = np.where(parent >= 0, np.minimum(keep, kv[parent]), 0)  # (a second pass starts from what the first made)
        pages = max(total, int((-(-(keep + new) // page)).sum())) + n
        out |= {"parent": parent.astype(np.int32), "keep": keep.astype(np.int32), "new": new.astype(np.int32)}
    ids = g.permutation(pages)[:total].astype(np.int32)
    j = np.arange(width)
    own_page = ids[np.clip(off[:, None] + j - half[:, None], 0, total - 1)]
    lead_page = ids[np.clip(off[lead][:, None] + j, 0, total - 1)]
    row = np.where(j < half[:, None], lead_page, own_page)
    out["table"] = np.where(j < have[:, None], row, -1).astype(np.int32)
    out["ref"] = np.bincount(out["table"][out["table"] >= 0], minlength=pages).astype(np.int32)
    return out


def work(case):
    op = case["op"]
    if op == "rope":
        n = case["tokens"] * (case["heads"] + case["kv_heads"])
        size = TYPES[case["dtype"]].itemsize
        return {"bytes": 2 * n * case["dim"] * size + 4 * case["axes"] * case["tokens"], "flops": 3 * n * case["rot"]}
    if op == "copy":
        tokens = sum(_move_tokens(case))
        return {"bytes": 4 * tokens * case["kv_heads"] * case["dim"] + case["moves"] * (16 * case["kv_heads"] + 12),
                "flops": tokens}
    if op in ("fork", "compact"):
        p = _pool(case, 0)
        entries, pages, n = int((p["table"] >= 0).sum()), p["ref"].size, case["slots"]
        return {"bytes": 8 * (entries + pages) + (40 * n if op == "fork" else 6 * pages), "flops": entries + pages}
    cu, prefix, kv, new = _members(case)
    live = [(k, n) for k, n in zip(kv, new) if k]
    keys = sum(prefix) + sum(k - prefix[g] for g in range(len(prefix)) for k in kv[cu[g]:cu[g + 1]] if k)
    pairs = sum(n * k - n * (n - 1) // 2 for k, n in live)
    return {"bytes": 2 * keys * case["kv_heads"] * case["dim"] + 4 * sum(new) * case["heads"] * case["dim"],
            "flops": 4 * pairs * case["heads"] * case["dim"]}


# ---------------------------------------------------------------- the inputs

def _axis_of(case):
    """The axis of each pair: blocks of a quarter, then equal parts, or axes that take turns."""
    half, axes = case["rot"] // 2, case["axes"]
    if case["order"] == "turns":
        return [i % axes for i in range(half)]
    first = half // 4 if axes > 2 else half // 2
    return [0 if i < first else 1 + (i - first) * (axes - 1) // (half - first) for i in range(half)]


def _frequencies(case):
    """Radians per position of each pair, in 64 bits; `restart`: each axis has the whole range of them."""
    axis = np.array(_axis_of(case))
    half = axis.size
    if not case["restart"]:
        return 1e6 ** (-np.arange(half) / half)
    same = axis[:, None] == axis
    rank = np.tril(same, -1).sum(1)
    return 1e6 ** (-rank / same.sum(1))


def _move_tokens(case):
    r = random.Random(case["moves"] * 1000003 + case["pages"])
    return [case["page"] if case["whole"] else r.randint(1, case["page"] - 1) for _ in range(case["moves"])]


def _block_scale(amax):
    """The smallest power of two s >= 2^-64 with amax <= 448 s."""
    m, e = torch.frexp(amax)
    e = torch.where(m > 0.875, e - 8, e - 9)
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e.clamp(min=-64)), 2.0 ** -64)


def _store(g, pages, kv_heads, page, dim):
    """Codes and scales of a pool of pages in use: channels of different size, pages of different size."""
    codes = torch.empty(pages, kv_heads, page, dim, device=DEV, dtype=F8)
    scales = torch.empty(pages, kv_heads, device=DEV)
    channel = torch.exp(0.5 * torch.randn(kv_heads, 1, dim, device=DEV, generator=g))
    step = max(1, (1 << 27) // (kv_heads * page * dim))
    for a in range(0, pages, step):
        x = torch.randn(min(step, pages - a), kv_heads, page, dim, device=DEV, generator=g) * channel
        x *= torch.exp(0.3 * torch.randn(x.shape[0], kv_heads, 1, 1, device=DEV, generator=g))
        s = _block_scale(x.abs().amax((2, 3)))
        codes[a:a + step] = (x / s[..., None, None]).to(F8)
        scales[a:a + step] = s
    return codes, scales


def _int32(x):
    return torch.as_tensor(np.asarray(x, np.int32), device=DEV)


def _inputs(case, seed):
    g = torch.Generator(DEV)
    g.manual_seed(seed)
    op, s = case["op"], {"case": case}

    def randn(*shape):
        return torch.randn(*shape, device=DEV, generator=g)

    if op == "rope":
        t, axes, dtype = case["tokens"], case["axes"], TYPES[case["dtype"]]
        if t <= 256:  # tokens of different sequences
            s["pos"] = torch.randint(0, case["max_pos"], (axes, t), device=DEV, generator=g).to(torch.int32)
        else:  # text, then patches: frames of side x side, the last two axes within a frame
            first = torch.randint(0, case["max_pos"], (1,), device=DEV, generator=g)
            side, text = max(2, int(math.sqrt(t / 8))), t // 8
            i = torch.arange(t, device=DEV)
            patch = (i - text).clamp(min=0)
            place = [patch // (side * side)] * (axes - 2) + [patch // side % side, patch % side]
            s["pos"] = torch.stack([first + torch.where(i < text, i, text + p) for p in place]).to(torch.int32)
        s["q"], s["k"] = randn(t, case["heads"], case["dim"]).to(dtype), randn(t, case["kv_heads"], case["dim"]).to(dtype)
        return s
    if op in ("fork", "compact"):
        for name, x in _pool(case, seed).items():
            s[name] = _int32(x)
        return s
    page, hkv, dim = case["page"], case["kv_heads"], case["dim"]
    if op == "copy":
        order = torch.randperm(case["pages"], device=DEV, generator=g)
        n = case["moves"]
        s["moves"] = torch.stack((order[:n].sort().values, order[n:2 * n].sort().values,
                                  torch.tensor(_move_tokens(case), device=DEV)), 1).to(torch.int32).contiguous()
        s["k_codes"], s["k_scale"] = _store(g, case["pages"], hkv, page, dim)
        s["v_codes"], s["v_scale"] = _store(g, case["pages"], hkv, page, dim)
        return s
    cu, prefix, kv, new = _members(case)
    # a prefix's pages, then each sequence's own from the page in which its prefix ends (a copy, if it begins there)
    ends = [(p // page, -(-p // page)) for p in prefix]
    of = [b for b in range(case["groups"]) for _ in range(cu[b], cu[b + 1])]
    mine = [max(0, -(-k // page) - ends[b][0]) for b, k in zip(of, kv)]
    total = sum(e[1] for e in ends) + sum(mine)
    ids = torch.randperm(total + 3, device=DEV, generator=g)[:total].cpu().numpy()
    table = np.full((case["groups"], max(e[1] for e in ends)), -1, np.int32)
    seq_table = np.full((case["seqs"], max(max(-(-k // page), 1) for k in kv)), -1, np.int32)
    at = 0
    for b, (_, n) in enumerate(ends):
        table[b, :n], at = ids[at:at + n], at + n
    for i, (b, n) in enumerate(zip(of, mine)):
        if kv[i]:
            seq_table[i, :ends[b][0]] = table[b, :ends[b][0]]
            seq_table[i, ends[b][0]:ends[b][0] + n], at = ids[at:at + n], at + n
    s |= {"table": _int32(seq_table), "prefix_table": _int32(table), "kv_len": _int32(kv), "cu_seq": _int32(cu),
          "prefix_len": _int32(prefix), "cu_q": _int32(np.concatenate(([0], np.cumsum(new)))), "n_tokens": sum(new),
          "max_q": max(new), "max_kv": max(kv), "max_prefix": max(prefix),
          "max_group": max(sum(new[cu[b]:cu[b + 1]]) for b in range(case["groups"])),
          "max_own": max(k - prefix[b] if k else 1 for b, k in zip(of, kv))}
    s["k_codes"], s["k_scale"] = _store(g, total + 3, hkv, page, dim)
    s["v_codes"], s["v_scale"] = _store(g, total + 3, hkv, page, dim)
    s["q"] = (1.2 * randn(s["n_tokens"], case["heads"], dim)).to(torch.bfloat16)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "rope":
        s["freq"] = torch.from_numpy(_frequencies(case)).to(DEV)
        s["axis"] = torch.tensor(_axis_of(case), device=DEV)
    if op == "fork":
        n = case["slots"]
        s |= {"cu_q": torch.zeros(n + 1, device=DEV, dtype=torch.int32), "free": torch.zeros(1, device=DEV, dtype=torch.int32)}
    if op == "compact":
        s["free"] = torch.zeros(1, device=DEV, dtype=torch.int32)
    if own:
        import int4_routed_expert_gb300 as m
        if op == "rope":
            s["rope"] = m.Rope(case["rot"], inv_freq=_frequencies(case), interleaved=case["interleaved"], axes=_axis_of(case))
        elif op in ("fork", "compact"):
            s["pool"] = m.PagePool(s["table"], s["kv_len"], s["ref"], case["page"])
        else:
            s["cache"] = m.KVCache(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"],
                                   n_q_heads=case.get("heads", case["kv_heads"]), max_seqs=case.get("seqs", 1),
                                   max_tokens=s.get("n_tokens", 1), max_kv_len=s.get("max_kv", 1))
        if op == "shared":
            s["batch"] = m.SeqBatch(s["cu_q"], s["kv_len"], s["table"], s["n_tokens"], s["max_q"], s["max_kv"])
            s["prefix"] = m.SharedPrefix(s["cu_seq"], s["prefix_len"], s["prefix_table"], s["max_group"], s["max_prefix"])
    return s


# -------------------------------------------------------------- the plain form

def _plain_rope(s):
    c = s["case"]
    rot = c["rot"]
    angle = s["pos"].double()[s["axis"]].T * s["freq"]
    cos, sin = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]

    def rotate(x):
        y = x.float()
        if c["interleaved"]:
            a, b = y[..., 0:rot:2], y[..., 1:rot:2]
            r = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
        else:
            a, b = y[..., :rot // 2], y[..., rot // 2:rot]
            r = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
        return torch.cat((r, y[..., rot:]), -1).to(x.dtype)

    return rotate(s["q"]), rotate(s["k"])


def _plain_copy(s):
    src, dst, n = s["moves"].long().unbind(1)
    page = s["case"]["page"]
    stays = (torch.arange(page, device=DEV) >= n[:, None])[:, None, :, None]

    def move(codes, scales):
        raw = codes.view(torch.uint8)
        raw[dst] = torch.where(stays, raw[dst], raw[src])
        scales[dst] = scales[src]

    move(s["k_codes"], s["k_scale"])
    move(s["v_codes"], s["v_scale"])
    return s["k_codes"], s["k_scale"], s["v_codes"], s["v_scale"]


def _uses(table, pages):
    """How often each page stands in a table."""
    at = torch.where(table >= 0, table, pages).flatten().long()
    return torch.zeros(pages + 1, device=DEV, dtype=torch.int32).index_add_(0, at, torch.ones_like(at, dtype=torch.int32))[:pages]


def _plain_fork(s):
    table, ref, page = s["table"], s["ref"], s["case"]["page"]
    (n, width), pages = table.shape, ref.shape[0]
    parent, new = s["parent"].long(), s["new"].long()
    i, j = torch.arange(n, device=DEV), torch.arange(width, device=DEV)
    p = parent.clamp(min=0)
    keep = torch.where(parent >= 0, torch.minimum(s["keep"].long().clamp(min=0), s["kv_len"].long()[p]), 0)
    kept, have = (keep + page - 1) // page, (keep + new + page - 1) // page
    row = torch.where(j < kept[:, None], table[p], -1)
    ref1 = ref - _uses(table, pages) + _uses(row, pages)
    # sequences that write into a page others use too: they copy it, but for the first where all of its users do
    lands = (keep % page != 0) & (new > 0)
    x = torch.where(lands, row.gather(1, (kept - 1).clamp(min=0)[:, None])[:, 0].long(), pages)
    landers = torch.zeros(pages + 1, device=DEV, dtype=torch.int32).index_add_(0, x, torch.ones_like(x, dtype=torch.int32))
    first = torch.full((pages + 1,), n, device=DEV).scatter_reduce(0, x, i, "amin")
    shared = torch.cat((ref1, ref1.new_zeros(1)))[x]
    copies = lands & (shared > 1) & ~((landers[x] == shared) & (first[x] == i))
    need = copies.long() + have - kept
    off = need.cumsum(0) - need
    free = torch.sort((ref1 != 0).to(torch.int8), stable=True).indices  # free pages first, in their order
    at = off[:, None] + copies[:, None] + j - kept[:, None]
    at = torch.where(copies[:, None] & (j == kept[:, None] - 1), off[:, None], at)
    fresh = ((j >= kept[:, None]) & (j < have[:, None])) | (copies[:, None] & (j == kept[:, None] - 1))
    row = torch.where(fresh, free[at.clamp(0, pages - 1)].to(torch.int32), row)
    to = row.gather(1, (kept - 1).clamp(min=0)[:, None])[:, 0].long()
    moves = torch.full((n + 1, 3), -1, device=DEV, dtype=torch.int32)
    moves[torch.where(copies, copies.long().cumsum(0) - 1, n)] = torch.stack((x, to, keep % page), 1).to(torch.int32)
    moves[n] = -1
    s["ref"].copy_(ref - _uses(table, pages) + _uses(row, pages))
    s["table"].copy_(row)
    s["kv_len"].copy_(keep + new)
    s["cu_q"][1:] = new.cumsum(0)
    s["free"].copy_((s["ref"] == 0).sum())
    return s["table"], s["kv_len"], s["ref"], s["cu_q"], s["free"], moves[:n]


def _plain_compact(s):
    table, ref = s["table"], s["ref"]
    pages = ref.shape[0]
    ids = torch.arange(pages, device=DEV)
    used = ref != 0
    n_used = used.sum()
    mover, hole = used & (ids >= n_used), ~used & (ids < n_used)
    end = pages // 2
    moves = torch.full((end + 1, 3), -1, device=DEV, dtype=torch.int32)
    rank = mover.cumsum(0) - 1
    moves[torch.where(mover, rank, end), 0] = ids.to(torch.int32)
    moves[torch.where(hole, hole.cumsum(0) - 1, end), 1] = ids.to(torch.int32)
    moves[:, 2] = torch.where(moves[:, 0] >= 0, s["case"]["page"], -1)
    to = torch.where(mover, moves[rank.clamp(0, end), 1].long(), ids)
    s["table"].copy_(torch.where(table >= 0, to[table.clamp(min=0).long()], -1))
    s["ref"].copy_(torch.zeros_like(ref).index_add_(0, to, torch.where(used, ref, 0)))
    s["free"].copy_(pages - n_used)
    return s["table"], s["ref"], s["free"], moves[:end]


def _plain_shared(s):
    c = s["case"]
    d, hkv, heads, page = c["dim"], c["kv_heads"], c["heads"], c["page"]
    gq = heads // hkv
    cu_q, cu_seq, kv = s["cu_q"].long(), s["cu_seq"].long(), s["kv_len"].long()
    n_seqs, groups = kv.numel(), s["prefix_len"].numel()
    t = torch.arange(s["n_tokens"], device=DEV)
    seq = torch.searchsorted(cu_q, t, right=True) - 1
    pos = kv[seq] - cu_q[seq + 1] + t
    group = torch.searchsorted(cu_seq, torch.arange(n_seqs, device=DEV), right=True) - 1  # of a sequence
    prefix = s["prefix_len"].long()
    joins = kv - (cu_q[1:] - cu_q[:-1]) >= prefix[group]
    begin = torch.where(joins, prefix[group], 0)  # of a sequence's own keys

    def rows(at, index, width):  # queries as [batch][kv heads][heads of it * width][d]
        q = torch.zeros(at, width, heads, d, device=DEV)
        q[index] = s["q"].float()
        return q.view(at, width, hkv, gq, d).permute(0, 2, 3, 1, 4).reshape(at, hkv, gq * width, d)

    def back(x, at, index, width):  # ... and as [tokens][heads][...] again
        return x.view(at, hkv, gq, width, -1).permute(0, 3, 1, 2, 4).reshape(at, width, heads, -1)[index]

    def part(q, keys, values, hidden):  # (sums, largest, sum of weights) of rows
        score = torch.matmul(q, keys.transpose(2, 3)) * d ** -0.5
        score = score.masked_fill_(hidden, -math.inf)
        top = score.amax(-1, keepdim=True).clamp(min=-1e30)
        e = torch.exp(score.sub_(top))
        return torch.matmul(e, values), top, e.sum(-1, keepdim=True)

    def whole(codes, scales):
        table = s["prefix_table"].long().clamp(min=0)
        x = codes[table].float() * scales[table][..., None, None]
        return x.transpose(1, 2).reshape(groups, hkv, table.shape[1] * page, d)

    of = group[seq]
    index = (of, t - cu_q[cu_seq[:-1]][of])
    q = rows(groups, index, s["max_group"])
    hidden = (torch.arange(s["prefix_table"].shape[1] * page, device=DEV) >= prefix[:, None])[:, None, None]
    p = part(q, whole(s["k_codes"], s["k_scale"]), whole(s["v_codes"], s["v_scale"]), hidden)
    o1, m1, l1 = (back(x, groups, index, s["max_group"]) for x in p)
    out = ~joins[seq][:, None, None]  # rows of sequences that have less than the prefix
    o1, l1, m1 = o1.masked_fill(out, 0.0), l1.masked_fill(out, 0.0), m1.masked_fill(out, -1e30)

    j = begin[:, None] + torch.arange(s["max_own"], device=DEV)
    at = s["table"].long().gather(1, (j // page).clamp(max=s["table"].shape[1] - 1)).clamp(min=0)

    def mine(codes, scales):
        return (codes[at, :, j % page].float() * scales[at][..., None]).transpose(1, 2)

    index = (seq, t - cu_q[seq])
    q = rows(n_seqs, index, s["max_q"])
    p = torch.full((n_seqs, s["max_q"]), -1, device=DEV, dtype=torch.int64)
    p[index] = pos
    hidden = (j[:, None] > p[..., None])[:, None, None].expand(-1, 1, gq, -1, -1).flatten(2, 3)
    p = part(q, mine(s["k_codes"], s["k_scale"]), mine(s["v_codes"], s["v_scale"]), hidden)
    o2, m2, l2 = (back(x, n_seqs, index, s["max_q"]) for x in p)
    top = torch.maximum(m1, m2)
    f1, f2 = torch.exp(m1 - top), torch.exp(m2 - top)
    return ((o1 * f1 + o2 * f2) / (l1 * f1 + l2 * f2).clamp(min=1e-30)).to(s["q"].dtype)


def run(s):
    op = s["case"]["op"]
    if own:
        if op == "rope":
            return s["rope"].apply(s["q"], s["pos"], k=s["k"])
        if op == "copy":
            s["cache"].copy(s["moves"])
            return s["k_codes"], s["k_scale"], s["v_codes"], s["v_scale"]
        if op == "fork":
            moves = s["pool"].fork(s["parent"], s["new"], keep=s["keep"])
            return s["table"], s["kv_len"], s["ref"], s["pool"].cu_q, s["pool"].free, moves
        if op == "compact":
            moves = s["pool"].compact()
            return s["table"], s["ref"], s["pool"].free, moves
        return s["cache"].attend(s["q"], s["batch"], prefix=s["prefix"])
    if op == "rope":
        return _plain_rope(s)
    if op == "copy":
        return _plain_copy(s)
    if op == "fork":
        return _plain_fork(s)
    if op == "compact":
        return _plain_compact(s)
    return _plain_shared(s)


# ------------------------------------------------------- the definition, in 64 bits

def _exact_fork(case, seed):
    p, page = _pool(case, seed), case["page"]
    table, kv, ref, new = (p[k].tolist() for k in ("table", "kv_len", "ref", "new"))
    keeps = [min(max(k, 0), kv[b]) if b >= 0 else 0 for b, k in zip(p["parent"].tolist(), p["keep"].tolist())]
    rows = [table[b][:-(-k // page)] for b, k in zip(p["parent"].tolist(), keeps)]
    uses = [0] * len(ref)
    for row in rows:
        for x in row:
            uses[x] += 1
    writes = {}  # pages that hold a sequence's last kept token and its next one: their writers
    for i, (k, n) in enumerate(zip(keeps, new)):
        if k % page and n:
            writes.setdefault(rows[i][-1], []).append(i)
    free, moves = iter([x for x, u in enumerate(uses) if u == 0]), []
    for i, (k, n) in enumerate(zip(keeps, new)):
        x = rows[i][-1] if k % page and n else -1
        if x >= 0 and uses[x] > 1 and not (len(writes[x]) == uses[x] and writes[x][0] == i):
            rows[i][-1] = next(free)
            moves.append([x, rows[i][-1], k % page])
        while len(rows[i]) * page < k + n:
            rows[i].append(next(free))
    out, uses = np.full(p["table"].shape, -1), np.zeros(len(ref))
    for i, row in enumerate(rows):
        out[i, :len(row)] = row
        np.add.at(uses, row, 1)
    moves += [[-1, -1, -1]] * (len(rows) - len(moves))
    return [_int32(v) for v in (out, np.array(keeps) + new, uses, [0, *np.cumsum(new)], [int((uses == 0).sum())], moves)]


def _exact_compact(case, seed):
    p = _pool(case, seed)
    table, ref = p["table"].astype(np.int64), p["ref"].tolist()
    used = [x for x, uses in enumerate(ref) if uses]
    holes = [x for x, uses in enumerate(ref) if not uses and x < len(used)]
    to, moves = np.arange(len(ref)), []
    for dst, src in zip(holes, used[len(used) - len(holes):]):
        to[src] = dst
        moves.append([src, dst, case["page"]])
        ref[dst], ref[src] = ref[src], 0
    moves += [[-1, -1, -1]] * (len(ref) // 2 - len(moves))
    return [_int32(v) for v in (np.where(table >= 0, to[table], -1), ref, [len(ref) - len(used)], np.array(moves).reshape(-1, 3))]


def exact(case, seed):
    op = case["op"]
    if op == "fork":
        return _exact_fork(case, seed) if case["slots"] * case["kv"] // case["page"] < 1 << 20 else None
    if op == "compact":
        return _exact_compact(case, seed)
    s = _inputs(case, seed)
    if op == "rope":
        r, out = case["rot"], []
        angle = torch.empty(case["tokens"], r // 2, dtype=torch.float64, device=DEV)
        for pair, (axis, f) in enumerate(zip(_axis_of(case), _frequencies(case).tolist())):
            angle[:, pair] = s["pos"][axis].double() * f
        turn = torch.polar(torch.ones_like(angle), angle)[:, None]
        for x in (s["q"].double(), s["k"].double()):
            y = x.clone()
            pick = (slice(0, r, 2), slice(1, r, 2)) if case["interleaved"] else (slice(0, r // 2), slice(r // 2, r))
            z = torch.complex(x[..., pick[0]].contiguous(), x[..., pick[1]].contiguous()) * turn
            y[..., pick[0]], y[..., pick[1]] = z.real, z.imag
            out.append(y)
        return tuple(out)
    page = case["page"]
    if op == "copy":
        out = [x.clone() for x in (s["k_codes"], s["k_scale"], s["v_codes"], s["v_scale"])]
        for src, dst, n in s["moves"].tolist():
            for codes, scales, was, scale_was in ((out[0], out[1], s["k_codes"], s["k_scale"]),
                                                  (out[2], out[3], s["v_codes"], s["v_scale"])):
                codes[dst, :, :n] = was[src, :, :n]
                scales[dst] = scale_was[src]
        return tuple(x.double() for x in out)
    cu, prefix, kv, new = _members(case)
    cu_q = s["cu_q"].tolist()

    def tokens(codes, scales, row, a, z):  # keys or values a..z of a table's row, [kv heads][z - a][dim]
        pages = row[a // page:-(-z // page)].long()
        x = codes[pages].double() * scales[pages].double()[..., None, None]
        return x.transpose(0, 1).flatten(1, 2)[:, a % page:a % page + z - a]

    g = case["heads"] // case["kv_heads"]
    out = torch.zeros(s["n_tokens"], case["heads"], case["dim"], device=DEV, dtype=torch.float64)
    for b in range(case["groups"]):
        first = [tokens(c, x, s["prefix_table"][b], 0, prefix[b])
                 for c, x in ((s["k_codes"], s["k_scale"]), (s["v_codes"], s["v_scale"]))]
        for i in range(cu[b], cu[b + 1]):
            if kv[i] == 0:
                continue
            k, v = (torch.cat((f, tokens(c, x, s["table"][i], prefix[b], kv[i])), 1)
                    for f, c, x in zip(first, (s["k_codes"], s["v_codes"]), (s["k_scale"], s["v_scale"])))
            sees = torch.arange(kv[i], device=DEV) <= torch.arange(kv[i] - new[i], kv[i], device=DEV)[:, None]
            q = s["q"][cu_q[i]:cu_q[i + 1]].double().transpose(0, 1)
            for h in range(case["kv_heads"]):
                w = torch.softmax(torch.where(sees, q[h * g:h * g + g] @ k[h].T / math.sqrt(case["dim"]), -math.inf), -1)
                out[cu_q[i]:cu_q[i + 1], h * g:h * g + g] = (w @ v[h]).transpose(0, 1)
    return out
