"""Workloads of the attention-side serving operators: rotary positions, the 8-bit paged cache, attention over it.

A decoder layer around the MoE layer of this package calls them in this order: rotate the step's queries and
keys (``Rope.apply``), quantise its keys and values into the paged cache (``KVCache.write``), attend over the
cache (``KVCache.attend``); ``KVCache.read`` gives cached tokens back (inspection, migration, recomputation).

Every case has a plain form in elementary torch operations (``own`` False) and the package's calls (``own``
True).  The layouts are those of the package:
  cache codes  [pages][kv heads][page][dim] float8_e4m3fn, one fp32 scale per (page, kv head), for keys and values
  a batch      sequence b has ``kv_len[b]`` tokens in the cache, the last ``cu_q[b+1] - cu_q[b]`` of them are the
               call's; ``page_table[b][i]`` holds tokens ``i * page`` onwards
The hidden size of the layer is 6144: 48 heads of 128; the other head layouts are generic.
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

def _rope(name, tokens, heads, kv_heads, dim, rot, interleaved, scaling, dtype, max_pos):
    return {"name": name, "op": "rope", "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "dim": dim, "rot": rot,
            "interleaved": interleaved, "scaling": scaling, "dtype": dtype, "max_pos": max_pos}


def _cache(name, op, seqs, new, kv, ragged, kv_heads, dim, page, dtype):
    return {"name": name, "op": op, "seqs": seqs, "new": new, "kv": kv, "ragged": ragged, "kv_heads": kv_heads,
            "dim": dim, "page": page, "dtype": dtype}


def _attn(name, seqs, new, kv, ragged, heads, kv_heads, dim, page, window=0, sinks=0):
    return {"name": name, "op": "attn", "seqs": seqs, "new": new, "kv": kv, "ragged": ragged, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "window": window, "sinks": sinks, "dtype": "bf16"}


def listed():
    return [
        # a decoding step's rotation of a few tokens in fp32 activations, half layout, whole head: latency
        _rope("rope_step", 7, 48, 8, 128, 128, False, "none", "f32", 131072),
        # a prompt's rotation: half of each head, adjacent pairs, frequencies stretched for a long context
        _rope("rope_prompt", 8192, 48, 8, 128, 64, True, "yarn", "bf16", 131072),
        # one new token for each of 48 decoding sequences, into half-filled pages
        _cache("write_step", "write", 48, 1, 2000, True, 8, 128, 64, "bf16"),
        # three prompts of different lengths written at once, one of them starting inside a page
        _cache("write_prompt", "write", 3, 8191, 9000, True, 8, 128, 64, "bf16"),
        # reading back one short sequence
        _cache("read_short", "read", 1, 333, 333, False, 4, 64, 16, "f32"),
        # reading back long sequences for migration
        _cache("read_long", "read", 5, 16384, 16384, True, 8, 128, 32, "bf16"),
        # the first tokens of a chat, one sequence: the smallest call
        _attn("token_short", 1, 1, 777, False, 48, 8, 128, 64),
        # a serving step: 64 sequences of very different lengths, an idle slot among them
        _attn("token_batch", 64, 1, 16384, True, 64, 8, 128, 64),
        # speculative verify of 4 tokens over long contexts
        _attn("verify_long", 4, 4, 131072, True, 48, 4, 128, 128),
        # one whole prompt
        _attn("prompt", 1, 8192, 8192, False, 48, 8, 128, 64),
        # chunks of a few long prompts, heads of 64
        _attn("chunk", 3, 700, 24001, True, 32, 2, 64, 32),
        # a windowed layer with 4 first tokens that stay visible, chunked
        _attn("window", 4, 1025, 32768, True, 48, 8, 128, 16, window=4096, sinks=4),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rope", "write", "read", "attn", "attn", "attn"))
    dim = rng.choice((64, 128))
    kv_heads = rng.choice((1, 2, 4, 8))
    page = rng.choice((16, 32, 64, 128))
    if op == "rope":
        heads = kv_heads * rng.choice((1, 2, 3, 4, 6, 8))
        c = _rope("", _log_int(rng, 1, 8192), heads, kv_heads, dim, rng.choice((dim // 4, dim // 2, dim)),
                  rng.random() < 0.5, rng.choice(("none", "linear", "ntk", "yarn")), rng.choice(("bf16", "f32")),
                  _log_int(rng, 2048, 1 << 20))
    elif op in ("write", "read"):
        seqs = _log_int(rng, 1, 64)
        kv = _log_int(rng, 1, 131072 // seqs)
        new = min(kv, _log_int(rng, 1, 16384))
        c = _cache("", op, seqs, kv if op == "read" else new, kv, rng.random() < 0.7, kv_heads, dim, page,
                   rng.choice(("bf16", "f32")))
    else:
        heads = kv_heads * rng.choice((1, 2, 3, 4, 6, 7, 8, 12))
        kind = rng.choice(("token", "verify", "chunk", "prompt"))
        if kind == "prompt":
            seqs = _log_int(rng, 1, 4)
            kv = new = _log_int(rng, 16, 4096)
        elif kind == "chunk":
            seqs, new = _log_int(rng, 1, 4), _log_int(rng, 9, 1500)
            kv = _log_int(rng, new, 32768)
        else:
            new = 1 if kind == "token" else rng.randint(2, 8)
            seqs = _log_int(rng, 1, 64)
            kv = _log_int(rng, 16, min(262144, (1 << 20) // seqs))
        windowed = rng.random() < 0.3
        c = _attn("", seqs, new, kv, rng.random() < 0.7, heads, kv_heads, dim, page,
                  _log_int(rng, 16, 8192) if windowed else 0, rng.choice((0, 1, 4, 20)) if windowed else 0)
    del c["name"]
    return c


def _lengths(case):
    """(kv_len, new tokens) of each sequence, by the case alone."""
    r = random.Random(case["seqs"] * 1000003 + case["kv"])
    kv, new = [case["kv"]], [case["new"]]
    for _ in range(1, case["seqs"]):
        u = r.uniform(0.02, 1.0) if case["ragged"] else 1.0
        length = max(1, int(case["kv"] * u))
        if case["new"] == case["kv"]:
            n = length
        else:
            n = case["new"] if case["new"] <= 8 else max(1, int(case["new"] * u))
        kv.append(length)
        new.append(min(length, n))
    if case["op"] == "attn" and case["ragged"] and case["seqs"] >= 16:
        kv[-1] = 0  # a slot of the batch that has no sequence now: its query sees nothing
    return kv, new


def _visible(length, n, window, sinks):
    """Visible (query, key) pairs of one sequence and the keys that some query sees."""
    p = np.arange(length - n, length, dtype=np.int64)
    p = p[p >= 0]
    if not len(p):
        return 0, 0
    if not window:
        return int((p + 1).sum()), length
    lo = np.maximum(p - window + 1, 0)
    return int((p + 1 - lo + np.minimum(lo, sinks)).sum()), int(length - lo[0] + min(lo[0], sinks))


def work(case):
    if case["op"] == "rope":
        n = case["tokens"] * (case["heads"] + case["kv_heads"])
        size = TYPES[case["dtype"]].itemsize
        return {"bytes": 2 * n * case["dim"] * size + 4 * case["tokens"], "flops": 3 * n * case["rot"]}
    kv, new = _lengths(case)
    hd = case["kv_heads"] * case["dim"]
    if case["op"] in ("write", "read"):
        size = TYPES[case["dtype"]].itemsize
        pages = sum((length - 1) // case["page"] - (length - n) // case["page"] + 1 for length, n in zip(kv, new))
        return {"bytes": 2 * sum(new) * hd * (size + 1) + 8 * pages * case["kv_heads"], "flops": 2 * sum(new) * hd * 2}
    pairs, keys = (sum(v) for v in zip(*(_visible(length, n, case["window"], case["sinks"]) for length, n in zip(kv, new))))
    return {"bytes": 2 * keys * hd + 4 * sum(new) * case["heads"] * case["dim"],
            "flops": 4 * pairs * case["heads"] * case["dim"]}


# ---------------------------------------------------------------- the inputs

def _scaling(case):
    """(kind, factor, original length) of a case's rotary frequencies."""
    return {"none": (None, 1.0, 0), "linear": ("linear", 8.0, 0), "ntk": ("ntk", 4.0, 0),
            "yarn": ("yarn", 16.0, 8192)}[case["scaling"]]


THETA = 1e6


def _frequencies(case):
    """Radians per position of each pair in 64 bits, and the amplitude of its sine and cosine."""
    kind, factor, original = _scaling(case)
    rot = case["rot"]
    i = np.arange(rot // 2, dtype=np.float64)
    theta = THETA * factor ** (rot / (rot - 2)) if kind == "ntk" else THETA
    f = theta ** (-2 * i / rot)
    if kind == "linear":
        return f / factor, 1.0
    if kind != "yarn":
        return f, 1.0

    def at(turns):  # the pair that makes so many turns over the original length
        return rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(THETA))

    low, high = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot - 1)
    ramp = np.clip((i - low) / max(high - low, 1e-3), 0.0, 1.0)
    return f * (1 - ramp) + f / factor * ramp, 0.1 * math.log(factor) + 1.0


def _block_scale(amax):
    """The smallest power of two s >= 2^-64 with amax <= 448 s."""
    m, e = torch.frexp(amax)
    e = torch.where(m > 0.875, e - 8, e - 9)
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e.clamp(min=-64)), 2.0 ** -64)


def _pool(g, pages, kv_heads, page, dim):
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


def _inputs(case, seed):
    g = torch.Generator(DEV)
    g.manual_seed(seed)
    dtype = TYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, device=DEV, generator=g)

    if case["op"] == "rope":
        t, d = case["tokens"], case["dim"]
        first = torch.randint(0, max(1, case["max_pos"] - t), (1,), device=DEV, generator=g)
        if t <= 256:  # tokens of different sequences
            pos = torch.randint(0, case["max_pos"], (t,), device=DEV, generator=g)
        else:
            pos = first + torch.arange(t, device=DEV)
        return {"case": case, "pos": pos.to(torch.int32), "q": randn(t, case["heads"], d).to(dtype),
                "k": randn(t, case["kv_heads"], d).to(dtype)}
    kv, new = _lengths(case)
    page, hkv, dim = case["page"], case["kv_heads"], case["dim"]
    counts = [max(1, -(-length // page)) for length in kv]
    total, width = sum(counts) + 3, max(counts)
    order = torch.randperm(total, device=DEV, generator=g).to(torch.int32)
    count = torch.tensor(counts, device=DEV)
    at = torch.arange(width, device=DEV)
    table = torch.where(at < count[:, None], order[((count.cumsum(0) - count)[:, None] + at).clamp(max=total - 1)], -1)
    s = {"case": case, "table": table.to(torch.int32).contiguous(), "kv_len": torch.tensor(kv, device=DEV, dtype=torch.int32),
         "cu_q": torch.tensor([0] + list(np.cumsum(new)), device=DEV, dtype=torch.int32),
         "n_tokens": sum(new), "max_q": max(new), "max_kv": max(kv)}
    s["k_codes"], s["k_scale"] = _pool(g, total, hkv, page, dim)
    s["v_codes"], s["v_scale"] = _pool(g, total, hkv, page, dim)
    if case["op"] == "write":
        s["k"] = (randn(s["n_tokens"], hkv, dim) * torch.exp(0.5 * randn(hkv, dim))).to(dtype)
        s["v"] = (randn(s["n_tokens"], hkv, dim) * torch.exp(0.5 * randn(hkv, dim))).to(dtype)
    if case["op"] == "attn":
        s["q"] = (1.2 * randn(s["n_tokens"], case["heads"], dim)).to(dtype)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "rope":
        f, s["amplitude"] = _frequencies(case)
        s["freq"] = torch.from_numpy(f).to(DEV)
    if own:
        import int4_routed_expert_gb300 as m
        if case["op"] == "rope":
            kind, factor, original = _scaling(case)
            s["rope"] = m.Rope(case["rot"], theta=THETA, interleaved=case["interleaved"], scaling=kind, factor=factor,
                               original_len=original)
        else:
            s["cache"] = m.KVCache(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"],
                                   n_q_heads=case.get("heads", case["kv_heads"]), max_seqs=case["seqs"],
                                   max_tokens=s["n_tokens"], max_kv_len=s["max_kv"])
            s["batch"] = m.SeqBatch(s["cu_q"], s["kv_len"], s["table"], s["n_tokens"], s["max_q"], s["max_kv"])
    return s


# -------------------------------------------------------------- the plain form

def _places(s):
    """Sequence, position, page and slot of each of the call's tokens."""
    t = torch.arange(s["n_tokens"], device=DEV)
    seq = torch.searchsorted(s["cu_q"].long(), t, right=True) - 1
    pos = s["kv_len"].long()[seq] - s["cu_q"].long()[seq + 1] + t
    page = s["table"].long()[seq, pos.clamp(min=0) // s["case"]["page"]]
    return seq, pos, page, pos % s["case"]["page"]


def _plain_rope(s):
    c = s["case"]
    rot = c["rot"]
    angle = s["pos"].double()[:, None] * s["freq"]
    cos = (torch.cos(angle) * s["amplitude"]).float()[:, None, :]
    sin = (torch.sin(angle) * s["amplitude"]).float()[:, None, :]

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


def _plain_write(s, x, codes, scales):
    page_size = s["case"]["page"]
    x = x.float()
    hkv = x.shape[1]
    _, _, page, slot = _places(s)
    new_max = torch.zeros_like(scales).scatter_reduce(0, page[:, None].expand(-1, hkv), x.abs().amax(-1), "amax")
    first = s["kv_len"].long() - (s["cu_q"][1:] - s["cu_q"][:-1]).long()  # each sequence's first new position
    begun = s["table"].long().gather(1, (first // page_size).clamp(max=s["table"].shape[1] - 1)[:, None])[:, 0]
    old = (first % page_size != 0)[:, None]  # whose page holds older tokens, with a scale of their own
    need = _block_scale(new_max)
    kept = torch.zeros_like(scales).index_put((begun.clamp(min=0),), torch.where(old, scales[begun], 0.0))
    scale = torch.maximum(need, kept)
    seen = torch.zeros(scales.shape[0], dtype=torch.bool, device=DEV).index_fill(0, page, True)[:, None]
    scale = torch.where(seen, scale, scales)
    ratio = torch.where(old, scales[begun] / scale[begun], 1.0)[..., None, None]
    ratio = torch.where(torch.arange(page_size, device=DEV)[:, None] < (first % page_size)[:, None, None, None], ratio, 1.0)
    codes[begun] = (codes[begun].float() * ratio).to(F8)
    codes[page, :, slot] = (x / scale[page][..., None]).to(F8)
    scales.copy_(scale)
    return codes, scales


def _plain_read(s, codes, scales):
    _, _, page, slot = _places(s)
    return (codes[page, :, slot].float() * scales[page][..., None]).to(TYPES[s["case"]["dtype"]])


def _plain_attend(s):
    c = s["case"]
    d, hkv, g = c["dim"], c["kv_heads"], c["heads"] // c["kv_heads"]
    b, n, width = s["kv_len"].numel(), s["max_q"], s["table"].shape[1]
    table = s["table"].long().clamp(min=0)

    def whole(codes, scales):  # [sequences][kv heads][tokens][dim]
        x = codes[table].float() * scales[table][..., None, None]
        return x.transpose(1, 2).reshape(b, hkv, width * c["page"], d)

    seq, pos, _, _ = _places(s)
    i = torch.arange(s["n_tokens"], device=DEV) - s["cu_q"].long()[seq]
    q = torch.zeros(b, n, c["heads"], d, device=DEV)
    q[seq, i] = s["q"].float()
    q = q.view(b, n, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, g * n, d)
    score = torch.matmul(q, whole(s["k_codes"], s["k_scale"]).transpose(2, 3)) * d ** -0.5
    p = torch.full((b, n), -1, device=DEV, dtype=torch.int64)
    p[seq, i] = pos
    j = torch.arange(width * c["page"], device=DEV)
    hidden = j > p[..., None]
    if c["window"]:
        hidden |= (j <= p[..., None] - c["window"]) & (j >= c["sinks"])
    score = score.view(b, hkv, g, n, -1).masked_fill_(hidden[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    e = torch.exp(score.sub_(top))
    del score
    o = torch.matmul(e.view(b, hkv, g * n, -1), whole(s["v_codes"], s["v_scale"])).view(b, hkv, g, n, d)
    o = o / e.sum(-1, keepdim=True).clamp(min=1e-30)
    return o.permute(0, 3, 1, 2, 4).reshape(b, n, c["heads"], d)[seq, i].to(s["q"].dtype)


def run(s):
    op = s["case"]["op"]
    if own:
        if op == "rope":
            return s["rope"].apply(s["q"], s["pos"], k=s["k"])
        if op == "write":
            s["cache"].write(s["k"], s["v"], s["batch"])
            return s["k_codes"], s["k_scale"], s["v_codes"], s["v_scale"]
        if op == "read":
            return s["cache"].read(s["batch"], dtype=TYPES[s["case"]["dtype"]])
        return s["cache"].attend(s["q"], s["batch"], window=s["case"]["window"], sinks=s["case"]["sinks"])
    if op == "rope":
        return _plain_rope(s)
    if op == "write":
        return (*_plain_write(s, s["k"], s["k_codes"], s["k_scale"]), *_plain_write(s, s["v"], s["v_codes"], s["v_scale"]))
    if op == "read":
        return _plain_read(s, s["k_codes"], s["k_scale"]), _plain_read(s, s["v_codes"], s["v_scale"])
    return _plain_attend(s)


# ------------------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "rope":
        f, amplitude = _frequencies(case)
        turn = torch.polar(torch.full((case["tokens"], case["rot"] // 2), amplitude, dtype=torch.float64, device=DEV),
                           torch.outer(s["pos"].double(), torch.from_numpy(f).to(DEV)))[:, None]
        out = []
        for x in (s["q"].double(), s["k"].double()):
            y, r = x.clone(), case["rot"]
            pick = (slice(0, r, 2), slice(1, r, 2)) if case["interleaved"] else (slice(0, r // 2), slice(r // 2, r))
            z = torch.complex(x[..., pick[0]].contiguous(), x[..., pick[1]].contiguous()) * turn
            y[..., pick[0]], y[..., pick[1]] = z.real, z.imag
            out.append(y)
        return tuple(out)
    kv, new, page = s["kv_len"].tolist(), (s["cu_q"][1:] - s["cu_q"][:-1]).tolist(), case["page"]
    table, cu = s["table"].tolist(), s["cu_q"].tolist()
    if case["op"] == "write":
        if sum(n // page + 2 for n in new) > 6000:
            return None
        out = []
        for x, codes, scales in ((s["k"], s["k_codes"], s["k_scale"]), (s["v"], s["v_codes"], s["v_scale"])):
            x, codes, scales = x.double(), codes.double(), scales.double()
            for b, (length, n) in enumerate(zip(kv, new)):
                t = length - n
                while t < length:  # one page after the other
                    at, p, end = t % page, table[b][t // page], min(length, (t // page + 1) * page)
                    rows = x[cu[b] + t - (length - n):cu[b] + end - (length - n)].transpose(0, 1)
                    amax = rows.abs().amax((1, 2))
                    need = torch.exp2(torch.ceil(torch.log2(amax / 448)).clamp(min=-63))
                    need = torch.where(amax <= 224 * need, need / 2, need)  # a logarithm just above a whole number
                    scale = torch.maximum(scales[p], need) if at else need
                    codes[p, :, :at] = (codes[p, :, :at] * (scales[p] / scale)[:, None, None]).to(F8).double()
                    codes[p, :, at:at + end - t] = (rows / scale[:, None, None]).to(F8).double()
                    scales[p] = scale
                    t = end
            out += [codes, scales]
        return tuple(out)

    def tokens(codes, scales, b, a, z):  # keys or values a..z of sequence b, [kv heads][z - a][dim]
        pages = torch.tensor(table[b][a // page:-(-z // page)], device=DEV, dtype=torch.int64)
        x = codes[pages].double() * scales[pages].double()[..., None, None]
        return x.transpose(0, 1).flatten(1, 2)[:, a % page:a % page + z - a]

    if case["op"] == "read":
        return tuple(torch.cat([tokens(c, x, b, length - n, length).transpose(0, 1) for b, (length, n) in enumerate(zip(kv, new))])
                     for c, x in ((s["k_codes"], s["k_scale"]), (s["v_codes"], s["v_scale"])))
    g = case["heads"] // case["kv_heads"]
    out = torch.zeros(s["n_tokens"], case["heads"], case["dim"], device=DEV, dtype=torch.float64)
    for b, (length, n) in enumerate(zip(kv, new)):
        if length == 0:
            continue
        k, v = tokens(s["k_codes"], s["k_scale"], b, 0, length), tokens(s["v_codes"], s["v_scale"], b, 0, length)
        j = torch.arange(length, device=DEV)
        for a in range(max(0, n - length), n, 1024):
            z = min(n, a + 1024)
            p = torch.arange(length - n + a, length - n + z, device=DEV)[:, None]
            sees = j <= p
            if case["window"]:
                sees &= (j > p - case["window"]) | (j < case["sinks"])
            for h in range(case["heads"]):
                q = s["q"][cu[b] + a:cu[b] + z, h].double()
                w = torch.softmax(torch.where(sees, q @ k[h // g].T / math.sqrt(case["dim"]), -math.inf), -1)
                out[cu[b] + a:cu[b] + z, h] = w @ v[h // g]
    return out
