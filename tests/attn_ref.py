"""64-bit references of the attention-side operators, from their definitions (one token or one row at a time)."""
from __future__ import annotations

import math
import random

import torch

F8 = torch.float8_e4m3fn


def pow2_scale(amax: float) -> float:
    """Smallest power of two s >= 2^-64 with amax <= 448 s."""
    s = 2.0 ** -64
    while amax > 448 * s:
        s *= 2
    return s


def rope(x, positions, inv_freq, amplitude, interleaved):
    """x [T, H, D] -> float64, pair by pair."""
    y = x.double().clone()
    rot = 2 * len(inv_freq)
    f = torch.tensor(inv_freq, dtype=torch.float64, device=x.device)
    a = positions.double()[:, None, None] * f
    c, s = amplitude * torch.cos(a), amplitude * torch.sin(a)
    if interleaved:
        u, v = x.double()[..., 0:rot:2], x.double()[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = u * c - v * s, u * s + v * c
    else:
        u, v = x.double()[..., :rot // 2], x.double()[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = u * c - v * s, u * s + v * c
    return y


class Batch:
    """Lengths, new-token counts and shuffled pages of a batch, and its SeqBatch."""

    def __init__(self, lens, news, page, dev, seed=0, spare=2, base=0, pool=None, slack=0):
        import int4_routed_expert_gb300 as m
        self.lens, self.news, self.page = lens, news, page
        r = random.Random(seed)
        need = [max(1, -(-n // page)) for n in lens]
        ids = [base + i for i in range(sum(need) + spare)]
        r.shuffle(ids)
        width = max(need) + slack
        self.table, at = [], 0
        for n in need:
            self.table.append(ids[at:at + n] + [-1] * (width - n))
            at += n
        self.n_pages = pool or (base + sum(need) + spare)
        self.cu = [0]
        for n in news:
            self.cu.append(self.cu[-1] + n)
        i32 = dict(dtype=torch.int32, device=dev)
        self.b = m.SeqBatch(torch.tensor(self.cu, **i32), torch.tensor(lens, **i32), torch.tensor(self.table, **i32),
                            self.cu[-1], max(max(news), 1), max(max(lens), 1))

    def places(self):
        """(row, sequence, position) of every token of the call at a position >= 0."""
        for b, (length, n) in enumerate(zip(self.lens, self.news)):
            for i in range(n):
                if length - n + i >= 0:
                    yield self.cu[b] + i, b, length - n + i


def tokens(codes, scales, bt, b, length):
    """Sequence b's first `length` tokens as float64 [kv heads, length, D]."""
    n = -(-length // bt.page)
    p = torch.tensor(bt.table[b][:n], device=codes.device, dtype=torch.int64)
    x = codes.view(F8)[p].double() * scales[p].double()[..., None, None]
    return x.transpose(0, 1).flatten(1, 2)[:, :length]


def attend(q, k_codes, v_codes, k_scale, v_scale, bt, scale, causal=True, window=0, sinks=0):
    """(out, lse, tolerance) in float64: the row's softmax over what it sees.

    The tolerance of an output counts the roundings of the computation: half a step of bf16 on the result
    (2^-8), half a step of f16 on each weight (2^-11), and what the logits may be off: each of the D products'
    sums in fp32, up to 2^-22 of the sum of magnitudes a step, moves a weight by its relative size, in the
    numerator and in the denominator; 2^-18 for exponentials, logarithms and fp32 sums.  Weights (the block's
    value scale in them) are f16 relative to 2^-10 of the row's largest, so below 2^-24 of that their step is
    2^-24: half of it on each code the row sees."""
    T, H, D = q.shape
    g = H // k_codes.shape[1]
    out = torch.zeros(T, H, D, dtype=torch.float64, device=q.device)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device=q.device)
    tol = torch.full((T, H, D), 1e-37, dtype=torch.float64, device=q.device)
    for b, (length, n) in enumerate(zip(bt.lens, bt.news)):
        if length == 0 or n == 0:
            continue
        k, v = tokens(k_codes, k_scale, bt, b, length), tokens(v_codes, v_scale, bt, b, length)
        code = tokens(v_codes, torch.ones_like(v_scale), bt, b, length).nan_to_num()
        block = tokens(torch.full_like(v_codes.view(torch.uint8), 0x38), v_scale, bt, b, length)[..., 0]  # 0x38 is 1
        p = torch.arange(length - n, length, device=q.device)[:, None]
        j = torch.arange(length, device=q.device)[None]
        sees = (j <= p) if causal else torch.ones_like(j <= p)
        if causal and window:
            sees = sees & ((j > p - window) | (j < sinks))
        any_ = sees.any(1)
        for h in range(H):
            x = q[bt.cu[b]:bt.cu[b] + n, h].double()
            kk, vv = k[h // g].nan_to_num(), v[h // g].nan_to_num()
            s = torch.where(sees, x @ kk.T * scale, -math.inf)
            off = torch.where(sees, x.abs() @ kk.abs().T * abs(scale), 0.0).amax(1) * D * 2.0 ** -22
            top = s.amax(1, keepdim=True)
            w = torch.exp(s - torch.where(any_[:, None], top, 0.0))
            den = w.sum(1, keepdim=True)
            w = torch.where(any_[:, None], w / den, 0.0)
            rows = slice(bt.cu[b], bt.cu[b] + n)
            out[rows, h] = w @ vv
            lse[rows, h] = torch.where(any_, top[:, 0] + torch.log(den[:, 0]), -math.inf)
            spread = w @ vv.abs()
            step = 2.0 ** -35 * (w * block[h // g].nan_to_num()).amax(1)
            tol[rows, h] += step[:, None] * (sees.double() @ code[h // g].abs())
            tol[rows, h] += 2.0 ** -8 * out[rows, h].abs() + (2.0 ** -11 + 2.0 ** -18 + 2 * off)[:, None] * spread * 1.01
    return out, lse, tol


def write(x, codes, scales, bt):
    """The cache's write, one page at a time, on float64 copies of (code values, scales)."""
    x, codes, scales = x.double(), codes.view(F8).double(), scales.double().clone()
    for b, (length, n) in enumerate(zip(bt.lens, bt.news)):
        first = max(length - n, 0)
        t = first
        while t < length:
            end = min(length, (t // bt.page + 1) * bt.page)
            page, at = bt.table[b][t // bt.page], t % bt.page
            r = bt.cu[b] + t - (length - n)
            for h in range(codes.shape[1]):
                rows = x[r:r + end - t, h]
                fin = rows[rows.isfinite()]
                need = pow2_scale(float(fin.abs().max()) if fin.numel() else 0.0)
                s = max(float(scales[page, h]), need) if at else need
                if at:
                    codes[page, h, :at] = (codes[page, h, :at] * (float(scales[page, h]) / s)).to(F8).double()
                y = (rows / s).clamp(-448, 448)
                codes[page, h, at:at + end - t] = torch.where(y.isnan(), 0.0, y).to(F8).double()
                scales[page, h] = s
            t = end
    return codes, scales
