"""Plain forms, in 64 bits, of the 4-bit cache, the attention over it and the
eviction by accumulated weight (torch tensors on any device)."""
from __future__ import annotations

import math

import torch

D, GROUP = 128, 32


def key_channel(nibble: int) -> int:
    """Channel held by nibble 0..127 of a key row: word 4c + g, channels 32g + 8c + e."""
    word, n = divmod(nibble, 8)
    c, g = divmod(word, 4)
    return 32 * g + 8 * c + (2 * n if n < 4 else 2 * n - 7)


def value_channel(nibble: int) -> int:
    """Of a value row: halfword 4r + g, channels 32g + 4r + i."""
    half, i = divmod(nibble, 4)
    r, g = divmod(half, 4)
    return 32 * g + 4 * r + i


KEY_ORDER = [key_channel(i) for i in range(D)]
VALUE_ORDER = [value_channel(i) for i in range(D)]


def quantise(x: torch.Tensor):
    """(codes c in [-7, 7], scales s) of bf16 rows, both float64; s = NaN, c = 0 for a group that is not finite."""
    v = x.double().unflatten(-1, (D // GROUP, GROUP))
    a = v.abs().amax(-1)
    fin = torch.isfinite(v).all(-1)
    # bf16 of the exact quotient: a has 8 significant bits, so a / 7 in float64 is on the same side of every bf16 midpoint
    s = torch.where(fin, (a / 7).to(torch.float32).to(torch.bfloat16).double(), math.nan)
    f = s[..., None]
    c = torch.where(f > 0, torch.round(v / torch.where(f > 0, f, 1.0)).clamp(-7, 7), 0.0)
    return c.flatten(-2), s


def values(c: torch.Tensor, s: torch.Tensor) -> torch.Tensor:
    return (c.unflatten(-1, (D // GROUP, GROUP)) * s[..., None]).flatten(-2)


def pack(c: torch.Tensor, order) -> torch.Tensor:
    n = (c[..., torch.tensor(order, device=c.device)] + 8).to(torch.uint8)
    return n[..., 0::2] + 16 * n[..., 1::2]


def unpack(codes: torch.Tensor, order) -> torch.Tensor:
    n = torch.stack((codes % 16, codes // 16), -1).flatten(-2).double() - 8
    out = torch.empty_like(n)
    out[..., torch.tensor(order, device=codes.device)] = n
    return out


def to_pool(rows: torch.Tensor, table: torch.Tensor, bs: int, pool: torch.Tensor) -> None:
    """Logical rows [B, Hkv, cap, w] into the pages [num_pages, Hkv, bs, w] of a table [B, nb]."""
    B, _, cap, _ = rows.shape
    for b in range(B):
        for i in range(-(-cap // bs)):
            n = min(bs, cap - i * bs)
            pool[table[b, i], :, :n] = rows[b, :, i * bs: i * bs + n]


def from_pool(pool: torch.Tensor, table: torch.Tensor, cap: int) -> torch.Tensor:
    x = pool[table.long()]                     # [B, nb, Hkv, bs, w]
    return x.transpose(1, 2).flatten(2, 3)[:, :, :cap]


def block_means(rows: torch.Tensor, lens, bs: int) -> torch.Tensor:
    """fp32 sums in token order of fp32 rows [B, Hkv, cap, D], divided by the count; NaN where a block is empty."""
    B, Hkv, cap, _ = rows.shape
    nb = -(-cap // bs)
    out = torch.full((B, Hkv, nb, D), math.nan, dtype=torch.float32, device=rows.device)
    for b, n in enumerate(lens):
        for i in range(-(-n // bs)):
            t0, t1 = i * bs, min((i + 1) * bs, n)
            acc = torch.zeros((Hkv, D), dtype=torch.float32, device=rows.device)
            for t in range(t0, t1):
                acc = acc + rows[b, :, t]
            # a tensor as divisor: on a GPU torch multiplies by a scalar's reciprocal
            out[b, :, i] = acc / torch.full_like(acc, t1 - t0)
    return out


def attend(q, k, v, lens, sel, scale, bs):
    """(out, lse, w, spread) in float64.  q [B, Hq, D], k / v values [B, Hkv,
    cap, D], sel: a list per (b, h) of kept blocks, or None.  w [B, Hkv, cap]:
    each token's weight summed over the group; spread [B, Hq, D]: sum_t p |v|."""
    B, Hq, _ = q.shape
    Hkv, cap = k.shape[1], k.shape[2]
    g = Hq // Hkv
    out = torch.zeros((B, Hq, D), dtype=torch.float64, device=q.device)
    spread = torch.zeros_like(out)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device=q.device)
    w = torch.zeros((B, Hkv, cap), dtype=torch.float64, device=q.device)
    for b, n in enumerate(lens):
        for h in range(Hkv):
            blocks = range(-(-n // bs)) if sel is None else [i for i in sel[b][h] if i >= 0]
            tok = [t for i in blocks for t in range(i * bs, min((i + 1) * bs, n))]
            if not tok:
                continue
            tok = torch.tensor(tok, device=q.device)
            z = scale * q[b, h * g:(h + 1) * g].double() @ k[b, h, tok].double().T
            l = torch.logsumexp(z, -1)
            p = torch.exp(z - l[:, None])
            out[b, h * g:(h + 1) * g] = p @ v[b, h, tok].double()
            spread[b, h * g:(h + 1) * g] = p @ v[b, h, tok].double().abs()
            lse[b, h * g:(h + 1) * g] = l
            w[b, h].index_add_(0, tok, p.sum(0))
    return out, lse, w, spread


def kept(acc, n: int, n_keep: int, n_sink: int, n_recent: int):
    """The kept tokens of one pair, ascending, by sorting (acc: a list of floats)."""
    if n <= n_keep:
        return list(range(n))
    lo, hi = n_sink, n - n_recent

    def rank(t):  # NaN last
        return (1, 0.0, t) if acc[t] != acc[t] else (0, -acc[t], t)

    best = sorted(range(lo, hi), key=rank)[: n_keep - n_sink - n_recent]
    return sorted(list(range(lo)) + list(range(hi, n)) + best)
