"""Measured cases of the KV-cache operators: the cache held in 4 bits (store,
read back, append, attend) and the eviction by accumulated attention weight
(attention that accumulates the weights, the eviction itself).

The 4-bit cache.  A row is one token's key or value of one KV head, D = 128
channels.  Every group of 32 channels of a row holds
    a = max |x|,  s = bf16(a / 7),  c = clamp(round_half_even(x / s), -7, 7)
(c = 0 where s = 0; s = NaN and c = 0 where the group holds NaN or an
infinity) and stands for c s.  A row's codes are 64 bytes, each code as the
nibble c + 8, low nibble first, in one order of the channels for keys
(K_ORDER) and one for values (V_ORDER); its scales are 4 bf16.  A block's
mean key is the fp32 mean of the values held.

Attention reads the tokens of the kept blocks (or of every block):
    z = q K^T / sqrt(D),  out = softmax(z) V,  lse = log sum exp z,
and, where weights are accumulated, acc[b, h, t] += sum_j exp(z_jt - lse_j)
over the query heads j of KV head h.  The eviction keeps the first n_sink and
the last n_recent tokens and the best of the rest by acc (ties to the lower
index), n_keep in all, and moves them, in order, to another cache.
"""
import math

import torch

own = False

D = 128
GROUP = 32


def _k_order():
    """Channel of each of a key row's 128 nibbles (byte by byte, low nibble
    first): word 4 c + g holds channels 32 g + 8 c + e, e even in nibbles
    0..3, e odd in nibbles 4..7."""
    order = []
    for word in range(16):
        c, g = word // 4, word % 4
        for nib in range(8):
            order.append(32 * g + 8 * c + (2 * nib if nib < 4 else 2 * (nib - 4) + 1))
    return order


def _v_order():
    """The same for a value row: halfword 4 r + g holds channels 32 g + 4 r + i, i = 0..3."""
    order = []
    for half in range(32):
        r, g = half // 4, half % 4
        order += [32 * g + 4 * r + i for i in range(4)]
    return order


K_ORDER, V_ORDER = _k_order(), _v_order()


def _orders(dev):
    """Both orders on the device, as a program keeps them: a row's channels nibble by nibble, and the other way round."""
    o = {}
    for name, order in (("k", K_ORDER), ("v", V_ORDER)):
        o[name] = torch.tensor(order, device=dev)
        o[name + "_at"] = o[name].argsort()
    return o


# ------------------------------------------------------------------ cases

def _case(name, op, B, Hkv, Hq, bs, lmin, lmax, cap, **more):
    c = {"name": name, "op": op, "B": B, "Hkv": Hkv, "Hq": Hq, "bs": bs, "lmin": lmin, "lmax": lmax, "cap": cap,
         "paged": False, "int4": True, "k": 0, "acc": False, "n_new": 0, "n_keep": 0, "n_sink": 0, "n_recent": 0,
         "means_bf16": False}
    c.update(more)
    return c


def listed():
    return [
        # a prefilled 32K batch put into 4 bits and read back
        _case("store_32k", "store", 4, 8, 32, 16, 32768, 32768, 32768),
        # a few short ragged prompts in a page pool, some of a single token
        _case("store_ragged_paged", "store", 5, 8, 40, 32, 1, 701, 768, paged=True, means_bf16=True),
        # the append of one decode step of a batch of 32
        _case("append_1", "append", 32, 8, 32, 16, 4001, 8000, 8192, n_new=1),
        # a chunk of a prompt appended to caches of ragged lengths, ending inside a block
        _case("append_333_paged", "append", 4, 8, 64, 32, 0, 2000, 2400, n_new=333, paged=True),
        # the smallest decode call: one sequence, one KV head
        _case("attn4_tiny", "attn", 1, 1, 4, 16, 4096, 4096, 4096, k=32),
        # decode attention of a batch of 32 at 32K, 256 of 2048 blocks kept
        _case("attn4_32k", "attn", 32, 8, 32, 16, 32768, 32768, 32768, k=256),
        # ragged 8K-32K paged batch, weights accumulated as an evicting server does
        _case("attn4_ragged_paged_acc", "attn", 64, 8, 40, 16, 8192, 32768, 32768, k=128, paged=True, acc=True),
        # a bf16 cache: sparse decode attention of a 32K batch with accumulated weights
        _case("attn_acc_32k", "attn", 32, 8, 32, 16, 32768, 32768, 32768, k=256, int4=False, acc=True),
        # every token of short ragged caches (a cache that eviction keeps short is read whole)
        _case("attn_acc_dense", "attn", 8, 8, 16, 32, 900, 2100, 2112, int4=False, acc=True),
        # one sequence of 8 heads halved
        _case("evict_small", "evict", 1, 8, 32, 16, 2047, 2047, 2048, int4=False, n_keep=1024, n_sink=4, n_recent=256),
        # a 32K batch cut to 4096 tokens a head
        _case("evict_32k", "evict", 16, 8, 32, 16, 32768, 32768, 32768, int4=False, n_keep=4096, n_sink=16, n_recent=512),
        # a ragged 4-bit paged batch, one sequence below the budget
        _case("evict4_ragged_paged", "evict", 24, 8, 40, 32, 1500, 16001, 16384, n_keep=2001, n_sink=1, n_recent=130,
              paged=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["store", "append", "attn", "attn", "attn", "evict", "evict"])
    Hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 5, 8])
    bs = rng.choice([16, 32, 64, 128])
    int4 = True if op in ("store", "append") else rng.random() < 0.5
    # tokens over all sequences and KV heads, at most what the largest listed case of the kind holds
    B = _log_int(rng, 1, 32 if op != "attn" else 64)
    lmax = _log_int(rng, 1, 32768)
    most = {"store": 1 << 20, "append": 1 << 20, "attn": 1 << 23, "evict": 1 << 22}[op]
    lmax = max(1, min(lmax, most // (B * Hkv)))
    lmin = lmax if rng.random() < 0.3 else _log_int(rng, 1, lmax)
    more = {"paged": rng.random() < 0.5, "int4": int4, "means_bf16": rng.random() < 0.3}
    cap = lmax + rng.choice([0, 1, 17, 100])
    if op == "append":
        more["n_new"] = _log_int(rng, 1, 512)
        lmin = rng.choice([0, lmin])
        cap = lmax + more["n_new"] + rng.choice([0, 5])
    elif op == "attn":
        nb = -(-cap // bs)
        # every block where that stays small, else at most 1M kept tokens
        most_k = max(2, (1 << 20) // (B * Hkv * bs))
        dense = rng.random() < 0.25 and nb <= most_k
        more["k"] = 0 if dense else _log_int(rng, 2, max(2, min(nb, most_k)))
        more["acc"] = (not int4) or rng.random() < 0.5
    elif op == "evict":
        most_keep = max(1, min(lmax, (1 << 19) // (B * Hkv)))
        more["n_keep"] = _log_int(rng, 1, most_keep)
        more["n_sink"] = rng.randint(0, min(more["n_keep"], 16))
        more["n_recent"] = rng.randint(0, (more["n_keep"] - more["n_sink"]) // 2)
    c = _case("drawn", op, B, Hkv, g * Hkv, bs, lmin, lmax, cap, **more)
    del c["name"]
    return c


def _lens(c):
    """The sequence lengths before the call: spread evenly over [lmin, lmax]."""
    if c["B"] == 1:
        return [c["lmax"]]
    return [c["lmin"] + (c["lmax"] - c["lmin"]) * i // (c["B"] - 1) for i in range(c["B"])]


def _row_bytes(c):
    return 2 * (64 + 8) if c["int4"] else 2 * 2 * D


def work(c):
    lens, Hkv, bs = _lens(c), c["Hkv"], c["bs"]
    pairs = c["B"] * Hkv
    mean_bytes = D * (2 if c["means_bf16"] else 4)
    if c["op"] == "store":
        rows = Hkv * sum(lens)
        blocks = Hkv * sum(-(-n // bs) for n in lens)
        # the bf16 rows in, the codes and scales, the means; the rows read back (zero past each length)
        return {"bytes": rows * (4 * D + 144) + blocks * mean_bytes + pairs * c["cap"] * 4 * D, "flops": rows * 4 * D}
    if c["op"] == "append":
        n = c["n_new"]
        rows = pairs * n
        old = Hkv * sum(m % bs for m in lens)  # rows of partial blocks whose means change
        blocks = Hkv * sum((m + n - 1) // bs - m // bs + 1 for m in lens)
        return {"bytes": rows * (2 * 4 * D + 144) + old * 72 + blocks * mean_bytes, "flops": rows * 4 * D}
    if c["op"] == "attn":
        kept = 0
        for m in lens:
            nb = -(-m // bs)
            kept += m if c["k"] == 0 or c["k"] >= nb else (c["k"] - 1) * bs + m - (nb - 1) * bs
        kept *= Hkv
        ends = c["B"] * c["Hq"] * (4 * D + 4) + (0 if c["k"] == 0 else pairs * (c["k"] * 4 + 4))
        return {"bytes": kept * (_row_bytes(c) + (8 if c["acc"] else 0)) + ends,
                "flops": kept * (c["Hq"] // Hkv) * 4 * D}
    keep = [min(m, c["n_keep"]) for m in lens]
    blocks = Hkv * sum(-(-m // bs) for m in keep)
    rows = Hkv * sum(keep)
    back = rows * 4 * D if c["int4"] else 0  # the rows of the 4-bit cache read back
    cap = _dst_cap(c)
    return {"bytes": Hkv * sum(lens) * 4 + rows * 2 * _row_bytes(c) + back + blocks * mean_bytes
            + pairs * (cap + c["n_keep"]) * 4, "flops": rows * D}


def _dst_cap(c):
    """The capacity of the cache that the kept tokens move to: room for one more block of new ones."""
    return min(c["n_keep"], c["cap"]) + c["bs"]


# ----------------------------------------------------------- the 4-bit rows

def _quantise(x):
    """Codes c (int8) and scales (bf16, [..., 4]) of rows x ([..., 128] bf16)."""
    v = x.float().unflatten(-1, (D // GROUP, GROUP))
    a = v.abs().amax(-1)
    s = torch.where(torch.isfinite(a), a / 7, torch.full_like(a, math.nan)).to(torch.bfloat16)
    f = s.float()[..., None]
    c = torch.where(f > 0, torch.round(v / f).clamp(-7, 7), torch.zeros_like(v))
    return c.to(torch.int8).flatten(-2), s


def _pack(c, order):
    n = (c[..., order] + 8).to(torch.uint8)
    return n[..., 0::2] | (n[..., 1::2] << 4)


def _unpack(codes, at):
    n = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    return n[..., at].float() - 8


def _values(codes, scales, at):
    """The values of 4-bit rows, in fp32 (each is exact); at: the nibble of each channel."""
    return (_unpack(codes, at).unflatten(-1, (D // GROUP, GROUP)) * scales.float()[..., None]).flatten(-2)


# ------------------------------------------------------------------- state

def _gen(seed, dev):
    return torch.Generator(device=dev).manual_seed(seed)


def _rows_kv(c, cap, g, dev, heavy=True):
    """K and V rows [B, Hkv, cap, D] in bf16: standard normal, with a bias of
    deviation 2 on the keys of about 5% of the blocks (heavy hitters)."""
    B, Hkv, bs = c["B"], c["Hkv"], c["bs"]
    k = torch.randn((B, Hkv, cap, D), generator=g, device=dev, dtype=torch.bfloat16)
    v = torch.randn((B, Hkv, cap, D), generator=g, device=dev, dtype=torch.bfloat16)
    if heavy:
        beta = 2 * torch.randn((B, Hkv, 1, D), generator=g, device=dev, dtype=torch.bfloat16)
        hit = torch.rand((B, Hkv, -(-cap // bs)), generator=g, device=dev) < 0.05
        k += beta * hit.repeat_interleave(bs, 2)[:, :, :cap, None]
    return k, v


def _table(c, cap, g, dev):
    """A page table [B, ceil(cap / bs)] over a pool of that many pages, in random order."""
    nb = -(-cap // c["bs"])
    return torch.randperm(c["B"] * nb, generator=g, device=dev).to(torch.int32).view(c["B"], nb)


def _row_ids(c, cap, table, tokens):
    """Rows, in the flat cache or pool, of tokens [B, Hkv, n] (int64)."""
    B, Hkv, bs = c["B"], c["Hkv"], c["bs"]
    dev = tokens.device
    b = torch.arange(B, device=dev)[:, None, None]
    h = torch.arange(Hkv, device=dev)[None, :, None]
    if table is None:
        return (b * Hkv + h) * cap + tokens
    return (table[b, tokens // bs].long() * Hkv + h) * bs + tokens % bs


def _into(c, cap, table, rows):
    """Logical rows [B, Hkv, cap, w] as the cache that holds them: the same, or the pages of a pool."""
    if table is None:
        return rows.contiguous()
    B, Hkv, bs = c["B"], c["Hkv"], c["bs"]
    nb = -(-cap // bs)
    pool = torch.zeros((B * nb, Hkv, bs, rows.shape[-1]), dtype=rows.dtype, device=rows.device)
    at = _row_ids(c, cap, table, torch.arange(cap, device=rows.device).expand(B, Hkv, cap))
    pool.view(-1, rows.shape[-1])[at.flatten()] = rows.reshape(-1, rows.shape[-1])
    return pool


def _like_cache(c, cap, table, width, dtype, dev):
    B, Hkv, bs = c["B"], c["Hkv"], c["bs"]
    shape = (B, Hkv, cap, width) if table is None else (table.numel(), Hkv, bs, width)
    return torch.zeros(shape, dtype=dtype, device=dev)


def _block_means(c, cap, lens, values):
    """Mean key of every block below each length ([B, Hkv, nb, D], fp32; 0 beyond) of values [B, Hkv, cap, D]."""
    bs = c["bs"]
    nb = -(-cap // bs)
    t = torch.arange(cap, device=values.device)
    x = torch.where((t < lens[:, None])[:, None, :, None], values, torch.zeros_like(values))
    x = torch.nn.functional.pad(x, (0, 0, 0, nb * bs - cap)).unflatten(2, (nb, bs)).sum(3)
    count = (lens[:, None] - torch.arange(nb, device=values.device) * bs).clamp(0, bs)[:, None, :, None]
    return torch.where(count > 0, x / count.clamp(min=1), torch.zeros_like(x))


def _select(c, lens, q, kmean):
    """The blocks that a decode step keeps: the k best by group score, the first and the newest among them."""
    B, Hkv, bs, k = c["B"], c["Hkv"], c["bs"], c["k"]
    nb = kmean.shape[2]
    score = (q.float().view(B, Hkv, -1, D).sum(2)[:, :, None] * kmean).sum(-1)
    mine = (lens + bs - 1) // bs
    i = torch.arange(nb, device=q.device)
    score = torch.where(i < mine[:, None, None], score, -math.inf)
    score = torch.where((i == 0) | (i == mine[:, None, None] - 1), math.inf, score)
    if k > nb:
        score = torch.nn.functional.pad(score, (0, k - nb), value=-math.inf)
    top, idx = score.sort(dim=-1, descending=True, stable=True)
    gone = top[..., :k] == -math.inf
    sel = torch.where(gone, 1 << 30, idx[..., :k]).sort(-1).values
    cnt = (~gone).sum(-1).to(torch.int32)
    return torch.where(sel == 1 << 30, -1, sel).to(torch.int32).contiguous(), cnt.contiguous()


def prepare(c, seed):
    dev = torch.device("cuda")
    g = _gen(seed, dev)
    B, Hkv, Hq, bs, cap = c["B"], c["Hkv"], c["Hq"], c["bs"], c["cap"]
    nb = -(-cap // bs)
    lens = torch.tensor(_lens(c), dtype=torch.int32, device=dev)
    table = _table(c, cap, g, dev) if c["paged"] else None
    mean_t = torch.bfloat16 if c["means_bf16"] else torch.float32
    s = {"case": c, "lens": lens, "table": table, "order": _orders(dev)}
    k, v = _rows_kv(c, cap, g, dev)
    if c["op"] == "store":
        s["k"], s["v"] = _into(c, cap, table, k), _into(c, cap, table, v)
    elif c["int4"]:
        kc, s["ks"] = _quantise(k)
        vc, s["vs"] = _quantise(v)
        if c["op"] == "append":
            s["means"] = _block_means(c, cap, lens, (kc.float().unflatten(-1, (4, 32)) * s["ks"].float()[..., None]).flatten(-2)).to(mean_t)
        s["k"], s["v"] = _into(c, cap, table, _pack(kc, s["order"]["k"])), _into(c, cap, table, _pack(vc, s["order"]["v"]))
        s["ks"], s["vs"] = _into(c, cap, table, s["ks"]), _into(c, cap, table, s["vs"])
    else:
        s["k"], s["v"] = _into(c, cap, table, k), _into(c, cap, table, v)
    if c["op"] == "store":
        for n, w, t in (("k4", 64, torch.uint8), ("v4", 64, torch.uint8), ("ks", 4, torch.bfloat16), ("vs", 4, torch.bfloat16)):
            s[n] = _like_cache(c, cap, table, w, t, dev)
        s["means"] = torch.zeros((B, Hkv, nb, D), dtype=mean_t, device=dev)
        s["k_back"] = torch.zeros((B, Hkv, cap, D), dtype=torch.bfloat16, device=dev)
        s["v_back"] = torch.zeros_like(s["k_back"])
    elif c["op"] == "append":
        n = c["n_new"]
        s["k_new"], s["v_new"] = _rows_kv(c, n, g, dev)
        s["new_lens"] = torch.zeros_like(lens)
        s["k_back"] = torch.zeros((B, Hkv, n, D), dtype=torch.bfloat16, device=dev)
        s["v_back"] = torch.zeros_like(s["k_back"])
    elif c["op"] == "attn":
        s["q"] = torch.randn((B, Hq, D), generator=g, device=dev, dtype=torch.bfloat16)
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros((B, Hq), device=dev)
        s["acc"] = None
        if c["acc"]:  # as after some hundred steps: most tokens light, some heavy
            s["acc"] = torch.rand((B, Hkv, cap), generator=g, device=dev).pow_(8).mul_(Hq // Hkv)
        s["sel"] = s["cnt"] = None
        if c["k"]:
            s["sel"], s["cnt"] = _select(c, lens, s["q"], _block_means(c, cap, lens, k.float()))
    else:
        cap2 = _dst_cap(c)
        t2 = _table(c, cap2, g, dev) if c["paged"] else None
        s["acc"] = torch.rand((B, Hkv, cap), generator=g, device=dev).pow_(8).mul_(Hq // Hkv)
        # equal weights are common (tokens that no step has kept weigh nothing)
        s["acc"] *= torch.rand((B, Hkv, cap), generator=g, device=dev) < 0.7
        s["table2"] = t2
        w, t = (64, torch.uint8) if c["int4"] else (D, torch.bfloat16)
        s["k2"], s["v2"] = _like_cache(c, cap2, t2, w, t, dev), _like_cache(c, cap2, t2, w, t, dev)
        s["ks2"] = s["vs2"] = None
        if c["int4"]:
            s["ks2"], s["vs2"] = (_like_cache(c, cap2, t2, 4, torch.bfloat16, dev) for _ in range(2))
            s["k_back"] = torch.zeros((B, Hkv, cap2, D), dtype=torch.bfloat16, device=dev)
            s["v_back"] = torch.zeros_like(s["k_back"])
        s["acc2"] = torch.zeros((B, Hkv, cap2), device=dev)
        s["lens2"] = torch.zeros_like(lens)
        s["sel"] = torch.zeros((B, Hkv, c["n_keep"]), dtype=torch.int32, device=dev)
        s["means"] = torch.zeros((B, Hkv, -(-cap2 // bs), D), dtype=mean_t, device=dev)
    _plan(s)
    return s


def _plan(s):
    """What a program keeps beside its tensors: the framework's dims, cache handles and workspace."""
    if not own:
        return
    import block_top_sparse_kin_b200 as kin

    c = s["case"]
    s["dims"] = kin.make_dims(c["B"], c["Hkv"], c["Hq"], D, c["bs"], c["cap"])
    if c["op"] == "store":
        s["src"] = kin.KvCache(s["k"], s["v"], block_table=s["table"])
        s["kv"] = kin.KvCache(s["k4"], s["v4"], s["ks"], s["vs"], block_table=s["table"])
    else:
        s["kv"] = kin.KvCache(s["k"], s["v"], s.get("ks"), s.get("vs"), block_table=s["table"])
    if c["op"] == "attn":
        s["ws"] = kin.alloc_kv_attn_workspace(s["dims"], c["k"], acc=c["acc"])
    if c["op"] == "evict":
        s["dims2"] = kin.make_dims(c["B"], c["Hkv"], c["Hq"], D, c["bs"], _dst_cap(c))
        s["kv2"] = kin.KvCache(s["k2"], s["v2"], s["ks2"], s["vs2"], block_table=s["table2"])
        s["ws"] = kin.alloc_kv_evict_workspace(s["dims"], c["n_keep"])


# --------------------------------------------------------------------- run

def run(s):
    return {"store": _run_store, "append": _run_append, "attn": _run_attn, "evict": _run_evict}[s["case"]["op"]](s)


def _run_store(s):
    c = s["case"]
    if own:
        import block_top_sparse_kin_b200 as kin

        kin.kin_kv4_store(s["dims"], s["src"], s["kv"], s["lens"], s["means"])
        kin.kin_kv4_load(s["dims"], s["kv"], s["lens"], s["k_back"], s["v_back"])
        return {"k": s["k_back"], "v": s["v_back"], "means": s["means"]}
    B, Hkv, cap = c["B"], c["Hkv"], c["cap"]
    lens = s["lens"]
    t = torch.arange(cap, device=lens.device).expand(B, Hkv, cap)
    at = _row_ids(c, cap, s["table"], t).flatten()
    live = (t < lens[:, None, None])[..., None]
    kc, ks = _quantise(s["k"].view(-1, D)[at])
    vc, vs = _quantise(s["v"].view(-1, D)[at])
    s["k4"].view(-1, 64)[at], s["ks"].view(-1, 4)[at] = _pack(kc, s["order"]["k"]), ks
    s["v4"].view(-1, 64)[at], s["vs"].view(-1, 4)[at] = _pack(vc, s["order"]["v"]), vs
    k = (kc.float().unflatten(-1, (4, GROUP)) * ks.float()[..., None]).view(B, Hkv, cap, D)
    v = (vc.float().unflatten(-1, (4, GROUP)) * vs.float()[..., None]).view(B, Hkv, cap, D)
    means = _block_means(c, cap, lens, k)
    s["means"].copy_(means)
    s["k_back"].copy_(torch.where(live, k, torch.zeros_like(k)))
    s["v_back"].copy_(torch.where(live, v, torch.zeros_like(v)))
    return {"k": s["k_back"], "v": s["v_back"], "means": s["means"]}


def _run_append(s):
    c = s["case"]
    n = c["n_new"]
    if own:
        import block_top_sparse_kin_b200 as kin

        kin.kin_kv4_append(s["dims"], s["kv"], s["means"], s["lens"], s["new_lens"], s["k_new"], s["v_new"], n)
        kin.kin_kv4_load(s["dims"], s["kv"], s["new_lens"], s["k_back"], s["v_back"], starts=s["lens"])
        return {"k": s["k_back"], "v": s["v_back"], "means": s["means"], "lens": s["new_lens"]}
    B, Hkv, cap, bs = c["B"], c["Hkv"], c["cap"], c["bs"]
    lens = s["lens"]
    dev = lens.device
    t = (lens[:, None, None].long() + torch.arange(n, device=dev)).expand(B, Hkv, n)
    at = _row_ids(c, cap, s["table"], t)
    kc, ks = _quantise(s["k_new"])
    vc, vs = _quantise(s["v_new"])
    s["k"].view(-1, 64)[at], s["ks"].view(-1, 4)[at] = _pack(kc, s["order"]["k"]), ks
    s["v"].view(-1, 64)[at], s["vs"].view(-1, 4)[at] = _pack(vc, s["order"]["v"]), vs
    s["new_lens"].copy_(lens + n)
    # the touched blocks' means, from their held rows
    span = (n + bs - 2) // bs + 1  # blocks that n rows can touch
    blk = (lens[:, None].long() // bs + torch.arange(span, device=dev)).expand(B, span)
    tok = (blk[..., None] * bs + torch.arange(bs, device=dev)).view(B, 1, -1)
    live = tok < s["new_lens"][:, None, None]
    rows = _row_ids(c, cap, s["table"], torch.where(live, tok, 0).expand(B, Hkv, -1))
    x = _values(s["k"].view(-1, 64)[rows], s["ks"].view(-1, 4)[rows], s["order"]["k_at"]) * live[..., None]
    x = x.unflatten(2, (span, bs)).sum(3)
    count = live.view(B, 1, span, bs).sum(-1)[..., None]
    mean = (x / count.clamp(min=1)).to(s["means"].dtype)
    # a span past the last touched block writes the first one's mean once more
    touched = count > 0
    mean = torch.where(touched, mean, mean[:, :, :1])
    to = torch.where(touched[:, 0, :, 0], blk, blk[:, :1])[:, None]
    pair = torch.arange(B * Hkv, device=dev).view(B, Hkv, 1)
    s["means"].view(-1, D)[(pair * s["means"].shape[2] + to).flatten()] = mean.reshape(-1, D)
    s["k_back"].copy_((kc.float().unflatten(-1, (4, GROUP)) * ks.float()[..., None]).flatten(-2))
    s["v_back"].copy_((vc.float().unflatten(-1, (4, GROUP)) * vs.float()[..., None]).flatten(-2))
    return {"k": s["k_back"], "v": s["v_back"], "means": s["means"], "lens": s["new_lens"]}


def _kept_tokens(c, lens, sel):
    """Tokens of the kept blocks [B, Hkv, n] (0 where there is none) and which of them count."""
    B, Hkv, bs = c["B"], c["Hkv"], c["bs"]
    if sel is None:
        nb = -(-c["cap"] // bs)
        sel = torch.arange(nb, dtype=torch.int32, device=lens.device).expand(B, Hkv, nb)
    tok = (sel.long()[..., None] * bs + torch.arange(bs, device=lens.device)).flatten(2)
    live = (sel >= 0).repeat_interleave(bs, 2) & (tok < lens[:, None, None])
    return torch.where(live, tok, 0), live


def _run_attn(s):
    c = s["case"]
    if own:
        import block_top_sparse_kin_b200 as kin

        kin.kin_kv_decode_attn(s["dims"], s["q"], s["kv"], s["lens"], s["sel"], s["cnt"], c["k"], 0.0, s["out"], s["lse"],
                               s["ws"], acc=s["acc"])
        return _attn_outputs(s, s["out"], s["lse"])
    B, Hkv, Hq, cap = c["B"], c["Hkv"], c["Hq"], c["cap"]
    tok, live = _kept_tokens(c, s["lens"], s["sel"])
    at = _row_ids(c, cap, s["table"], tok)
    if c["int4"]:
        k = _values(s["k"].view(-1, 64)[at], s["ks"].view(-1, 4)[at], s["order"]["k_at"])
    else:
        k = s["k"].view(-1, D)[at].float()
    q = s["q"].float().view(B, Hkv, Hq // Hkv, D)
    z = torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(D)
    del k
    z = torch.where(live[:, :, None], z, -math.inf)
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - m)
    total = p.sum(-1, keepdim=True)
    lse = m + torch.log(total)
    if c["int4"]:
        v = _values(s["v"].view(-1, 64)[at], s["vs"].view(-1, 4)[at], s["order"]["v_at"])
    else:
        v = s["v"].view(-1, D)[at].float()
    out = (torch.matmul(p, v) / total).view(B, Hq, D).to(torch.bfloat16)
    if c["acc"]:
        w = torch.exp(z - lse).sum(2) * live
        ids = torch.arange(B * Hkv, device=tok.device).view(B, Hkv, 1) * cap + tok
        s["acc"].view(-1).index_add_(0, ids.flatten(), w.flatten())
    return _attn_outputs(s, out, lse.view(B, Hq))


def _attn_outputs(s, out, lse):
    r = {"out": out, "lse": lse}
    if s["acc"] is not None:
        r["acc"] = s["acc"]
    return r


def _evict_outputs(s):
    r = {"sel": s["sel"], "acc": s["acc2"], "lens": s["lens2"], "means": s["means"]}
    names = ("k_back", "v_back") if s["case"]["int4"] else ("k2", "v2")
    r["k"], r["v"] = s[names[0]], s[names[1]]
    return r


def _run_evict(s):
    c = s["case"]
    if own:
        import block_top_sparse_kin_b200 as kin

        kin.kin_kv_evict(s["dims"], s["kv"], s["acc"], s["lens"], c["n_keep"], c["n_sink"], c["n_recent"], s["dims2"],
                         s["kv2"], s["acc2"], s["lens2"], s["ws"], block_means=s["means"], sel_tokens=s["sel"])
        if c["int4"]:
            kin.kin_kv4_load(s["dims2"], s["kv2"], s["lens2"], s["k_back"], s["v_back"])
        return _evict_outputs(s)
    B, Hkv, cap, keep = c["B"], c["Hkv"], c["cap"], c["n_keep"]
    cap2, lens = _dst_cap(c), s["lens"]
    dev = lens.device
    t = torch.arange(cap, device=dev)
    there = (t < lens[:, None])[:, None]
    forced = ((t < c["n_sink"]) | (t >= lens[:, None] - c["n_recent"]))[:, None] & there
    key = torch.where(there, torch.where(forced, math.inf, s["acc"]), -math.inf)
    order = key.sort(dim=-1, descending=True, stable=True).indices[..., : min(keep, cap)]
    lens2 = lens.clamp(max=keep)
    n = order.shape[-1]
    live = torch.arange(n, device=dev) < lens2[:, None, None]
    sel = torch.where(live, order, 1 << 30).sort(-1).values
    live = live.expand(B, Hkv, n)
    s["sel"].fill_(-1)
    s["sel"][..., :n] = torch.where(live, sel, -1).to(torch.int32)
    s["lens2"].copy_(lens2)
    # past a sequence's kept tokens the first one is moved once more
    src = torch.where(live, sel, sel[..., :1])
    dst = torch.where(live, torch.arange(n, device=dev), 0)
    at = _row_ids(c, cap, s["table"], src).flatten()
    to = _row_ids(c, cap2, s["table2"], dst).flatten()
    w = 64 if c["int4"] else D
    s["k2"].view(-1, w)[to] = s["k"].view(-1, w)[at]
    s["v2"].view(-1, w)[to] = s["v"].view(-1, w)[at]
    s["acc2"].zero_()
    s["acc2"][..., :n] = torch.where(live, s["acc"].gather(-1, src), 0.0)
    some = live[..., None]
    if c["int4"]:
        s["ks2"].view(-1, 4)[to] = s["ks"].view(-1, 4)[at]
        s["vs2"].view(-1, 4)[to] = s["vs"].view(-1, 4)[at]
        k = _values(s["k"].view(-1, 64)[at], s["ks"].view(-1, 4)[at], s["order"]["k_at"]).view(B, Hkv, n, D) * some
        v = _values(s["v"].view(-1, 64)[at], s["vs"].view(-1, 4)[at], s["order"]["v_at"]).view(B, Hkv, n, D) * some
        s["k_back"][:, :, :n], s["v_back"][:, :, :n] = k.to(torch.bfloat16), v.to(torch.bfloat16)
        s["k_back"][:, :, n:], s["v_back"][:, :, n:] = 0, 0
    else:
        k = s["k"].view(-1, D)[at].float().view(B, Hkv, n, D) * some
    k = torch.nn.functional.pad(k, (0, 0, 0, cap2 - n))
    s["means"].copy_(_block_means(c, cap2, lens2, k))
    return _evict_outputs(s)


# ------------------------------------------------------------------- exact

def _exact_rows(c, s, names, b, tokens, order=None):
    """Rows of one sequence in 64 bits, by their definition: tokens [Hkv, n] of sequence b."""
    Hkv, cap, bs = c["Hkv"], c["cap"], c["bs"]
    got = []
    for h in range(Hkv):
        t = tokens[h]
        at = (b * Hkv + h) * cap + t if s["table"] is None else (s["table"][b].long()[t // bs] * Hkv + h) * bs + t % bs
        data = s[names[0]].flatten(0, 2)[at]
        if order is None:
            got.append(data.double())
            continue
        x = torch.zeros((t.numel(), D), dtype=torch.float64, device=t.device)
        nibbles = torch.empty((t.numel(), D), dtype=torch.int64, device=t.device)
        nibbles[:, 0::2], nibbles[:, 1::2] = (data % 16).long(), (data // 16).long()
        x[:, torch.tensor(order, device=t.device)] = (nibbles - 8).double()
        scale = s[names[1]].flatten(0, 2)[at].double()
        got.append(x * torch.repeat_interleave(scale, GROUP, dim=1))
    return torch.stack(got)


def _exact_quant(x):
    """The values that rows x stand for in 4 bits, in 64 bits."""
    y = x.double().reshape(-1, GROUP)
    a = y.abs().max(1, keepdim=True).values
    s = (a / 7).float().bfloat16().double()  # a / 7 is never within fp32's rounding of a bf16 midpoint unless it is one
    c = torch.where(s > 0, torch.clip(torch.round(y / torch.where(s > 0, s, 1.0)), -7, 7), 0.0)
    return (c * s).reshape(x.shape)


def _exact_means(c, x, n, nb):
    """Block means of one sequence's key values x [Hkv, >= n, D] of n tokens."""
    m = torch.zeros((c["Hkv"], nb, D), dtype=torch.float64, device=x.device)
    whole = n // c["bs"]
    if whole:
        m[:, :whole] = x[:, : whole * c["bs"]].reshape(c["Hkv"], whole, c["bs"], D).mean(2)
    if n > whole * c["bs"]:
        m[:, whole] = x[:, whole * c["bs"]: n].mean(1)
    return m


def exact(c, seed):
    s = prepare(c, seed)
    lens = _lens(c)
    dev = s["lens"].device
    B, Hkv, Hq, bs, cap = c["B"], c["Hkv"], c["Hq"], c["bs"], c["cap"]
    every = lambda n: torch.arange(n, device=dev).expand(Hkv, n)  # noqa: E731
    if c["op"] == "store":
        k = torch.zeros((B, Hkv, cap, D), dtype=torch.float64, device=dev)
        v, means = torch.zeros_like(k), []
        for b, n in enumerate(lens):
            k[b, :, :n] = _exact_quant(_exact_rows(c, s, ("k",), b, every(n)))
            v[b, :, :n] = _exact_quant(_exact_rows(c, s, ("v",), b, every(n)))
            means.append(_exact_means(c, k[b], n, s["means"].shape[2]))
        return {"k": k, "v": v, "means": torch.stack(means)}
    if c["op"] == "append":
        kn, vn = _exact_quant(s["k_new"]), _exact_quant(s["v_new"])
        means = []
        for b, n in enumerate(lens):
            held = _exact_rows(c, s, ("k", "ks"), b, every(n), K_ORDER)
            m = s["means"][b].double().clone()
            new = _exact_means(c, torch.cat((held, kn[b]), 1), n + c["n_new"], m.shape[1])
            first, last = n // bs, (n + c["n_new"] - 1) // bs
            m[:, first: last + 1] = new[:, first: last + 1]
            means.append(m)
        return {"k": kn, "v": vn, "means": torch.stack(means), "lens": s["lens"] + c["n_new"]}
    if c["op"] == "attn":
        outs, lses = [], []
        acc = None if s["acc"] is None else s["acc"].double()
        for b, n in enumerate(lens):
            if s["sel"] is None:
                tok = every(n)
                live = torch.ones_like(tok, dtype=torch.bool)
            else:
                blk = s["sel"][b].long()
                tok = (blk[:, :, None] * bs + torch.arange(bs, device=dev)).reshape(Hkv, -1)
                live = (blk[:, :, None].expand(-1, -1, bs).reshape(Hkv, -1) >= 0) & (tok < n)
                tok = tok * live
            if c["int4"]:
                k = _exact_rows(c, s, ("k", "ks"), b, tok, K_ORDER)
                v = _exact_rows(c, s, ("v", "vs"), b, tok, V_ORDER)
            else:
                k, v = _exact_rows(c, s, ("k",), b, tok), _exact_rows(c, s, ("v",), b, tok)
            q = s["q"][b].double().reshape(Hkv, Hq // Hkv, D)
            z = torch.einsum("hjd,htd->hjt", q, k) / math.sqrt(D)
            z = z.masked_fill(~live[:, None], -math.inf)
            lse = torch.logsumexp(z, -1, keepdim=True)
            w = torch.exp(z - lse)
            outs.append(torch.einsum("hjt,htd->hjd", w, v).reshape(Hq, D))
            lses.append(lse.reshape(Hq))
            if acc is not None:
                acc[b].scatter_add_(1, tok, w.sum(1))
        r = {"out": torch.stack(outs), "lse": torch.stack(lses)}
        if acc is not None:
            r["acc"] = acc
        return r
    cap2, keep = _dst_cap(c), c["n_keep"]
    k = torch.zeros((B, Hkv, cap2, D), dtype=torch.float64, device=dev)
    v = torch.zeros_like(k)
    acc = torch.zeros((B, Hkv, cap2), dtype=torch.float64, device=dev)
    sel = torch.full((B, Hkv, keep), -1, dtype=torch.int32, device=dev)
    means, lens2 = [], []
    for b, n in enumerate(lens):
        m = min(n, keep)
        lens2.append(m)
        if n <= keep:
            tok = every(n)
        else:
            first, last = c["n_sink"], n - c["n_recent"]
            a = s["acc"][b, :, first:last]
            best = torch.argsort(-a, dim=1, stable=True)[:, : keep - c["n_sink"] - c["n_recent"]] + first
            ends = torch.cat((torch.arange(first, device=dev), torch.arange(last, n, device=dev))).expand(Hkv, -1)
            tok = torch.cat((ends, best), 1).sort(1).values
        sel[b, :, :m] = tok.int()
        acc[b, :, :m] = s["acc"][b].double().gather(1, tok)
        if c["int4"]:
            k[b, :, :m] = _exact_rows(c, s, ("k", "ks"), b, tok, K_ORDER)
            v[b, :, :m] = _exact_rows(c, s, ("v", "vs"), b, tok, V_ORDER)
        else:
            k[b, :, :m], v[b, :, :m] = _exact_rows(c, s, ("k",), b, tok), _exact_rows(c, s, ("v",), b, tok)
        means.append(_exact_means(c, k[b], m, s["means"].shape[2]))
    if not c["int4"]:
        k, v = _into(c, cap2, s["table2"], k), _into(c, cap2, s["table2"], v)
    return {"sel": sel, "acc": acc, "lens": torch.tensor(lens2, dtype=torch.int32, device=dev), "means": torch.stack(means),
            "k": k, "v": v}
