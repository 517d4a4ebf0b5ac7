"""The 4-bit cache, the attention over either cache with its accumulated
weights, and the eviction, against plain forms in 64 bits.

Tolerances, from the arithmetic (u16 = 2^-8 for a bf16 result, each rounding
off by at most half a step):
  * codes, scales, moved rows, lengths, kept tokens and block means: equal
    (the means' sums run in fp32 in the plain form's order);
  * logits: a 4-bit key enters the products as 24 + c <= 31 times a query
    channel, beside -24 sum q, in fp32 sums of at most 4 steps of 16 products,
    so a group's sum is off by at most 4 * 17 * 2^-24 * 55 sum |q|; bf16 keys:
    8 * 17 * 2^-24 * sum |q k|; both times the scale, and 2^-22 for the
    scaling itself.  delta below is that bound, with a factor 2 for the
    matrix unit's truncation;
  * lse: delta + 2^-20 (1 + |lse|) (exp2 and log2 to 2^-21);
  * weights: each is off by a factor e^(2 delta + 2^-19), its sum in acc once
    more by 2^-24 of the total;
  * out: the weights' rounding (4 bit: two roundings to 11 bits, 2^-10; bf16:
    two bf16 numbers, 2^-16) and factor on sum p |v|, then u16 on the result.
    4-bit values enter as 8 + c <= 15 steps, 8 times the weights' sum comes off
    at the end: each of a warp's at most 32 tiles adds to sums of up to 15 and
    8 times sum p s (s: the group's step), truncated at 24 bits, so
    23 * 32 * 2^-23 < 2^-13 of sum p s.
"""
import math

import pytest
import torch

import block_top_sparse_kin_b200 as kin
import kin_kv_ref as ref

pytestmark = pytest.mark.gpu
D = 128


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rows16(seed, *shape, scale=1.0):
    return (scale * torch.randn(shape, generator=gen(seed), device="cuda")).to(torch.bfloat16)


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def table_for(B, nb, seed, spare=3):
    return torch.randperm(B * nb + spare, generator=gen(seed), device="cuda")[: B * nb].to(torch.int32).view(B, nb).contiguous()


class Cache:
    """Random bf16 rows for given lengths, and the same cache in the layouts
    under test.  Rows behind a length hold NaN (bf16) or noise (4 bit) that no
    call may read."""

    def __init__(self, lens, Hkv, bs, cap, paged, seed, scale=1.0):
        self.lens, self.Hkv, self.bs, self.cap, self.B = lens, Hkv, bs, cap, len(lens)
        self.nb = -(-cap // bs)
        self.k, self.v = rows16(seed, self.B, Hkv, cap, D, scale=scale), rows16(seed + 1, self.B, Hkv, cap, D, scale=scale)
        # a heavy block and some uneven groups
        self.k[:, :, : min(bs, cap)] += rows16(seed + 2, self.B, Hkv, 1, D)
        self.v[:, :, ::3, 32:64] *= 8
        for b, n in enumerate(lens):
            self.k[b, :, max(n, 0):] = math.nan
            self.v[b, :, max(n, 0):] = math.nan
        self.table = table_for(self.B, self.nb, seed + 3) if paged else None
        self.pages = self.B * self.nb + 3
        self.seq = ints(lens)

    def dims(self, g=1):
        return kin.make_dims(self.B, self.Hkv, self.Hkv * g, D, self.bs, self.cap)

    def place(self, rows, fill):
        """Logical rows as a cache tensor; places that hold no row: fill."""
        if self.table is None:
            return rows.clone()
        pool = torch.full((self.pages, self.Hkv, self.bs, rows.shape[-1]), fill, dtype=rows.dtype, device="cuda")
        ref.to_pool(rows, self.table, self.bs, pool)
        return pool

    def logical(self, t):
        return t if self.table is None else ref.from_pool(t, self.table, self.cap)

    def bf16(self):
        return kin.KvCache(self.place(self.k, math.nan), self.place(self.v, math.nan), block_table=self.table)

    def empty4(self):
        """A 4-bit cache of noise codes and NaN scales."""
        kv = kin.alloc_kv4(self.dims()) if self.table is None else \
            kin.alloc_kv4(self.dims(), num_pages=self.pages, block_table=self.table)
        for t in (kv.k, kv.v):
            t.fill_(0x5A)
        for t in (kv.k_scales, kv.v_scales):
            t.fill_(math.nan)
        return kv

    def stored(self):
        kv, st = self.empty4(), status()
        kin.kin_kv4_store(self.dims(), self.bf16(), kv, self.seq, dev_status=st)
        assert int(st.item()) == 0
        return kv

    def held(self):
        """The values a 4-bit cache of these rows stands for (float64; 0 behind the lengths)."""
        out = []
        for x in (self.k, self.v):
            c, s = ref.quantise(x)
            y = ref.values(c, s)
            for b, n in enumerate(self.lens):
                y[b, :, max(n, 0):] = 0
            out.append(y)
        return out

    def check4(self, kv, lens=None):
        """kv holds exactly the codes and scales of these rows."""
        for codes, scales, x, order in ((kv.k, kv.k_scales, self.k, ref.KEY_ORDER), (kv.v, kv.v_scales, self.v, ref.VALUE_ORDER)):
            c, s = ref.quantise(x)
            want, ws = ref.pack(c, order), s.to(torch.bfloat16)
            got, gs = self.logical(codes), self.logical(scales)
            for b, n in enumerate(self.lens if lens is None else lens):
                n = max(n, 0)
                assert torch.equal(got[b, :, :n], want[b, :, :n])
                assert torch.equal(gs[b, :, :n].view(torch.int16), ws[b, :, :n].view(torch.int16)) or \
                    torch.equal(gs[b, :, :n].nan_to_num(-1), ws[b, :, :n].nan_to_num(-1))
                assert (got[b, :, n:] == 0x5A).all() and gs[b, :, n:].isnan().all()


SHAPES = [  # lens, Hkv, bs, cap
    ([1], 1, 16, 1),
    ([0, 1, 17], 2, 16, 33),          # an odd capacity: scale rows start at 8 bytes
    ([40, 64, 63], 3, 32, 64),
    ([100, 0, 257, 130], 2, 64, 301),
    ([128, 300], 1, 128, 300),
]


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"bs{s[2]}_cap{s[3]}")
def test_store_and_load(shape, paged):
    c = Cache(*shape, paged, 11)
    kv, st = c.empty4(), status()
    means = torch.full((c.B, c.Hkv, c.nb, D), 7.0, device="cuda")
    kin.kin_kv4_store(c.dims(), c.bf16(), kv, c.seq, means, st)
    c.check4(kv)
    hk, hv = c.held()
    want = ref.block_means(hk.float(), c.lens, c.bs)
    assert torch.equal(means, torch.where(want.isnan(), torch.full_like(want, 7.0), want))
    k, v = torch.empty_like(c.k), torch.empty_like(c.v)
    kin.kin_kv4_load(c.dims(), kv, c.seq, k, v, dev_status=st)
    assert torch.equal(k, hk.to(torch.bfloat16)) and torch.equal(v, hv.to(torch.bfloat16))  # one rounding; zeros behind
    # a window that begins inside and ends behind the rows
    starts = ints([min(5, n) for n in c.lens])
    n = min(20, c.cap)
    k, v = (torch.full((c.B, c.Hkv, n, D), math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kin.kin_kv4_load(c.dims(), kv, c.seq, k, v, starts=starts, dev_status=st)
    for b in range(c.B):
        s = int(starts[b])
        pad = torch.zeros((c.Hkv, n, D), dtype=torch.float64, device="cuda")
        m = max(0, min(n, c.lens[b] - s))
        pad[:, :m] = hk[b, :, s: s + m]
        assert torch.equal(k[b], pad.to(torch.bfloat16))
    assert int(st.item()) == 0


@pytest.mark.parametrize("kind", ["bf16", "dual", "per_page"])
def test_store_other_means(kind):
    c = Cache([70, 33], 2, 32, 80, True, 21)
    kv, st = c.empty4(), status()
    want = ref.block_means(c.held()[0].float(), c.lens, c.bs)
    live = ~want.isnan()
    if kind == "bf16":
        means = torch.zeros((2, 2, c.nb, D), dtype=torch.bfloat16, device="cuda")
        kin.kin_kv4_store(c.dims(), c.bf16(), kv, c.seq, means, st)
        assert torch.equal(means[live], want.to(torch.bfloat16)[live])
    elif kind == "dual":
        # the same bytes as the means of a bf16 cache that holds the 4-bit values exactly cannot be had
        # (they need 11 bits): the fp32 part is compared, the bf16 part is its rounding
        means = kin.alloc_dual_means(c.dims())
        kin.kin_kv4_store(c.dims(), c.bf16(), kv, c.seq, means, st)
        n = want.numel()
        f = means[: 4 * n].view(torch.float32).view_as(want)
        h = means[4 * n: 6 * n].view(torch.bfloat16).view_as(want)
        rad = means[6 * n:].view(torch.float32).view(want.shape[:-1])
        assert torch.equal(f[live], want[live]) and torch.equal(h[live], want.to(torch.bfloat16)[live])
        miss = (want.double() - want.to(torch.bfloat16).double()).norm(dim=-1)
        ok = live.all(-1)
        assert (rad[ok] >= miss[ok]).all() and (rad[ok] <= 1.01 * miss[ok] + 2**-17 * want[ok].norm(dim=-1)).all()
    else:
        means = torch.zeros((c.pages, 2, D), device="cuda")
        kin.kin_kv4_store(c.dims(), c.bf16(), kv, c.seq, means, st, per_page=True)
        for b in range(2):
            for i in range(-(-c.lens[b] // 32)):
                assert torch.equal(means[c.table[b, i].long()], want[b, :, i])
    assert int(st.item()) == 0


def test_groups_at_the_edges_of_the_format():
    """Ties, zeros, the largest and smallest magnitudes, NaN and infinities."""
    x = torch.zeros((1, 1, 16, D), dtype=torch.bfloat16, device="cuda")
    g = gen(3)
    halves = (torch.arange(32, device="cuda") % 15 - 7).float() + 0.5
    x[0, 0, 0, :32] = halves.clamp(max=6.5)       # a tie at every code for s = 1 (with 7 present below)
    x[0, 0, 0, 0] = 7
    x[0, 0, 1, :32] = halves.clamp(max=6.5) * 3
    x[0, 0, 1, 1] = -21
    x[0, 0, 2] = 3.3e38
    x[0, 0, 3] = torch.finfo(torch.bfloat16).tiny
    x[0, 0, 4, :40] = 2.0**-133                   # the least subnormal: its scale rounds to zero
    x[0, 0, 5, 3], x[0, 0, 5, 50], x[0, 0, 5, 100] = math.nan, math.inf, -math.inf
    x[0, 0, 6] = (torch.randn(D, generator=g, device="cuda") * 1e-38).to(torch.bfloat16)
    x[0, 0, 7] = (torch.randn(D, generator=g, device="cuda") * 2.0**-120).to(torch.bfloat16)
    x[0, 0, 8:] = (torch.randn((8, D), generator=g, device="cuda") * 2 ** torch.randn((8, D), generator=g, device="cuda").mul(8)).to(torch.bfloat16)
    dims = kin.make_dims(1, 1, 1, D, 16, 16)
    kv, st = kin.alloc_kv4(dims), status()
    kin.kin_kv4_store(dims, kin.KvCache(x, x.clone()), kv, ints([16]), dev_status=st)
    c, s = ref.quantise(x)
    assert torch.equal(kv.k, ref.pack(c, ref.KEY_ORDER)) and torch.equal(kv.v, ref.pack(c, ref.VALUE_ORDER))
    want = s.to(torch.bfloat16)
    for got in (kv.k_scales, kv.v_scales):
        assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(-1), want.nan_to_num(-1))
    assert s[0, 0, 4, 0] == 0 and s[0, 0, 5, :2].isnan().all() and s[0, 0, 5, 3].isnan() and s[0, 0, 5, 2] == 0


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("n_new", [1, 15, 16, 100])
@pytest.mark.parametrize("in_place", [False, True])
def test_append_equals_store(n_new, paged, in_place):
    """Appending to a stored prefix leaves the bytes, means and lengths of storing everything."""
    before = [0, 1, 31, 64, 77]
    c = Cache([n + n_new for n in before], 2, 32, 77 + n_new + 1, paged, 31)
    st = status()
    whole = c.empty4()
    m_whole = torch.full((c.B, c.Hkv, c.nb, D), 3.0, device="cuda")
    kin.kin_kv4_store(c.dims(), c.bf16(), whole, c.seq, m_whole, st)
    kv, means = c.empty4(), torch.full_like(m_whole, 3.0)
    lens = ints(before)
    kin.kin_kv4_store(c.dims(), c.bf16(), kv, lens, means, st)
    new = [torch.stack([x[b, :, n: n + n_new] for b, n in enumerate(before)]).contiguous() for x in (c.k, c.v)]
    out = lens if in_place else torch.full_like(lens, -5)
    kin.kin_kv4_append(c.dims(), kv, means, lens, out, *new, n_new, st)
    assert int(st.item()) == 0 and out.tolist() == c.lens
    if not in_place:
        assert lens.tolist() == before
    c.check4(kv)
    assert torch.equal(means, m_whole)


def test_append_nothing_and_without_room():
    c = Cache([3, 16, 9], 1, 16, 16, False, 41)
    kv, st = c.stored(), status()
    out = torch.full((3,), -1, dtype=torch.int32, device="cuda")
    new = rows16(5, 3, 1, 4, D)
    kin.kin_kv4_append(c.dims(), kv, None, c.seq, out, new[:1, :, :1, :8].contiguous(), new, 0, st)  # nothing is read of it
    assert out.tolist() == [3, 16, 9] and int(st.item()) == 0
    c.check4(kv)
    kin.kin_kv4_append(c.dims(), kv, None, c.seq, out, new, new, 4, st)  # the second has no room
    assert out.tolist() == [7, 16, 13] and int(st.item()) == 5
    got = kv.k[1, 0]
    assert torch.equal(got, ref.pack(ref.quantise(c.k[1, 0])[0], ref.KEY_ORDER))


def test_bad_lengths_and_pages_are_skipped_and_flagged():
    c = Cache([40, 40], 1, 16, 48, True, 51)
    kv, src = c.empty4(), c.bf16()
    st = status()
    kin.kin_kv4_store(c.dims(), src, kv, ints([40, 49]), dev_status=st)
    assert int(st.item()) == 5
    c.check4(kv, [40, 0])
    st = status()
    good = c.table.clone()
    bad = good.clone()
    bad[0, 1], bad[1, 0] = -1, c.pages
    st = status()
    kv = c.empty4()
    kv_bad = kin.KvCache(kv.k, kv.v, kv.k_scales, kv.v_scales, block_table=bad)
    kin.kin_kv4_store(c.dims(), src, kv_bad, c.seq, dev_status=st)
    assert int(st.item()) == 5
    assert (kv.k[good[0, 1].long()] == 0x5A).all() and (kv.k[good[0, 0].long(), 0] != 0x5A).any()
    # reading back: the bad pages' rows are zeros
    st = status()
    kv = c.stored()
    k, v = torch.ones_like(c.k), torch.ones_like(c.v)
    kin.kin_kv4_load(c.dims(), kin.KvCache(kv.k, kv.v, kv.k_scales, kv.v_scales, block_table=bad), c.seq, k, v, dev_status=st)
    assert int(st.item()) == 5
    hk = c.held()[0].to(torch.bfloat16)
    hk[0, :, 16:32] = 0
    hk[1, :, :16] = 0
    assert torch.equal(k, hk)
    # attention: those blocks are left out
    st = status()
    q = rows16(52, 2, 2, D)
    out, lse, acc = torch.empty_like(q), torch.empty((2, 2), device="cuda"), torch.zeros((2, 1, 48), device="cuda")
    d = c.dims(2)
    kin.kin_kv_decode_attn(d, q, kin.KvCache(kv.k, kv.v, kv.k_scales, kv.v_scales, block_table=bad), c.seq, None, None, 0, 0.0,
                           out, lse, kin.alloc_kv_attn_workspace(d, 0, acc=True), acc=acc, dev_status=st)
    assert int(st.item()) == 5
    check_attention(c, q, out, lse, acc, None, True, sel=[[[0, 2]], [[1, 2]]])


def logit_delta(c, q, int4, scale, g):
    """The bound on a logit's error (see above), over all tokens: a float."""
    k, _ = (c.held() if int4 else (c.k.double().nan_to_num(0), None))
    qg = q.double().view(c.B, c.Hkv, g, D)
    if int4:
        s = ref.quantise(c.k)[1].nan_to_num(0)
        for b, n in enumerate(c.lens):
            s[b, :, max(n, 0):] = 0
        top = s.amax(2)  # [B, Hkv, 4]
        per = qg.abs().unflatten(-1, (4, 32)).sum(-1) * 55 * top[:, :, None]
        each = 2 * 4 * 17 * 2.0**-24 * per.sum(-1)
    else:
        top = k.abs().amax(2)
        each = 2 * 8 * 17 * 2.0**-24 * (qg.abs() * top[:, :, None]).sum(-1)
    return float(each.max()) * scale + 2.0**-22 * 64


def check_attention(c, q, out, lse, acc, acc0, int4, sel=None, scale=1 / math.sqrt(D), tiles=32):
    g = q.shape[1] // c.Hkv
    hk, hv = c.held() if int4 else (c.k.double().nan_to_num(0), c.v.double().nan_to_num(0))
    o, l, w, spread = ref.attend(q, hk, hv, [max(n, 0) for n in c.lens], sel, scale, c.bs)
    delta = logit_delta(c, q, int4, scale, g)
    some = torch.isfinite(l)
    assert torch.equal(torch.isfinite(lse), some)
    assert ((lse.double() - l)[some].abs() <= delta + 2.0**-20 * (1 + l[some].abs())).all()
    tol = 2.0**-8 * o.abs() + (2.0**-10 if int4 else 2.0**-16) * spread + (2 * delta + 2.0**-19) * spread + 2.0**-140
    if int4:
        step = ref.quantise(c.v)[1].nan_to_num(0).repeat_interleave(32, -1)
        tol += tiles / 32 * 2.0**-13 * ref.attend(q, hk, step, [max(n, 0) for n in c.lens], sel, scale, c.bs)[0]
    err = (out.double() - o).abs()
    assert (err <= tol).all(), float((err / tol).max())
    assert (out[~some] == 0).all()
    if acc is not None:
        base = torch.zeros_like(w) if acc0 is None else acc0.double()
        werr = (acc.double() - base - w).abs()
        assert (werr <= w * (2 * delta + 2.0**-18) + 2.0**-24 * (base + w)).all()
        assert torch.equal(acc[w == 0], (torch.zeros_like(acc) if acc0 is None else acc0)[w == 0])


def random_selection(c, k, seed):
    """k kept blocks a pair (or all): ascending, -1 padded; also as lists."""
    sel = torch.full((c.B, c.Hkv, k), -1, dtype=torch.int32)
    cnt = torch.zeros((c.B, c.Hkv), dtype=torch.int32)
    g = torch.Generator().manual_seed(seed)
    for b, n in enumerate(c.lens):
        nb = -(-max(n, 0) // c.bs)
        for h in range(c.Hkv):
            m = min(k, nb)
            pick = torch.randperm(nb, generator=g)[:m].sort().values.int()
            sel[b, h, :m], cnt[b, h] = pick, m
    return sel, cnt


ATTN = [  # lens, Hkv, bs, cap, g, kept blocks (0: all)
    ([1], 1, 16, 1, 1, 0),
    ([17, 1, 100], 2, 16, 101, 4, 3),
    ([333, 15, 16, 200], 2, 32, 335, 3, 0),
    ([1000, 64, 129], 1, 64, 1001, 8, 9),
    ([2000], 3, 128, 2000, 5, 7),
    ([3001, 1600], 2, 16, 3001, 2, 150),      # several chunks a pair
    ([5000], 1, 16, 5003, 7, 0),
    ([20000], 1, 32, 20000, 8, 0),            # several merge batches
]


@pytest.mark.parametrize("int4", [True, False], ids=["int4", "bf16"])
@pytest.mark.parametrize("paged", [False, True], ids=["flat", "paged"])
@pytest.mark.parametrize("case", ATTN, ids=lambda a: f"bs{a[2]}_g{a[4]}_k{a[5]}_cap{a[3]}")
def test_attention(case, paged, int4):
    lens, Hkv, bs, cap, g, k = case
    c = Cache(lens, Hkv, bs, cap, paged, 61)
    kv = c.stored() if int4 else c.bf16()
    d, st = c.dims(g), status()
    q = rows16(62, c.B, Hkv * g, D)
    sel, cnt = random_selection(c, k, 63) if k else (None, None)
    dev = (sel.cuda(), cnt.cuda()) if k else (None, None)
    out, lse = torch.full_like(q, 9.0), torch.full((c.B, Hkv * g), 9.0, device="cuda")
    acc0 = torch.rand((c.B, Hkv, cap), generator=gen(64), device="cuda")
    acc = acc0.clone()
    ws = kin.alloc_kv_attn_workspace(d, k, acc=True)
    kin.kin_kv_decode_attn(d, q, kv, c.seq, *dev, k, 0.0, out, lse, ws, acc=acc, dev_status=st)
    assert int(st.item()) == 0
    lists = None if not k else sel.tolist()
    check_attention(c, q, out, lse, acc, acc0, int4, lists)
    # without weights and without lse: the same bits; the workspace is ready again
    out2 = torch.full_like(q, 9.0)
    kin.kin_kv_decode_attn(d, q, kv, c.seq, *dev, k, 0.0, out2, None, ws, dev_status=st)
    assert torch.equal(out2, out)
    # another scale
    kin.kin_kv_decode_attn(d, q, kv, c.seq, *dev, k, 0.31, out, lse, ws, dev_status=st)
    check_attention(c, q, out, lse, None, None, int4, lists, scale=0.31)
    assert int(st.item()) == 0


@pytest.mark.parametrize("int4", [True, False], ids=["int4", "bf16"])
@pytest.mark.parametrize("B,k", [(64, 128), (32, 256), (61, 10), (3, 129)])
def test_attention_ranges_over_many_pairs(B, k, int4):
    """Ragged batches that fill the card: ranges that run over one pair's end
    into the next, over several short pairs, and pairs of one range each; some
    pairs keep fewer blocks than the budget, one sequence is empty."""
    lens = [(1 + 37 * i * i) % 4300 for i in range(B)]
    lens[1], lens[2], lens[-1] = 0, 1, 4300
    c = Cache(lens, 8, 16, 4300, True, 65)
    g = 2
    kv, d, st = (c.stored() if int4 else c.bf16()), c.dims(g), status()
    q = rows16(66, B, 8 * g, D)
    sel, cnt = random_selection(c, k, 67)
    out, lse = torch.full_like(q, 9.0), torch.full((B, 8 * g), 9.0, device="cuda")
    acc = torch.zeros((B, 8, 4300), device="cuda")
    ws = kin.alloc_kv_attn_workspace(d, k, acc=True)
    for _ in range(2):  # the second call meets the first one's workspace
        acc.zero_()
        kin.kin_kv_decode_attn(d, q, kv, c.seq, sel.cuda(), cnt.cuda(), k, 0.0, out, lse, ws, acc=acc, dev_status=st)
        check_attention(c, q, out, lse, acc, None, int4, sel.tolist())
    assert int(st.item()) == 5  # the empty sequence


def test_attention_bf16_values_of_any_magnitude():
    """Weights below 1: the largest finite values average without overflow."""
    c = Cache([300], 1, 16, 300, False, 68)
    c.v = (c.v.float().clamp(-1, 1) * 3e38).to(torch.bfloat16)
    q = rows16(69, 1, 2, D)
    out, lse, d = torch.empty_like(q), torch.empty((1, 2), device="cuda"), c.dims(2)
    kin.kin_kv_decode_attn(d, q, c.bf16(), c.seq, None, None, 0, 0.0, out, lse, kin.alloc_kv_attn_workspace(d, 0))
    check_attention(c, q, out, lse, None, None, False)


def test_attention_queries_of_any_magnitude():
    """Each head's queries are scaled on their own: tiny beside huge ones, and zeros."""
    c = Cache([120], 1, 16, 120, False, 70)
    q = rows16(71, 1, 6, D).float()
    q *= torch.tensor([1, 2.0**-40, 2.0**40, 0, 2.0**-126, 2.0**100], device="cuda")[None, :, None]
    q = q.to(torch.bfloat16)
    c.k[:, :, :, :] *= 2.0**-7
    out, lse, d = torch.empty_like(q), torch.empty((1, 6), device="cuda"), c.dims(6)
    hk, hv = c.held()
    for j, scale in enumerate([0.2, 2.0**39, 2.0**-41, 0.2, 0.2, 2.0**-102]):
        kin.kin_kv_decode_attn(d, q, c.stored(), c.seq, None, None, 0, scale, out, lse, kin.alloc_kv_attn_workspace(d, 0))
        o, l, _, _ = ref.attend(q, hk, hv, [120], None, scale, 16)
        assert abs(float(lse[0, j]) - float(l[0, j])) < 1e-4
        assert (out[0, j].double() - o[0, j]).abs().max() < 2.0**-7 * o[0, j].abs().max()


@pytest.mark.parametrize("int4", [True, False], ids=["int4", "bf16"])
def test_attention_empty_and_bad_sequences(int4):
    """Lengths of 0 and beyond the capacity and pairs that keep nothing: out 0,
    lse -inf, weights untouched; a block listed beyond the length is left out."""
    c = Cache([0, 50, 50, 40], 1, 16, 50, False, 71)
    kv = c.stored() if int4 else c.bf16()
    d, st = c.dims(2), status()
    q = rows16(72, 4, 2, D)
    lens = ints([0, 51, 50, 40])
    acc = torch.zeros((4, 1, 50), device="cuda")
    out, lse = torch.full_like(q, 9.0), torch.full((4, 2), 9.0, device="cuda")
    ws = kin.alloc_kv_attn_workspace(d, 0, acc=True)
    kin.kin_kv_decode_attn(d, q, kv, lens, None, None, 0, 0.0, out, lse, ws, acc=acc, dev_status=st)
    assert int(st.item()) == 5
    c.lens = [0, 0, 50, 40]
    check_attention(c, q, out, lse, acc, None, int4)
    st = status()
    sel = ints([[[0, 1]], [[0, 1]], [[1, 7]], [[2, -1]]])
    cnt = ints([[2], [0], [2], [1]])
    acc.zero_()
    ws = kin.alloc_kv_attn_workspace(d, 2, acc=True)
    kin.kin_kv_decode_attn(d, q, kv, ints([0, 50, 50, 40]), sel, cnt, 2, 0.0, out, lse, ws, acc=acc, dev_status=st)
    assert int(st.item()) == 5
    c.lens = [0, 50, 50, 40]
    check_attention(c, q, out, lse, acc, None, int4, sel=[[[]], [[]], [[1]], [[2]]])


def test_a_block_listed_twice_weighs_twice():
    c = Cache([64], 1, 16, 64, False, 81)
    kv, d, q = c.stored(), c.dims(4), rows16(82, 1, 4, D)
    acc = torch.zeros((1, 1, 64), device="cuda")
    out, lse = torch.empty_like(q), torch.empty((1, 4), device="cuda")
    kin.kin_kv_decode_attn(d, q, kv, c.seq, ints([[[1, 2, 2]]]), ints([[3]]), 3, 0.0, out, lse,
                           kin.alloc_kv_attn_workspace(d, 3, acc=True), acc=acc)
    hk, hv = c.held()
    o, l, w, _ = ref.attend(q, hk, hv, [64], [[[1, 2, 2]]], 1 / math.sqrt(D), 16)
    assert torch.allclose(acc.double(), w, rtol=1e-4, atol=1e-7) and torch.allclose(lse.double(), l, atol=1e-4)
    assert (out.double() - o).abs().max() < 0.05


def test_values_of_very_different_scales():
    """Value scales that grow along the sequence over most of the range move
    the weights' common factor; a NaN group reaches its 32 channels alone."""
    c = Cache([256], 2, 16, 256, False, 91)
    grow = 2.0 ** torch.linspace(-60, 40, 256, device="cuda")
    c.v = (c.v.float() * grow[:, None]).to(torch.bfloat16)
    c.v[0, 1] = c.v[0, 1].flip(0)  # and shrink
    q = rows16(92, 1, 8, D, scale=0.1)
    out, lse = torch.empty_like(q), torch.empty((1, 8), device="cuda")
    d, st = c.dims(4), status()
    ws = kin.alloc_kv_attn_workspace(d, 0)
    kin.kin_kv_decode_attn(d, q, c.stored(), c.seq, None, None, 0, 0.0, out, lse, ws, dev_status=st)
    check_attention(c, q, out, lse, None, None, True)
    c.v[0, 0, 100, 40] = math.inf
    kin.kin_kv_decode_attn(d, q, c.stored(), c.seq, None, None, 0, 0.0, out, lse, ws, dev_status=st)
    assert out[0, :4, 32:64].isnan().all() and not out[0, :4, :32].isnan().any() and not out[0, :4, 64:].isnan().any()
    assert not out[0, 4:].isnan().any()
    # a NaN key poisons its head group's rows, as NaN logits do
    c.k[0, 1, 7, 3] = math.nan
    acc = torch.zeros((1, 2, 256), device="cuda")
    kin.kin_kv_decode_attn(d, q, c.stored(), c.seq, None, None, 0, 0.0, out, lse, kin.alloc_kv_attn_workspace(d, 0, acc=True),
                           acc=acc, dev_status=st)
    assert out[0, 4:].isnan().all() and lse[0, 4:].isnan().all() and acc[0, 1].isnan().all()
    assert not lse[0, :4].isnan().any() and not acc[0, 0].isnan().any()
    assert int(st.item()) == 0


def test_rows_beyond_32_bit_offsets():
    """A cache of more than 2^32 code bytes: the last head's rows."""
    Hkv, cap, bs = 20, 1 << 22, 128
    d = kin.make_dims(1, Hkv, Hkv, D, bs, cap)
    assert Hkv * cap * 64 > 1 << 32
    kv, st = kin.alloc_kv4(d), status()
    n = cap - 3
    lens = ints([n - 200])
    new = rows16(101, 1, Hkv, 200, D)
    out_lens = torch.zeros_like(lens)
    kin.kin_kv4_append(d, kv, None, lens, out_lens, new, new, 200, st)
    assert out_lens.tolist() == [n]
    k, v = torch.empty_like(new), torch.empty_like(new)
    kin.kin_kv4_load(d, kv, out_lens, k, v, starts=lens, dev_status=st)
    want = ref.values(*ref.quantise(new)).to(torch.bfloat16)
    assert torch.equal(k, want) and torch.equal(v, want)
    # attention over the last two blocks, weights to the far end of acc
    nb = -(-n // bs)
    sel = ints([[[nb - 2, nb - 1]]]).expand(1, Hkv, 2).contiguous()
    cnt = torch.full((1, Hkv), 2, dtype=torch.int32, device="cuda")
    q = rows16(102, 1, Hkv, D)
    out, lse = torch.empty_like(q), torch.empty((1, Hkv), device="cuda")
    acc = torch.zeros((1, Hkv, cap), device="cuda")
    kin.kin_kv_decode_attn(d, q, kv, out_lens, sel, cnt, 2, 0.0, out, lse, kin.alloc_kv_attn_workspace(d, 2, acc=True), acc=acc,
                           dev_status=st)
    t0 = (nb - 2) * bs
    tail = n - t0  # rows of the two blocks: zeros, then the new rows
    rows = torch.zeros((1, Hkv, tail, D), dtype=torch.float64, device="cuda")
    m = min(200, tail)
    rows[:, :, tail - m:] = ref.values(*ref.quantise(new))[:, :, 200 - m:]
    o, l, w, spread = ref.attend(q, rows, rows, [tail], None, 1 / math.sqrt(D), bs)
    assert ((lse.double() - l).abs() <= 1e-4).all()
    assert ((out.double() - o).abs() <= 2.0**-8 * o.abs() + 2.0**-10 * spread).all()
    assert ((acc[:, :, t0:n].double() - w).abs() <= 1e-3 * w).all() and float(acc[:, :, :t0].abs().max()) == 0
    assert int(st.item()) == 0


# ------------------------------------------------------------------ eviction

EVICT = [  # lens, Hkv, bs, cap, keep, sink, recent, dst capacity
    ([1], 1, 16, 1, 1, 0, 0, 1),
    ([0, 5, 40], 2, 16, 41, 7, 1, 2, 20),
    ([100, 64, 333], 2, 32, 333, 64, 4, 16, 64),
    ([700, 300], 1, 64, 701, 255, 0, 0, 300),
    ([900], 3, 128, 900, 400, 100, 300, 401),       # nothing to choose
    ([5000, 4097], 2, 16, 5001, 1000, 16, 64, 1024),  # 8 keys a thread
    ([9000, 33000], 1, 32, 33000, 4000, 4, 500, 4000),  # keys in shared memory, and in the scratch rows
]


def spread_weights(shape, seed):
    a = torch.rand(shape, generator=gen(seed), device="cuda") ** 8
    return a * (torch.rand(shape, generator=gen(seed + 1), device="cuda") < 0.6)


@pytest.mark.parametrize("int4", [True, False], ids=["int4", "bf16"])
@pytest.mark.parametrize("paged", [False, True], ids=["flat", "paged"])
@pytest.mark.parametrize("case", EVICT, ids=lambda e: f"bs{e[2]}_cap{e[3]}_keep{e[4]}")
def test_evict(case, paged, int4):
    lens, Hkv, bs, cap, keep, sink, recent, cap2 = case
    c = Cache(lens, Hkv, bs, cap, paged, 111)
    acc = spread_weights((c.B, Hkv, cap), 112)
    check_evict(c, acc, keep, sink, recent, cap2, paged, int4)


def check_evict(c, acc, keep, sink, recent, cap2, paged, int4):
    kv = c.stored() if int4 else c.bf16()
    c2 = Cache([0] * c.B, c.Hkv, c.bs, cap2, paged, 113)  # the destination: noise or NaN everywhere
    dst = c2.empty4() if int4 else c2.bf16()
    old = [t.clone() for t in ((dst.k, dst.v, dst.k_scales, dst.v_scales) if int4 else (dst.k, dst.v))]
    dst_acc = torch.full((c.B, c.Hkv, cap2), math.nan, device="cuda")
    dst_lens = torch.full((c.B,), -1, dtype=torch.int32, device="cuda")
    sel = torch.full((c.B, c.Hkv, keep), -9, dtype=torch.int32, device="cuda")
    means = torch.full((c.B, c.Hkv, c2.nb, D), 5.0, device="cuda")
    st = status()
    ws = kin.alloc_kv_evict_workspace(c.dims(), keep)
    kin.kin_kv_evict(c.dims(), kv, acc, c.seq, keep, sink, recent, c2.dims(), dst, dst_acc, dst_lens, ws, block_means=means,
                     sel_tokens=sel, dev_status=st)
    assert int(st.item()) == 0
    want_lens = [min(n, keep) for n in c.lens]
    assert dst_lens.tolist() == want_lens
    new = (dst.k, dst.v, dst.k_scales, dst.v_scales) if int4 else (dst.k, dst.v)
    src = (kv.k, kv.v, kv.k_scales, kv.v_scales) if int4 else (kv.k, kv.v)
    raw = (lambda t: t.view(torch.int16) if t.dtype == torch.bfloat16 else t)
    held = c.held()[0].float() if int4 else c.k.float()
    moved = torch.zeros((c.B, c.Hkv, cap2, D), device="cuda")
    got, was, frm = [[raw(side.logical(t)) for t in ts] for side, ts in ((c2, new), (c2, old), (c, src))]
    for b, n in enumerate(c.lens):
        m = want_lens[b]
        for h in range(c.Hkv):
            tok = ref.kept(acc[b, h].tolist(), n, keep, sink, recent)
            assert sel[b, h].tolist() == tok + [-1] * (keep - m)
            at = torch.tensor(tok, dtype=torch.long, device="cuda")
            assert torch.equal(dst_acc[b, h, :m].nan_to_num(-1), acc[b, h, at].nan_to_num(-1)) and (dst_acc[b, h, m:] == 0).all()
            for x, y, z in zip(got, was, frm):
                assert torch.equal(x[b, h, :m], z[b, h, at]) and torch.equal(x[b, h, m:], y[b, h, m:])
            moved[b, h, :m] = held[b, h, at]
    want = ref.block_means(moved, want_lens, c.bs)
    assert torch.equal(means, torch.where(want.isnan(), torch.full_like(want, 5.0), want))
    # the same move without the optional outputs
    dst2 = c2.empty4() if int4 else c2.bf16()
    kin.kin_kv_evict(c.dims(), kv, acc, c.seq, keep, sink, recent, c2.dims(), dst2, None, dst_lens, ws, dev_status=st)
    assert torch.equal(raw(dst2.k), raw(dst.k)) and torch.equal(raw(dst2.v), raw(dst.v)) and int(st.item()) == 0


@pytest.mark.parametrize("n", [300, 5000, 9000])
@pytest.mark.parametrize("kind", ["equal", "nan_inf", "signed_zero"])
def test_evict_awkward_weights(kind, n):
    c = Cache([n], 1, 16, n, False, 121)
    acc = torch.full((1, 1, n), 0.25, device="cuda")
    if kind == "nan_inf":
        acc = spread_weights((1, 1, n), 122)
        acc[0, 0, 5::7], acc[0, 0, 11::97], acc[0, 0, 13::50] = math.nan, math.inf, -math.inf
    elif kind == "signed_zero":
        acc.zero_()
        acc[0, 0, ::2] = -0.0
        acc[0, 0, 100:110] = 1e-42
    check_evict(c, acc, n // 3, 2, 9, n // 3, False, True)


def test_evict_within_one_pool_and_bad_data():
    """To other pages of the same pool; a bad source page's rows stay as they
    were, a bad length keeps nothing."""
    c = Cache([60, 60], 2, 16, 64, True, 131)
    kv = c.stored()
    free = 2 * 2  # two pages a sequence
    big = [torch.cat((t, torch.full((free,) + t.shape[1:], 0, dtype=t.dtype, device="cuda"))) for t in (kv.k, kv.v, kv.k_scales, kv.v_scales)]
    table2 = torch.arange(c.pages, c.pages + free, dtype=torch.int32, device="cuda").view(2, 2)
    src = kin.KvCache(*big, block_table=c.table)
    dst = kin.KvCache(*big, block_table=table2)
    acc = spread_weights((2, 2, 64), 132)
    d2 = kin.make_dims(2, 2, 2, D, 16, 30)
    lens2, st = torch.zeros(2, dtype=torch.int32, device="cuda"), status()
    sel = torch.zeros((2, 2, 30), dtype=torch.int32, device="cuda")
    ws = kin.alloc_kv_evict_workspace(c.dims(), 30)
    kin.kin_kv_evict(c.dims(), src, acc, c.seq, 30, 1, 5, d2, dst, None, lens2, ws, sel_tokens=sel, dev_status=st)
    assert int(st.item()) == 0 and lens2.tolist() == [30, 30]
    rows, frm = ref.from_pool(big[0], table2, 30), ref.from_pool(kv.k, c.table, 64)
    for b in range(2):
        for h in range(2):
            assert torch.equal(rows[b, h], frm[b, h, sel[b, h].long()])
    bad = c.table.clone()
    bad[0, 0] = 1 << 20
    big[0][c.pages:] = 77
    kin.kin_kv_evict(c.dims(), kin.KvCache(*big, block_table=bad), acc, ints([60, 65]), 30, 1, 5, d2, dst, None, lens2, ws,
                     sel_tokens=sel, dev_status=st)
    assert int(st.item()) == 5 and lens2.tolist() == [30, 0]
    rows = ref.from_pool(big[0], table2, 30)
    for h in range(2):
        tok = sel[0, h].long()
        gone = tok < 16
        assert (rows[0, h][gone] == 77).all() and torch.equal(rows[0, h][~gone], frm[0, h, tok[~gone]])
    assert (rows[1] == 77).all() and (sel[1] == -1).all()


# ------------------------------------------------------------ used together

def decode(c, g, int4, steps, budget, use_graph=False):
    """Steps of a server: append, select, attend with weights, and an eviction
    whenever the cache is full; every step against the plain form."""
    B, Hkv, bs = c.B, c.Hkv, c.bs
    room = budget + 2 * bs
    d = kin.make_dims(B, Hkv, Hkv * g, D, bs, room)
    st = status()
    nb = -(-room // bs)
    sides = []
    for _ in range(2):
        kv = kin.alloc_kv4(d)
        sides.append(dict(kv=kv, means=torch.zeros((B, Hkv, nb, D), device="cuda"), acc=torch.zeros((B, Hkv, room), device="cuda"),
                          lens=torch.zeros(B, dtype=torch.int32, device="cuda")))
    # the model of it: logical rows a pair
    keys = [[[] for _ in range(Hkv)] for _ in range(B)]
    a = sides[0]
    k_sel = 4
    ws = kin.alloc_kv_attn_workspace(d, k_sel, acc=True)
    ews = kin.alloc_kv_evict_workspace(d, budget)
    n = 0
    for step in range(steps):
        kn, vn = rows16(1000 + step, B, Hkv, 1, D), rows16(2000 + step, B, Hkv, 1, D)
        q = rows16(3000 + step, B, Hkv * g, D)
        kin.kin_kv4_append(d, a["kv"], a["means"], a["lens"], a["lens"], kn, vn, 1, st)
        n += 1
        for b in range(B):
            for h in range(Hkv):
                keys[b][h].append((kn[b, h, 0], vn[b, h, 0]))
        sel = torch.empty((B, Hkv, k_sel), dtype=torch.int32, device="cuda")
        cnt = torch.empty((B, Hkv), dtype=torch.int32, device="cuda")
        out, lse = torch.empty_like(q), torch.empty((B, Hkv * g), device="cuda")
        kin.kin_block_topk_select(d, q, a["means"], a["lens"], k_sel, sel, cnt, ws, st)
        before = a["acc"].clone()
        kin.kin_kv_decode_attn(d, q, a["kv"], a["lens"], sel, cnt, k_sel, 0.0, out, lse, ws, acc=a["acc"], dev_status=st)
        now = Cache([n] * B, Hkv, bs, n, False, 1)
        now.k = torch.stack([torch.stack([torch.stack([r[0] for r in keys[b][h]]) for h in range(Hkv)]) for b in range(B)])
        now.v = torch.stack([torch.stack([torch.stack([r[1] for r in keys[b][h]]) for h in range(Hkv)]) for b in range(B)])
        check_attention(now, q, out, lse, a["acc"][:, :, :n].contiguous(), before[:, :, :n].contiguous(), True, sel.tolist())
        assert torch.equal(a["means"][:, :, : -(-n // bs)], ref.block_means(now.held()[0].float(), now.lens, bs))
        if n == room:
            z = sides[1]
            toks = torch.empty((B, Hkv, budget), dtype=torch.int32, device="cuda")
            kin.kin_kv_evict(d, a["kv"], a["acc"], a["lens"], budget, 2, bs, d, z["kv"], z["acc"], z["lens"], ews,
                             block_means=z["means"], sel_tokens=toks, dev_status=st)
            for b in range(B):
                for h in range(Hkv):
                    want = ref.kept(a["acc"][b, h].tolist(), n, budget, 2, bs)
                    assert toks[b, h].tolist() == want
                    keys[b][h] = [keys[b][h][t] for t in want]
            sides.reverse()
            a = sides[0]
            n = budget
            assert a["lens"].tolist() == [n] * B
    assert int(st.item()) == 0


def test_decode_with_eviction():
    decode(Cache([0, 0], 2, 16, 1, False, 1), 4, True, 90, 40)


def test_captured_and_replayed():
    """A captured step (append, attention with weights, eviction) gives, each
    time it is replayed on new inputs, what eager calls give; two graphs with
    their own workspaces run side by side on two streams."""
    def setup(seed):
        c = Cache([200, 131], 2, 16, 232, False, seed)
        s = dict(c=c, kv=c.stored(), seq=c.seq.clone(), new=torch.zeros_like(c.seq), q=rows16(seed + 7, 2, 8, D), d=c.dims(4),
                 acc=spread_weights((2, 2, 232), seed + 8), kn=rows16(seed + 9, 2, 2, 3, D), means=torch.zeros((2, 2, 15, D), device="cuda"),
                 d2=kin.make_dims(2, 2, 8, D, 16, 64), st=status())
        s["ws"], s["ews"] = kin.alloc_kv_attn_workspace(s["d"], 0, acc=True), kin.alloc_kv_evict_workspace(s["d"], 50)
        s["kv2"] = kin.alloc_kv4(s["d2"])
        s["out"], s["lse"] = torch.zeros_like(s["q"]), torch.zeros((2, 8), device="cuda")
        s["acc2"], s["lens2"] = torch.zeros((2, 2, 64), device="cuda"), torch.zeros_like(c.seq)
        return s

    def step(s):
        kin.kin_kv4_append(s["d"], s["kv"], s["means"], s["seq"], s["new"], s["kn"], s["kn"], 3, s["st"])
        kin.kin_kv_decode_attn(s["d"], s["q"], s["kv"], s["new"], None, None, 0, 0.0, s["out"], s["lse"], s["ws"], acc=s["acc"],
                               dev_status=s["st"])
        kin.kin_kv_evict(s["d"], s["kv"], s["acc"], s["new"], 50, 2, 10, s["d2"], s["kv2"], s["acc2"], s["lens2"], s["ews"],
                         dev_status=s["st"])

    def results(s):
        return [t.clone() for t in (s["out"], s["lse"], s["acc"], s["acc2"], s["lens2"], s["new"], s["kv2"].k, s["kv2"].v_scales, s["means"])]

    def fresh(s, seed):
        s["q"].copy_(rows16(seed, 2, 8, D))
        s["kn"].copy_(rows16(seed + 1, 2, 2, 3, D))
        s["acc"].copy_(spread_weights((2, 2, 232), seed + 2))

    eager, graphs = [setup(1), setup(301)], [setup(1), setup(301)]
    for s in eager + graphs:
        step(s)
    streams, caps = [torch.cuda.Stream() for _ in range(2)], []
    torch.cuda.synchronize()
    for s, stream in zip(graphs, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            step(s)
        caps.append(g)
    for seed in (500, 600, 700):
        for i, s in enumerate(eager):
            fresh(s, seed + 10 * i)
            step(s)
        for i, s in enumerate(graphs):
            fresh(s, seed + 10 * i)
        torch.cuda.synchronize()
        for g, stream in zip(caps, streams):
            with torch.cuda.stream(stream):
                g.replay()
        torch.cuda.synchronize()
        for s, e in zip(graphs, eager):
            assert all(torch.equal(x, y) for x, y in zip(results(s), results(e)))
            assert int(s["st"].item()) == 0 and int(e["st"].item()) == 0


def test_on_another_stream():
    """Calls go to the stream they are given, whatever stream is current."""
    c = Cache([500], 2, 16, 500, False, 141)
    q = rows16(142, 1, 4, D)
    d = c.dims(2)
    out, lse = torch.zeros_like(q), torch.zeros((1, 4), device="cuda")
    s = torch.cuda.Stream()
    ws = kin.alloc_kv_attn_workspace(d, 0)
    kv, src = c.empty4(), c.bf16()
    torch.cuda.synchronize()
    kin.kin_kv4_store(d, src, kv, c.seq, stream=s)
    with torch.cuda.stream(s):
        kin.kin_kv_decode_attn(d, q, kv, c.seq, None, None, 0, 0.0, out, lse, ws)
    s.synchronize()
    check_attention(c, q, out, lse, None, None, True)


def test_binding_refuses_short_and_foreign_tensors():
    c = Cache([30], 1, 16, 40, False, 151)
    kv, d = c.stored(), c.dims(2)
    q = rows16(152, 1, 2, D)
    out, lse, ws = torch.empty_like(q), torch.empty((1, 2), device="cuda"), kin.alloc_kv_attn_workspace(d, 0, acc=True)
    call = lambda kv=kv, acc=None, q=q: kin.kin_kv_decode_attn(d, q, kv, c.seq, None, None, 0, 0.0, out, lse, ws, acc=acc)  # noqa: E731
    for bad in (kin.KvCache(kv.k[..., :32], kv.v, kv.k_scales, kv.v_scales), kin.KvCache(kv.k.cpu(), kv.v, kv.k_scales, kv.v_scales),
                kin.KvCache(kv.k, kv.v, kv.k_scales[:, :, :39].contiguous(), kv.v_scales),
                kin.KvCache(kv.k, kv.v.to(torch.int32), kv.k_scales, kv.v_scales)):
        with pytest.raises(ValueError):
            call(kv=bad)
    with pytest.raises(ValueError):
        call(acc=torch.zeros((1, 1, 39), device="cuda"))
    with pytest.raises(ValueError):
        call(q=q[:, :1])
    with pytest.raises(kin.KinError):
        kin.kin_kv4_load(d, c.bf16(), c.seq, c.k.clone(), c.v.clone())  # not a 4-bit cache


@pytest.mark.parametrize("int4", [True, False], ids=["int4", "bf16"])
@pytest.mark.parametrize("lens, Hkv, bs, cap", [
    ([113_003], 2, 16, 113_100),          # few pairs, a range for every resident CTA
    ([16_000, 1, 0, 4_097], 24, 16, 16_001),   # 96 pairs: ranges of 250 tiles, cut anew for the short ones
    ([17, 7_000], 4, 64, 131_072),        # short sequences in a large cache
], ids=["one_long", "long_ranges", "large_cache"])
def test_long_dense_ranges(lens, Hkv, bs, cap, int4):
    """Every token of sequences whose ranges hold up to 256 tiles, 64 a warp:
    23 * 64 * 2^-23 < 2^-12 of sum p s, twice the bound above.  Sums: a thread
    adds 2 weights a tile and head and 222 ranges at most are merged, each
    addition to 2^-24: 350 * 2^-24 < 2^-15.5.  delta holds 2^-22 * 64 = 2^-16
    for a scaling that takes 2^-19 (logits below 32); with 2^-20 (1 + |lse|),
    lse > 9 where that many ranges meet, the lse has 2^-15.3 for it, and a
    weight, with delta twice, 2^-15."""
    c = Cache(lens, Hkv, bs, cap, False, 171)
    g, st = 2, status()
    q = rows16(172, c.B, Hkv * g, D)
    d = c.dims(g)
    kv = c.stored() if int4 else c.bf16()
    out, lse = torch.full_like(q, 7.0), torch.full((c.B, Hkv * g), 7.0, device="cuda")
    acc = torch.zeros((c.B, Hkv, cap), device="cuda")
    ws = kin.alloc_kv_attn_workspace(d, 0, acc=True)
    kin.kin_kv_decode_attn(d, q, kv, c.seq, None, None, 0, 0.0, out, lse, ws, acc=acc, dev_status=st)
    assert int(st.item()) == (5 if 0 in lens else 0)
    check_attention(c, q, out, lse, acc, None, int4, tiles=64)
