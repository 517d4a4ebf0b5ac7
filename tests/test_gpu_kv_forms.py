"""Forms of the 4-bit cache's and the eviction's calls: every layout of the
block means beside append and eviction, batches of more (sequence, KV head)
pairs than SMs (whose tokens a kernel of 512 threads selects, two on an SM),
weights as a generation leaves them, and decode steps over a bf16 cache that
evicts.  Everything compared here is equal but the attention, whose tolerances
are test_gpu_kv's."""
import math

import pytest
import torch

import block_top_sparse_kin_b200 as kin
import kin_kv_ref as ref
from test_gpu_kv import Cache, D, check_attention, check_evict, gen, ints, rows16, spread_weights, status

pytestmark = pytest.mark.gpu

KINDS = ["bf16", "dual", "fp32_page", "bf16_page", "dual_page"]


class Means:
    """A block-means buffer of one kind for cache c, filled with a byte that no mean writes by itself."""

    def __init__(self, c, kind):
        self.c, self.kind, self.page = c, kind, kind.endswith("page")
        self.rows = c.pages * c.Hkv if self.page else c.B * c.Hkv * c.nb
        if kind.startswith("dual"):
            self.t = kin.alloc_dual_page_means(c.dims(), c.pages) if self.page else kin.alloc_dual_means(c.dims())
        else:
            shape = (c.pages, c.Hkv, D) if self.page else (c.B, c.Hkv, c.nb, D)
            self.t = torch.zeros(shape, dtype=torch.float32 if kind.startswith("fp32") else torch.bfloat16, device="cuda")
        self.t.view(torch.uint8).fill_(0x55)

    def logical(self, x):
        """Rows [rows, w] as [B, Hkv, nb, w]."""
        c = self.c
        return x.view(c.pages, c.Hkv, -1)[c.table.long()].transpose(1, 2) if self.page else x.view(c.B, c.Hkv, c.nb, -1)

    def check(self, want):
        """Equal to the fp32 means want [B, Hkv, nb, D], untouched where they are NaN."""
        live = ~want.isnan()
        none = torch.full((1,), 0x55555555, dtype=torch.int32, device="cuda").view(torch.float32)
        n = self.rows
        if self.kind.startswith("dual"):
            raw = self.t.flatten()
            parts = [raw[: 4 * n * D].view(torch.float32).view(n, D), raw[4 * n * D: 6 * n * D].view(torch.bfloat16).view(n, D)]
            rad = self.logical(raw[6 * n * D: 6 * n * D + 4 * n].view(torch.float32).view(n, 1))[..., 0]
            ok = live.all(-1)
            miss = (want.double() - want.to(torch.bfloat16).double()).norm(dim=-1)
            assert (rad[ok] >= miss[ok]).all() and (rad[ok] <= 1.01 * miss[ok] + 2**-17 * want[ok].norm(dim=-1)).all()
            assert (rad[~ok] == none).all()
        else:
            parts = [self.t.view(n, D)]
        for x in parts:
            got = self.logical(x)
            assert torch.equal(got[live], want.to(x.dtype)[live])
            assert (got[~live] == none.view(x.dtype)[0]).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n_new", [1, 40])
def test_append_with_other_means(kind, n_new):
    """The means after an append are those of the rows held: of a new block, a block begun before, and the others as they were."""
    before = [0, 1, 31, 64, 77]
    c = Cache([n + n_new for n in before], 2, 32, 77 + n_new + 40, True, 301)
    kv, st, lens = c.empty4(), status(), ints(before)
    means = Means(c, kind)
    kin.kin_kv4_store(c.dims(), c.bf16(), kv, lens, means.t, st, per_page=means.page)
    new = [torch.stack([x[b, :, n: n + n_new] for b, n in enumerate(before)]).contiguous() for x in (c.k, c.v)]
    kin.kin_kv4_append(c.dims(), kv, means.t, lens, lens, *new, n_new, st, per_page=means.page)
    assert int(st.item()) == 0 and lens.tolist() == c.lens
    c.check4(kv)
    means.check(ref.block_means(c.held()[0].float(), c.lens, c.bs))


def test_append_into_a_shared_pool():
    """Two sequences that share a prompt's pages, per-page means: an append goes to each one's own last page."""
    c = Cache([64, 64], 2, 32, 96, True, 311)
    c.table[1, :2] = c.table[0, :2]
    c.k[1], c.v[1] = c.k[0], c.v[0]
    kv, st, means = c.empty4(), status(), Means(c, "fp32_page")
    kin.kin_kv4_store(c.dims(), c.bf16(), kv, c.seq, means.t, st, per_page=True)
    new = rows16(312, 2, 2, 5, D)
    kin.kin_kv4_append(c.dims(), kv, means.t, c.seq, c.seq, new, new, 5, st, per_page=True)
    c.k[:, :, 64:69], c.v[:, :, 64:69], c.lens = new, new, [69, 69]
    assert int(st.item()) == 0 and c.seq.tolist() == c.lens
    c.check4(kv)
    means.check(ref.block_means(c.held()[0].float(), c.lens, c.bs))


@pytest.mark.parametrize("int4", [True, False], ids=["int4", "bf16"])
@pytest.mark.parametrize("kind", KINDS)
def test_evict_with_other_means(kind, int4):
    c = Cache([300, 40, 0], 2, 16, 301, True, 321)
    acc = spread_weights((3, 2, 301), 322)
    kv, st = c.stored() if int4 else c.bf16(), status()
    c2 = Cache([0, 0, 0], 2, 16, 90, True, 323)
    dst, means = c2.empty4() if int4 else c2.bf16(), Means(c2, kind)
    sel, lens = torch.empty((3, 2, 75), dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    kin.kin_kv_evict(c.dims(), kv, acc, c.seq, 75, 3, 20, c2.dims(), dst, None, lens, kin.alloc_kv_evict_workspace(c.dims(), 75),
                     block_means=means.t, sel_tokens=sel, dev_status=st, per_page=means.page)
    assert int(st.item()) == 0 and lens.tolist() == [75, 40, 0]
    held = c.held()[0].float() if int4 else c.k.float()
    moved = torch.zeros((3, 2, 90, D), device="cuda")
    for b in range(3):
        for h in range(2):
            tok = ref.kept(acc[b, h].tolist(), c.lens[b], 75, 3, 20)
            assert sel[b, h].tolist() == tok + [-1] * (75 - len(tok))
            moved[b, h, : len(tok)] = held[b, h, tok]
    means.check(ref.block_means(moved, lens.tolist(), 16))


def generation_weights(shape, seed):
    """Weights as long generations leave them, another kind for each sequence:
    log-normal and Pareto sums (most of them in a sliver of the range), many
    equal ones, NaN and infinities among them, and rand^8."""
    z = torch.randn(shape, generator=gen(seed), device="cuda")
    u = torch.rand(shape, generator=gen(seed + 1), device="cuda").clamp(min=1e-7)
    acc = spread_weights(shape, seed + 2)
    for b in range(shape[0]):
        if b % 5 == 0:
            acc[b] = torch.exp(2 * z[b])
        elif b % 5 == 1:
            acc[b] = u[b].reciprocal()
        elif b % 5 == 2:
            acc[b] = torch.floor(4 * u[b]) / 8
        elif b % 5 == 3:
            acc[b, :, 3::7], acc[b, :, 5::91], acc[b, :, 6::97] = math.nan, math.inf, -math.inf
    return acc


@pytest.mark.parametrize("keep, sink, recent", [(700, 4, 100), (140, 40, 100)], ids=["some", "nothing_free"])
@pytest.mark.parametrize("cap", [2050, 4100, 16384, 16385])
def test_evict_of_more_pairs_than_sms(cap, keep, sink, recent):
    """More pairs than SMs: up to 16384 tokens two CTAs of 512 threads an SM,
    with 4 and 8 keys a thread and keys in memory on both sides of each switch;
    beyond, 1024 threads."""
    lens = [cap, 1, keep, keep + 1, 2047, 2048, 2049, 4095, 4096, 4097, 8191, 8192, 8193, 16383, 16384]
    lens = [n for n in lens if n <= cap][:10] + [cap - 3, cap - 2, cap - 1]
    c = Cache(lens, 16, 16, cap, False, 331)
    assert c.B * c.Hkv > torch.cuda.get_device_properties(0).multi_processor_count
    check_evict(c, generation_weights((c.B, 16, cap), 332), keep, sink, recent, keep + 9, False, cap == 4100)


@pytest.mark.parametrize("n", [3000, 12000, 40000])
def test_evict_by_generation_weights(n):
    """The same kinds of weights with one CTA of 1024 threads a pair: keys in registers, shared memory and scratch."""
    c = Cache([n] * 5, 1, 32, n, False, 341)
    check_evict(c, generation_weights((5, 1, n), 342), n // 8, 4, 64, n // 8 + 1, False, True)


def test_decode_with_eviction_over_bf16_rows():
    """Steps of a server over a bf16 cache: append, select, attend with
    weights, and an eviction whenever the cache is full; every step against the
    plain form."""
    B, Hkv, bs, g, budget, k_sel = 2, 2, 16, 4, 40, 4
    room = budget + 2 * bs
    nb = -(-room // bs)
    d, st = kin.make_dims(B, Hkv, Hkv * g, D, bs, room), status()
    sides = [dict(kv=kin.KvCache(*(torch.zeros((B, Hkv, room, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))),
                  means=torch.zeros((B, Hkv, nb, D), device="cuda"), acc=torch.zeros((B, Hkv, room), device="cuda"),
                  lens=torch.zeros(B, dtype=torch.int32, device="cuda")) for _ in range(2)]
    ws, ews = kin.alloc_kv_attn_workspace(d, k_sel, acc=True), kin.alloc_kv_evict_workspace(d, budget)
    k, v = (torch.zeros((B, Hkv, room, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))  # what it should hold
    n, evictions = 0, 0
    for step in range(110):
        a = sides[0]
        kn, vn, q = rows16(5000 + step, B, Hkv, 1, D), rows16(6000 + step, B, Hkv, 1, D), rows16(7000 + step, B, Hkv * g, D)
        kin.kin_block_means_update(d, a["kv"].k, a["kv"].v, a["means"], a["lens"], kn, vn, 1, st)
        k[:, :, n], v[:, :, n] = kn[:, :, 0], vn[:, :, 0]
        n += 1
        sel = torch.empty((B, Hkv, k_sel), dtype=torch.int32, device="cuda")
        cnt = torch.empty((B, Hkv), dtype=torch.int32, device="cuda")
        out, lse, before = torch.empty_like(q), torch.empty((B, Hkv * g), device="cuda"), a["acc"].clone()
        kin.kin_block_topk_select(d, q, a["means"], a["lens"], k_sel, sel, cnt, ws, st)
        kin.kin_kv_decode_attn(d, q, a["kv"], a["lens"], sel, cnt, k_sel, 0.0, out, lse, ws, acc=a["acc"], dev_status=st)
        now = Cache([n] * B, Hkv, bs, n, False, 1)
        now.k, now.v = k[:, :, :n].clone(), v[:, :, :n].clone()
        check_attention(now, q, out, lse, a["acc"][:, :, :n].contiguous(), before[:, :, :n].contiguous(), False, sel.tolist())
        assert torch.equal(a["means"][:, :, : -(-n // bs)], ref.block_means(now.k.float(), now.lens, bs))
        if n == room:
            z = sides[1]
            kin.kin_kv_evict(d, a["kv"], a["acc"], a["lens"], budget, 2, bs, d, z["kv"], z["acc"], z["lens"], ews,
                             block_means=z["means"], dev_status=st)
            for b in range(B):
                for h in range(Hkv):
                    tok = ref.kept(a["acc"][b, h].tolist(), n, budget, 2, bs)
                    k[b, h, :budget], v[b, h, :budget] = k[b, h, tok], v[b, h, tok]
            n, evictions = budget, evictions + 1
            sides.reverse()
            assert sides[0]["lens"].tolist() == [n] * B and torch.equal(sides[0]["kv"].k[:, :, :n], k[:, :, :n])
    assert int(st.item()) == 0 and evictions == 2
