"""The calls on 4-bit caches, attention weights and eviction, without a GPU:
their host checks, workspace sizes and the row format."""
import ctypes

import pytest
import torch

import block_top_sparse_kin_b200 as kin
import kin_kv_ref as ref

FAKE = 1 << 20  # aligned, never dereferenced: every call below fails its host checks
INVALID, WORKSPACE, CAPACITY = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    return kin.load_library()


def dims(B=2, Hkv=2, Hq=8, D=128, bs=16, L=256):
    return kin.make_dims(B, Hkv, Hq, D, bs, L)


def kv4(at=FAKE, **kw):
    f = dict(format=kin.KIN_KV_INT4, num_pages=0, block_table=None, k=at, v=at + 4096, k_scales=at, v_scales=at)
    f.update(kw)
    return kin.kin_kv(*f.values())


def kv16(at=FAKE, **kw):
    return kv4(at, **{**dict(format=kin.KIN_KV_BF16, k_scales=None, v_scales=None), **kw})


BAD_KV4 = [kv4(format=2), kv4(k=None), kv4(v=None), kv4(k_scales=None), kv4(v_scales=None), kv4(k=FAKE + 8), kv4(v=FAKE + 2),
           kv4(k_scales=FAKE + 8), kv4(block_table=FAKE, num_pages=0)]


def test_store_refuses(lib):
    def call(d=dims(), src=kv16(), dst=kv4(), lens=FAKE, means=FAKE, dtype=0):
        return lib.kin_kv4_store(ctypes.byref(d), ctypes.byref(src), ctypes.byref(dst), lens, means, dtype, None, None)
    assert call(d=dims(D=64)) == INVALID
    assert call(src=kv4()) == INVALID and call(dst=kv16()) == INVALID
    for bad in BAD_KV4:
        assert call(dst=bad) == INVALID
    assert call(src=kv16(k=None)) == INVALID
    assert call(src=kv16(block_table=FAKE, num_pages=-1)) == INVALID
    assert call(lens=None) == INVALID
    assert call(dtype=3) == INVALID and call(means=FAKE + 4) == INVALID
    assert call(dtype=kin.KIN_MEANS_PER_PAGE) == INVALID  # per page needs a table
    assert call(d=dims(L=16 * 32768 + 1)) == CAPACITY
    assert lib.kin_kv4_store(ctypes.byref(dims()), None, ctypes.byref(kv4()), FAKE, None, 0, None, None) == INVALID


def test_append_refuses(lib):
    def call(kv=kv4(), lens=FAKE, new=FAKE, k=FAKE, v=FAKE, n=1, means=None, dtype=0):
        return lib.kin_kv4_append(ctypes.byref(dims()), ctypes.byref(kv), means, dtype, lens, new, k, v, n, None, None)
    assert call(n=-1) == INVALID and call(n=257) == CAPACITY
    assert call(kv=kv16()) == INVALID
    for bad in BAD_KV4:
        assert call(kv=bad) == INVALID
    assert call(lens=None) == INVALID and call(new=None) == INVALID
    assert call(k=None) == INVALID and call(v=FAKE + 8) == INVALID
    assert call(means=FAKE, dtype=7) == INVALID
    assert call(n=0) == 0  # nothing to do in place


def test_load_refuses(lib):
    def call(kv=kv4(), lens=FAKE, n=4, k=FAKE, v=FAKE):
        return lib.kin_kv4_load(ctypes.byref(dims()), ctypes.byref(kv), lens, None, n, k, v, None, None)
    assert call(n=-1) == INVALID and call(n=257) == CAPACITY and call(n=0) == 0
    assert call(kv=kv16()) == INVALID and call(kv=BAD_KV4[0]) == INVALID
    assert call(lens=None) == INVALID and call(k=None) == INVALID and call(v=FAKE + 4) == INVALID


def test_attention_refuses(lib):
    def call(kv=kv4(), q=FAKE, lens=FAKE, sel=FAKE, cnt=FAKE, k=8, scale=0.0, out=FAKE, acc=None, ws=FAKE, n=1 << 30):
        return lib.kin_kv_decode_attn(ctypes.byref(dims()), q, ctypes.byref(kv), lens, sel, cnt, k, scale, out, None,
                                      acc, ws, n, None, None)
    for bad in BAD_KV4:
        assert call(kv=bad) == INVALID
    assert call(k=1) == INVALID and call(k=-2) == INVALID
    assert call(sel=None) == INVALID and call(cnt=None) == INVALID and call(k=0) == INVALID
    assert call(k=0, sel=None) == INVALID
    assert call(q=None) == INVALID and call(lens=None) == INVALID and call(out=FAKE + 2) == INVALID
    assert call(scale=float("nan")) == INVALID and call(scale=float("inf")) == INVALID
    assert call(ws=None) == WORKSPACE and call(ws=FAKE + 16) == WORKSPACE
    d = dims()
    need = kin.kin_kv_attn_workspace_bytes(d, 8)
    more = kin.kin_kv_attn_workspace_bytes(d, 8, True)
    assert more >= need + 4 * 8 * 16 * 4 * 4  # a logit per (pair, kept token, head)
    assert call(n=need - 1) == WORKSPACE and call(acc=FAKE, n=need) == WORKSPACE


def test_workspace_bytes(lib):
    assert kin.kin_kv_attn_workspace_bytes(dims(), 1) == 0 and kin.kin_kv_attn_workspace_bytes(dims(), -1) == 0
    assert kin.kin_kv_attn_workspace_bytes(dims(D=64), 8) == 0
    # one buffer serves the select as well
    for k in (2, 8, 16, 200):
        assert kin.kin_kv_attn_workspace_bytes(dims(), k) >= kin.kin_workspace_bytes(dims(), k)
    assert kin.kin_kv_attn_workspace_bytes(dims(), 0) > 0
    assert kin.kin_kv_evict_workspace_bytes(dims(), 0) == 0 and kin.kin_kv_evict_workspace_bytes(dims(), 257) == 0
    assert kin.kin_kv_evict_workspace_bytes(dims(), 100) >= 4 * 100 * 4
    long = dims(L=40000)  # beyond the shared-memory keys: a key row a pair as well
    assert kin.kin_kv_evict_workspace_bytes(long, 100) >= 4 * 40000 * 4


def test_evict_refuses(lib):
    far = FAKE + (1 << 24)

    def call(kv=kv4(), d=dims(), dd=dims(L=128), dst=kv4(far), acc=FAKE, lens=FAKE, keep=64, sink=4, recent=16, dacc=None,
             dlens=FAKE + 64, means=None, dtype=0, ws=FAKE, n=1 << 30):
        return lib.kin_kv_evict(ctypes.byref(d), ctypes.byref(kv), acc, lens, keep, sink, recent, ctypes.byref(dd),
                                ctypes.byref(dst), dacc, dlens, means, dtype, None, ws, n, None, None)
    for bad in BAD_KV4:
        assert call(kv=bad) == INVALID
    assert call(dst=kv16(far)) == INVALID  # one format on both sides
    assert call(keep=0) == INVALID and call(sink=-1) == INVALID and call(recent=-1) == INVALID
    assert call(sink=40, recent=40) == INVALID
    assert call(sink=2**31 - 1, recent=2**31 - 1) == INVALID
    assert call(keep=129) == CAPACITY and call(keep=257, dd=dims(L=512)) == CAPACITY
    for other in (dims(B=1, L=128), dims(Hkv=4, L=128), dims(Hq=4, L=128), dims(bs=32, L=128)):
        assert call(dd=other) == INVALID
    assert call(dst=kv4()) == INVALID  # in place
    assert call(dst=kv4(FAKE, block_table=FAKE, num_pages=4)) == INVALID  # a pool laid over the contiguous cache
    t = dict(block_table=FAKE, num_pages=4)
    assert call(kv=kv4(**t), dst=kv4(**t)) == INVALID  # the same pages
    assert call(acc=None) == INVALID and call(lens=None) == INVALID and call(dlens=None) == INVALID
    assert call(dacc=FAKE) == INVALID and call(dlens=FAKE) == INVALID  # the source's own
    assert call(means=FAKE, dtype=9) == INVALID
    assert call(ws=None) == WORKSPACE and call(n=64) == WORKSPACE


def test_binding_refuses_a_half_given_cache():
    t = torch.zeros(4, dtype=torch.uint8)
    with pytest.raises(ValueError):
        kin.KvCache(t, t, k_scales=t)
    with pytest.raises(ValueError):
        kin.alloc_kv4(dims(), num_pages=4, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        kin.kin_kv4_load(dims(), kin.alloc_kv4(dims(), device="cpu"), t, t[None, None, None], t)


def test_alloc_shapes():
    c = kin.alloc_kv4(dims(L=100), device="cpu")
    assert c.int4 and c.k.shape == (2, 2, 100, 64) and c.v_scales.shape == (2, 2, 100, 4)
    table = torch.zeros((2, 7), dtype=torch.int32)
    c = kin.alloc_kv4(dims(bs=32, L=200), num_pages=5, block_table=table, device="cpu")
    assert c.v.shape == (5, 2, 32, 64) and c.k_scales.shape == (5, 2, 32, 4) and c.block_table is table


def test_reference_format():
    """The plain form itself: orders are permutations, packing inverts, the
    value of a group is within half a step of its input."""
    assert sorted(ref.KEY_ORDER) == list(range(128)) and sorted(ref.VALUE_ORDER) == list(range(128))
    x = torch.randn((50, 128), generator=torch.Generator().manual_seed(1), dtype=torch.float32).to(torch.bfloat16)
    c, s = ref.quantise(x)
    for order in (ref.KEY_ORDER, ref.VALUE_ORDER):
        assert torch.equal(ref.unpack(ref.pack(c, order), order), c)
    step = s.repeat_interleave(32, -1)
    # half a step, and the clamp at 7 where the scale was rounded down (by at most 2^-8 of 7 steps)
    assert ((ref.values(c, s) - x.double()).abs() <= step * (0.5 + 7 * 2**-8)).all()


def test_plain_forms_agree_with_the_measured_ones():
    """The row format of perf/operators.py and of this plain form are one."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "perf", "operators.py")
    spec = importlib.util.spec_from_file_location("perf_operators", path)
    ops = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ops)
    assert ops.K_ORDER == ref.KEY_ORDER and ops.V_ORDER == ref.VALUE_ORDER
    x = torch.randn((9, 128), generator=torch.Generator().manual_seed(2), dtype=torch.float32).to(torch.bfloat16)
    x[0, 3], x[1, 40], x[2, :32] = float("nan"), float("-inf"), 0
    c, s = ref.quantise(x)
    c2, s2 = ops._quantise(x)
    assert torch.equal(c2.double(), c) and torch.equal(s2.double().nan_to_num(-1), s.nan_to_num(-1))


@pytest.mark.parametrize("n,keep,sink,recent,want", [
    (5, 8, 1, 2, [0, 1, 2, 3, 4]),              # fewer than the budget
    (6, 4, 1, 1, [0, 2, 3, 5]),                 # the best two of 1..4, tie between 3 and 4 to the lower
    (6, 1, 0, 0, [2]),
    (6, 2, 1, 1, [0, 5]),                       # no free slot
])
def test_reference_eviction(n, keep, sink, recent, want):
    assert ref.kept([0.1, 0.0, 0.9, 0.5, 0.5, float("nan")][:n], n, keep, sink, recent) == want
