"""The calls on 4-bit caches refuse outputs that share memory with what they
read, as far as the host can see it: every row is read and written in no order."""
import ctypes

import pytest

import block_top_sparse_kin_b200 as kin

FAKE = 1 << 30  # aligned, never dereferenced: every call below is refused by its host checks
INVALID, WORKSPACE = 1, 2
B, Hkv, L = 2, 2, 256
ROWS = B * Hkv * L


@pytest.fixture(scope="module")
def lib():
    return kin.load_library()


def dims(L=L):
    return kin.make_dims(B, Hkv, 8, 128, 16, L)


def kv4(at, rows=ROWS, **kw):
    """A 4-bit cache whose four tensors lie side by side from `at` on."""
    f = dict(format=kin.KIN_KV_INT4, num_pages=0, block_table=None, k=at, v=at + 64 * rows, k_scales=at + 128 * rows,
             v_scales=at + 136 * rows)
    f.update(kw)
    return kin.kin_kv(*f.values())


def kv16(at, rows=ROWS, **kw):
    return kv4(at, **{**dict(format=kin.KIN_KV_BF16, k=at, v=at + 256 * rows, k_scales=None, v_scales=None), **kw})


END4, END16 = 144 * ROWS, 512 * ROWS
POOL = dict(block_table=FAKE, num_pages=4)  # 128 rows


@pytest.mark.parametrize("at", [FAKE, FAKE + END16 - 16, FAKE - END4 + 16, FAKE + 256 * ROWS])
def test_store_refuses_shared_memory(lib, at):
    d = dims()
    assert lib.kin_kv4_store(ctypes.byref(d), ctypes.byref(kv16(FAKE)), ctypes.byref(kv4(at)), FAKE, None, 0, None, None) == INVALID


def test_store_refuses_scales_in_the_source(lib):
    d, far = dims(), FAKE + (1 << 28)
    for name in ("k_scales", "v_scales"):
        dst = kv4(far, **{name: FAKE + 1024})
        assert lib.kin_kv4_store(ctypes.byref(d), ctypes.byref(kv16(FAKE)), ctypes.byref(dst), FAKE, None, 0, None, None) == INVALID
    pool = kv16(FAKE, **POOL)  # a pool ends where its pages do
    dst = kv4(FAKE + 256 * 127)
    assert lib.kin_kv4_store(ctypes.byref(d), ctypes.byref(pool), ctypes.byref(dst), FAKE, None, 0, None, None) == INVALID


def test_append_refuses_lengths_that_overlap_in_part(lib):
    d = dims()
    for new in (FAKE + 4, FAKE - 4):
        assert lib.kin_kv4_append(ctypes.byref(d), ctypes.byref(kv4(FAKE + 4096)), None, 0, FAKE, new, FAKE, FAKE, 1, None,
                                  None) == INVALID


def test_load_refuses_shared_memory(lib):
    d, far, n = dims(), FAKE + (1 << 28), 8
    out = B * Hkv * n * 256
    for k, v in ((far, far), (far, far + out - 16), (FAKE, far), (far, FAKE + END4 - 16), (FAKE - out + 16, far)):
        assert lib.kin_kv4_load(ctypes.byref(d), ctypes.byref(kv4(FAKE)), far, None, n, k, v, None, None) == INVALID


def evict(lib, src, dst, acc=FAKE + (1 << 27), dacc=None, lens=FAKE + (1 << 26), dlens=FAKE + (1 << 26) + 4096):
    d, dd = dims(), dims(128)
    return lib.kin_kv_evict(ctypes.byref(d), ctypes.byref(src), acc, lens, 64, 4, 16, ctypes.byref(dd), ctypes.byref(dst), dacc,
                            dlens, None, 0, None, None, 0, None, None)


def test_evict_refuses_shared_memory(lib):
    far = FAKE + (1 << 28)
    src, half = kv4(FAKE), ROWS // 2
    assert evict(lib, src, kv4(far, half)) == WORKSPACE  # all that is wrong is the missing workspace
    assert evict(lib, src, kv4(FAKE + END4, half)) == WORKSPACE and evict(lib, src, kv4(FAKE - END4 // 2, half)) == WORKSPACE
    for at in (FAKE + 64, FAKE + END4 - 64, FAKE - END4 // 2 + 64):
        assert evict(lib, src, kv4(at, half)) == INVALID
    assert evict(lib, src, kv4(far, half, k_scales=FAKE + 128 * ROWS)) == INVALID
    assert evict(lib, kv16(FAKE), kv16(FAKE + 64, half)) == INVALID
    # one side in pages: laid over the other
    assert evict(lib, src, kv4(FAKE + 64, 64, **{**POOL, "num_pages": 1})) == INVALID
    # pages of one pool are the caller's to keep apart
    table2 = {**POOL, "block_table": FAKE + 4096}
    assert evict(lib, kv4(FAKE, 128, **POOL), kv4(FAKE, 128, **table2)) == WORKSPACE


def test_evict_refuses_weights_and_lengths_that_overlap(lib):
    far, acc, lens = FAKE + (1 << 28), FAKE + (1 << 27), FAKE + (1 << 26)
    src, dst = kv4(FAKE), kv4(far, ROWS // 2)
    for dacc in (acc, acc + 4 * ROWS - 4, acc - 2 * ROWS + 4):
        assert evict(lib, src, dst, acc=acc, dacc=dacc) == INVALID
    assert evict(lib, src, dst, acc=acc, dacc=acc + 4 * ROWS) == WORKSPACE
    for dlens in (lens, lens + 4, lens - 4):
        assert evict(lib, src, dst, lens=lens, dlens=dlens) == INVALID
