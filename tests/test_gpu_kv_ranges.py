"""Attention over caches where some tokens weigh far more than others, or have
far larger values.  Plain forms, caches and tolerances are test_gpu_kv's; what
they have to hold here besides:

A tile's product keeps 25 bits below the largest of its exponents' sums, and a
code enters as n 2^-18 (even channels) or, of a byte, as n 2^-24 + n' 2^-20
(odd ones), both with the exponent of 2^-14: a product loses at most 2^-39 of
the tile's largest weight, 2^-21 or 2^-19 after the scaling back, 16 of them
2^-15, and the tiles' largest weights add up to no more than sum p.  The
running sums take 9 tiles' additions, 23 * 9 * 2^-23 < 2^-15 of sum p s.  Both
stay below the 2^-13 of sum p s that check_attention allows.

Scales: where a warp's all lie within 2^10 of its largest vn, fp16 takes at
most 2 * 2^-25 vn from a small weight, and sum p s >= 2^-3 vn (in units where
the heaviest token has 2^7): 130 tokens * 2^-24 * 2^3 = 2^-14 of it.
Elsewhere a step's largest weight is 2^14 or more in fp16: 32 * 2^-25 * 2^-14.

bf16: a logit's distance from the reference is at most 64 here, so a weight's
exponent is rounded by 2^-19 at most, within the 2^-19 of check_attention.
"""
import pytest
import torch

import block_top_sparse_kin_b200 as kin
from test_gpu_kv import Cache, D, check_attention, gen, random_selection, rows16, status

pytestmark = pytest.mark.gpu


def pointed(c, tokens, at=-4.0):
    """Queries of four heads a pair, three along a direction u and one against
    it; the keys of `tokens` are at * u, 11.3 at nats from the others' logits."""
    u = torch.where(torch.rand(D, generator=gen(200), device="cuda") < 0.5, -1.0, 1.0).to(torch.bfloat16)
    c.k = (c.k.float() * 0.5).to(torch.bfloat16)
    c.k[:, :, tokens] = at * u
    return torch.stack([u, 0.75 * u, u * 0.5, -u]).repeat(c.Hkv, 1)[None].repeat(c.B, 1, 1).contiguous()


def attended(c, q):
    d, st = c.dims(4), status()
    out, lse = torch.full_like(q, 9.0), torch.empty(q.shape[:2], device="cuda")
    acc = torch.zeros((c.B, c.Hkv, c.cap), device="cuda")
    kin.kin_kv_decode_attn(d, q, c.stored(), c.seq, None, None, 0, 0.0, out, lse, kin.alloc_kv_attn_workspace(d, 0, acc=True),
                           acc=acc, dev_status=st)
    assert int(st.item()) == 0
    return out, lse, acc


PLACES = {"first": [0], "middle": [77], "last": [299], "tile": list(range(160, 176)), "several": [3, 40, 90, 130, 131, 250]}


@pytest.mark.parametrize("where", PLACES)
@pytest.mark.parametrize("at", [0.6, 0.8, 1.0, 1.2, 1.5])
def test_heavy_tokens_leave_the_light_ones_their_bits(at, where):
    """Tokens 7 to 17 nats above the others; where the heavy one's code is 0 the output is the others'."""
    c = Cache([300], 2, 16, 300, False, 211)
    q = pointed(c, PLACES[where], at=at)
    check_attention(c, q, *attended(c, q), None, True)


@pytest.mark.parametrize("where", PLACES)
@pytest.mark.parametrize("power", [7, 9, 11, 12, 18, 22, 26, 60, 78])
def test_huge_values_under_tiny_weights(power, where):
    """Tokens with huge values that weigh next to nothing leave the others'
    bits alone, and reach the output with what they do weigh: 2^-65, 2^-49 and
    2^-33 of the heaviest for three heads; the fourth reads them alone."""
    c = Cache([300], 2, 16, 300, False, 201)
    q = pointed(c, PLACES[where])
    c.v[:, :, PLACES[where]] *= 2.0**power
    check_attention(c, q, *attended(c, q), None, True)


@pytest.mark.parametrize("where", PLACES)
@pytest.mark.parametrize("power", [None, -78, -60, -30, -20, -12, -9])
def test_the_heaviest_tokens_have_small_values(power, where):
    """The tokens that take the whole softmax have no value, or a tiny one; the output is the others'."""
    c = Cache([300], 2, 16, 300, False, 211)
    q = pointed(c, PLACES[where], at=4.0)
    c.v[:, :, PLACES[where]] *= 0.0 if power is None else 2.0**power
    check_attention(c, q, *attended(c, q), None, True)


def test_values_grow_and_shrink_under_sharp_weights():
    """Every token's scale another power of two, over 2^70, rising, falling
    and mixed, with weights that rise and fall as steeply."""
    c = Cache([480, 480, 480], 2, 16, 480, True, 221)
    q = pointed(c, [], at=0.0)
    steep = torch.linspace(-35, 35, 480, device="cuda")
    mixed = steep[torch.randperm(480, generator=gen(222), device="cuda")]
    u = q[0, 0].float()
    for b, p in enumerate((steep, steep.flip(0), mixed)):
        c.v[b] = (c.v[b].float() * 2.0 ** p[:, None]).to(torch.bfloat16)
        # logits of the first head: -ln 2 of the scale's power, so every token weighs in alike
        c.k[b] = (c.k[b].float() * 0.2 - p[:, None] * (0.6931 * 11.3137 / 128) * u).to(torch.bfloat16)
    check_attention(c, q, *attended(c, q), None, True)


def test_a_not_finite_group_beside_wide_scales():
    """NaN and infinite values among scales far apart: their 32 channels alone are NaN."""
    c = Cache([300], 2, 16, 300, False, 231)
    q = pointed(c, [50])
    c.v[:, :, 50] *= 2.0**30
    c.v[0, 0, 20, 5], c.v[0, 0, 200, 70] = float("nan"), float("inf")
    out, lse, acc = attended(c, q)
    gone = torch.zeros((1, 8, D), dtype=torch.bool, device="cuda")
    gone[0, :4, :32], gone[0, :4, 64:96] = True, True
    assert torch.equal(out.isnan(), gone)
    c.v[0, 0, 20, :32], c.v[0, 0, 200, 64:96] = 0, 0  # the other groups are as without them
    out2, lse2, acc2 = attended(c, q)
    check_attention(c, q, out2, lse2, acc2, None, True)
    assert torch.equal(lse, lse2) and torch.equal(acc, acc2)


@pytest.mark.parametrize("n,bs", [(4096, 16), (20000, 128)])
def test_bf16_values_at_the_ends_of_their_range(n, bs):
    """Thousands of equal weights on the largest values of one sign average to
    that value; values near 2^-76 keep their bits."""
    c = Cache([n], 1, bs, n, False, 241)
    d = c.dims(8)
    ws = kin.alloc_kv_attn_workspace(d, 0)
    for v, q in ((torch.full_like(c.v, 3.3e38), torch.zeros((1, 8, D), dtype=torch.bfloat16, device="cuda")),
                 (torch.full_like(c.v, -3.3e38), rows16(242, 1, 8, D)),
                 ((c.v.float() * 2.0**-76).to(torch.bfloat16), rows16(243, 1, 8, D))):
        c.v = v
        out, lse = torch.full_like(q, 9.0), torch.empty((1, 8), device="cuda")
        kin.kin_kv_decode_attn(d, q, c.bf16(), c.seq, None, None, 0, 0.0, out, lse, ws)
        check_attention(c, q, out, lse, None, None, False)


@pytest.mark.parametrize("k", [0, 40], ids=["every_block", "kept_blocks"])
@pytest.mark.parametrize("g", [3, 8])
def test_scales_far_apart_over_long_ranges(g, k):
    """Warps of up to 64 tiles, ranges that are merged, ragged and paged
    sequences: rows without a value, huge values under tiny weights and light
    tokens beside heavy ones.  1024 tokens a warp: 1024 * 2^-24 * 2^3 = 2^-11
    of sum p s from the small weights, 23 * 64 * 2^-23 < 2^-12 from the running
    sums and 2^-15 from the tiles' products, less than 6 * 2^-13."""
    c = Cache([20000, 4097, 1], 2, 32, 20010, True, 251)
    u = pointed(c, list(range(50, 20000, 997)))[0, 0]
    c.k[0, :, 7000], c.k[0, :, 12345] = 1.5 * u, 1.2 * u
    c.v[0, :, 50::997] *= 2.0**40
    c.v[0, :, 64::640], c.v[1, :, 100:200] = 0, 0
    for b, n in enumerate(c.lens):
        c.k[b, :, n:], c.v[b, :, n:] = float("nan"), float("nan")
    q = (rows16(252, 3, 2 * g, D).float() * 0.1 + u.float() * torch.linspace(1, 0.2, 2 * g, device="cuda")[None, :, None]).to(torch.bfloat16)
    sel, cnt = random_selection(c, k, 253) if k else (None, None)
    dev = (sel.cuda(), cnt.cuda()) if k else (None, None)
    d, st = c.dims(g), status()
    out, lse, acc = torch.full_like(q, 9.0), torch.empty(q.shape[:2], device="cuda"), torch.zeros((3, 2, 20010), device="cuda")
    kin.kin_kv_decode_attn(d, q, c.stored(), c.seq, *dev, k, 0.0, out, lse, kin.alloc_kv_attn_workspace(d, k, acc=True), acc=acc,
                           dev_status=st)
    assert int(st.item()) == 0
    check_attention(c, q, out, lse, acc, None, True, sel.tolist() if k else None, tiles=192)
