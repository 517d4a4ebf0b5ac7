"""Attention over 4-bit caches where some tokens weigh far more than others.
Plain forms, caches and tolerances are test_gpu_kv's; what they have to hold
here besides:

A tile's product keeps 25 bits below the largest of its exponents' sums, and a
code enters as n 2^-18 (even channels) or, of a byte, as n 2^-24 + n' 2^-20
(odd ones), both with the exponent of 2^-14: a product loses at most 2^-39 of
the tile's largest weight, 2^-21 or 2^-19 after the scaling back, 16 of them
2^-15, and the tiles' largest weights add up to no more than sum p.  The
running sums take 9 tiles' additions, 23 * 9 * 2^-23 < 2^-15 of sum p s.  Both
stay below the 2^-13 of sum p s that check_attention allows.
"""
import pytest
import torch

import block_top_sparse_kin_b200 as kin
from test_gpu_kv import Cache, D, check_attention, gen, rows16, status

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
