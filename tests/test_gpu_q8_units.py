"""Many short units one after another in a CTA of the 8-bit decode kernel: units
of a single pair of tiles leave one softmax warpgroup without work, which must
neither fall behind nor run ahead of the units' query buffers."""
import pytest
import torch

import paged_kv_decode_31_b200 as pkv

import q8_helpers as Q

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,Hq,Hkv,sq,longest", [(64, 2, 1, 1, 256), (128, 16, 4, 1, 256), (128, 8, 1, 2, 700),
                                                 (64, 8, 2, 2, 300)])
def test_short_units_one_after_another(D, Hq, Hkv, sq, longest):
    """Twenty and more units a CTA, most of them one pair of tiles: no wait runs
    out, repeated calls give the same bits, and so does a request alone."""
    gen = torch.Generator().manual_seed(D + Hq + longest)
    B = 3000 // Hkv
    kc, vc, ks, vs = Q.make_cache8(64, 16, Hkv, D, gen, 3)
    dev = Q.cuda_cache(kc, vc, ks, vs)
    cols = -(-longest // 16)
    table = torch.randint(0, 64, (B, cols), generator=gen).to(torch.int32)
    lens = torch.randint(1, 257, (B,), generator=gen)
    some = torch.rand(B, generator=gen) < 0.3  # (beside them a few longer ones, and empty ones)
    lens = torch.where(some, torch.randint(0, longest + 1, (B,), generator=gen), lens).to(torch.int32)
    q = torch.randn(B, sq, Hq, D, generator=gen).to(torch.bfloat16)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    a = (q.cuda(), *dev, table.cuda(), lens.cuda())
    out, lse = pkv.paged_decode_attn_q8(*a, max_seqlen_k=longest, causal=True, err=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    for _ in range(40):
        o, l = pkv.paged_decode_attn_q8(*a, max_seqlen_k=longest, causal=True, err=err)
        assert torch.equal(o, out) and torch.equal(l, lse)
    assert int(err) == 0
    for b in (0, 1, B // 2, B - 1):
        one = slice(b, b + 1)
        o, l = pkv.paged_decode_attn_q8(a[0][one], *dev, a[5][one], a[6][one], max_seqlen_k=longest, causal=True)
        assert torch.equal(o[0], out[b]) and torch.equal(l[0], lse[b])
        Q.check_attention(o, l, *Q.attention(q[one], kc, vc, ks, vs, table[one], lens[one], D ** -0.5, True))
