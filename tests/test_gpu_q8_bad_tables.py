"""The append into an 8-bit cache with tables that cannot be followed: every
byte of the cache and of the scales, written and not, against the plain form with
the invalid columns left out."""
import pytest
import torch

import paged_kv_decode_31_b200 as pkv

import q8_helpers as Q

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,Hkv,bs,n", [(64, 2, 16, 2), (128, 1, 16, 40), (64, 5, 64, 70), (128, 2, 256, 300)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_only_valid_columns_are_written(D, Hkv, bs, n, interleaved):
    """Blocks outside the cache (high, negative), columns past the table's width,
    and a length below zero, between sequences that are right; no rotation, so
    every byte is the plain form's."""
    gen = torch.Generator().manual_seed(D + bs)
    sl = torch.tensor([0, 3, 2 * bs - 1, bs - 1, 5, -1], dtype=torch.int32)
    B, cols = len(sl), 2
    blocks = B * cols + 3
    table = torch.randperm(blocks, generator=gen)[:B * cols].to(torch.int32).view(B, cols)
    table[1, 0] = blocks       # one past the last block
    table[3, 1] = -1
    kc, vc, ks, vs = Q.make_cache8(blocks, bs, Hkv, D, gen, 3, interleaved)
    ks, vs = ks.clone(), vs.clone()
    k, v = (torch.randn(B, n, Hkv, D, generator=gen).mul(s).to(torch.bfloat16) for s in (300, 0.01))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    dev = Q.cuda_cache(kc, vc, ks, vs)
    pkv.kv_append_q8(k.cuda(), v.cuda(), *dev, table.cuda(), sl.cuda(), err=err)
    assert int(err) == 1 | 2
    want = [x.clone() for x in (kc, vc, ks, vs)]
    for b in range(B):
        n0 = int(sl[b])
        for col in range(max(n0, 0) // bs, (n0 + n - 1) // bs + 1):
            if n0 < 0 or col >= cols or not 0 <= int(table[b, col]) < blocks:
                continue
            lo, hi = max(n0, col * bs), min(n0 + n, (col + 1) * bs)
            Q.append_q8([k[b, lo - n0:hi - n0].double()], [v[b, lo - n0:hi - n0].double()], *want,
                        table[b:b + 1], torch.tensor([lo]), bs)
    for name, got, w in zip(("k_cache", "v_cache", "k_scale", "v_scale"), dev, want):
        got, w = got.cpu().view(torch.uint8), w.view(torch.uint8)
        # (a requantised zero keeps its sign, the plain form's may differ in that bit)
        if "cache" in name:
            same = (got == w) | ((got & 0x7F) == 0) & ((w & 0x7F) == 0)
            assert same.all(), name
        else:
            assert torch.equal(got, w), name
