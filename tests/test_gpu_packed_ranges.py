"""Packed appends whose cumulative lengths decrease or leave the token axis: the
error bit is set wherever such a range lies, a token or a block searched for in
it or not, and nothing is written but the other sequences' tokens."""
import pytest
import torch

import paged_kv_decode_31_b200 as pkv

import q8_helpers as Q

pytestmark = pytest.mark.gpu

TABLES = [([0, 5, 3, 8], 8), ([0, 100, 3, 160], 160), ([0, 500, 3, 800], 800), ([0, 0, 0, -1, 40], 40),
          ([0, 20, 10, 10, 10, 64], 64), ([0, 33, 70], 64), ([0, 16, 5000, 40, 64], 64), ([9, 8, 64], 64)]


@pytest.mark.parametrize("cu,total", TABLES)
@pytest.mark.parametrize("Hq", [0, 4])
def test_a_decreasing_range_is_reported(cu, total, Hq):
    B, bs, Hkv, D = len(cu) - 1, 16, 2, 64
    gen = torch.Generator().manual_seed(total)
    cols = -(-total // bs) + 1
    table = torch.arange(B * cols, dtype=torch.int32).view(B, cols).cuda()
    sl = torch.zeros(B, dtype=torch.int32, device="cuda")
    x = torch.randn(total, Hkv, D, generator=gen).to(torch.bfloat16).cuda()
    q = torch.randn(total, Hq, D, generator=gen).to(torch.bfloat16).cuda() if Hq else None
    f = pkv.rope_frequencies(32, device="cuda")[0]
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")

    def bits(call):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        call(err)
        return int(err)

    kc, vc = (torch.zeros(B * cols, bs, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    assert bits(lambda e: pkv.kv_append_rope(x, x, kc, vc, table, sl, f, q=q, cu_seqlens_new=cud, err=e)) == 8
    assert bits(lambda e: pkv.kv_append_rope_bwd(q, kc, vc, table, sl, f, cu_seqlens_new=cud, total_new=total,
                                                 err=e)) == 8
    c8 = Q.cuda_cache(*Q.make_cache8(B * cols, bs, Hkv, D, gen, nan=True))
    assert bits(lambda e: pkv.kv_append_q8(x, x, *c8, table, sl, q=q, inv_freq=f, cu_seqlens_new=cud, err=e)) == 8
    # what is written lies in the blocks of sequences with a range of their own
    for c in (kc.view(torch.int16) != 0, c8[0].view(torch.uint8) != 0x7F):
        wrote = c.flatten(1).any(1).view(B, cols).cpu()
        for b in range(B):
            n = cu[b + 1] - cu[b] if 0 <= cu[b] <= cu[b + 1] <= total else 0
            assert not wrote[b, -(-n // bs):].any()


@pytest.mark.parametrize("cu,total", [([0, 0, 7, 7, 40], 40), ([3, 9, 9, 30], 40), ([0, 40], 40)])
def test_good_ranges_are_not(cu, total):
    """Empty sequences, tokens before the first and behind the last."""
    B, bs, Hkv, D = len(cu) - 1, 16, 1, 64
    gen = torch.Generator().manual_seed(1)
    table = torch.arange(B * 4, dtype=torch.int32).view(B, 4).cuda()
    sl = torch.zeros(B, dtype=torch.int32, device="cuda")
    x = torch.randn(total, Hkv, D, generator=gen).to(torch.bfloat16).cuda()
    f = pkv.rope_frequencies(32, device="cuda")[0]
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kc, vc = (torch.zeros(B * 4, bs, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    pkv.kv_append_rope(x, x, kc, vc, table, sl, f, cu_seqlens_new=cud, err=err)
    assert int(err) == 0
    for b in range(B):
        n = cu[b + 1] - cu[b]
        assert torch.equal(vc.view(B, 4 * bs, D)[b, :n], x[cu[b]:cu[b + 1], 0])
    pkv.kv_append_q8(x, x, *Q.cuda_cache(*Q.make_cache8(B * 4, bs, Hkv, D, gen, nan=True)), table, sl,
                     cu_seqlens_new=cud, err=err)
    assert int(err) == 0
