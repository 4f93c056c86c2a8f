"""One KV head: its axis is never stepped over, so whatever stride it has, K and
V may lie in buffers of different shapes."""
import pytest
import torch

import paged_kv_decode_31_b200 as pkv

import q8_helpers as Q

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("wide", [2, 16, 40])
@pytest.mark.parametrize("sq", [1, 40])
def test_k_and_v_of_different_buffers(wide, sq):
    """K of its own, V the first head of a buffer of `wide` heads (and the other
    way round): the bits of two contiguous caches."""
    gen = torch.Generator().manual_seed(wide)
    D, bs, lens = 128, 16, [300, 41]
    table, blocks = Q.table_for(lens, bs, gen)
    dev = Q.cuda_cache(*Q.make_cache8(blocks, bs, 1, D, gen, 3, interleaved=False))
    q = torch.randn(2, sq, 4, D, generator=gen).to(torch.bfloat16).cuda()
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    want = pkv.paged_prefill_attn_q8(q, *dev, table.cuda(), sl, max_seqlen_k=300)
    for i in (0, 1):
        caches = list(dev)
        buf = torch.zeros(blocks, bs, wide, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        caches[i] = buf[:, :, :1]
        caches[i].view(torch.uint8).copy_(dev[i].view(torch.uint8))
        got = pkv.paged_prefill_attn_q8(q, *caches, table.cuda(), sl, max_seqlen_k=300)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
