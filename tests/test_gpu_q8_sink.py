"""Attention over the 8-bit cache where one token takes nearly all the weight and
the output comes from thousands of others, far below it."""
import math

import pytest
import torch

import paged_kv_decode_31_b200 as pkv

import q8_helpers as Q

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,Hq,sq", [(64, 1, 1), (128, 4, 1), (128, 8, 1), (64, 16, 1), (128, 1, 40), (64, 4, 40)])
@pytest.mark.parametrize("nats", [12, 13, 14, 15])
@pytest.mark.parametrize("n,sink", [(4096, 0), (4096, 2000), (300, 299), (9000, 4096), (9000, 8999)])
def test_sink_with_the_scale_of_its_block(D, Hq, sq, nats, n, sink):
    """All tokens share one V scale; the sink's V is zero in half of the channels,
    the others' are of one sign, so that nothing cancels what a small
    probability loses.

    The bound: one bf16 rounding of the result (2^-8 of it), 2^-11 of A = sum p
    |v| / sum p for each probability rounded to fp16 and as much again for fp32
    noise, and the step that the smallest keep: 2^-25 (half of fp16's last)
    against a largest one of at least 2^7 in its split, 2^-32 of |v| for each of
    a split's 4096 tokens at most -- 2^-20 of the largest |v|, whatever the
    number of tokens."""
    bs = 64
    gen = torch.Generator().manual_seed(n + sink + D)
    table, blocks = Q.table_for([n], bs, gen)
    kc, vc = (torch.zeros(blocks, bs, 1, D, dtype=torch.float8_e4m3fn) for _ in "kv")
    ks, vs = (torch.full((blocks, 1), b, dtype=torch.uint8) for b in (127, 124))
    v = Q.to_e4m3(1 + torch.rand(n, D, generator=gen, dtype=torch.float64))
    v[sink, :D // 2] = 0
    k = torch.zeros(n, D)
    k[sink, 0] = nats
    p = torch.arange(n)
    blk = table[0, p // bs].long()
    kc.view(torch.uint8)[blk, p % bs, 0] = k.to(torch.float8_e4m3fn).view(torch.uint8)
    vc.view(torch.uint8)[blk, p % bs, 0] = v.view(torch.uint8)
    q = torch.zeros(1, sq, Hq, D, dtype=torch.bfloat16)
    q[..., 0] = 1
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = pkv.paged_prefill_attn_q8(q.cuda(), *Q.cuda_cache(kc, vc, ks, vs), table.cuda(),
                                         torch.tensor([n], dtype=torch.int32, device="cuda"), max_seqlen_k=n,
                                         scale=1.0, causal=False, err=err)
    assert int(err) == 0
    w = torch.exp(k[:, 0].double() - nats)
    total, v = w.sum(), v.double() / 8
    ref = (w[:, None] * v).sum(0) / total
    tol = ref * (Q.BF16_HALF * 1.01 + 2.0 ** -10) + 2.0 ** -20 * v.max()
    over = ((out.cpu().double() - ref).abs() / tol).max().item()
    assert over <= 1, f"out off by {over:.2f} times its bound"
    assert (lse.cpu().double() - (nats + math.log(total))).abs().max() <= 1e-4
