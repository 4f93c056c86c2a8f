"""Attention over an 8-bit cache whose blocks' V scales lie as far apart as the
accepted exponents, -63 to 63: blocks of zeros beside the largest values."""
import pytest
import torch

import paged_kv_decode_31_b200 as pkv

import q8_helpers as Q

pytestmark = pytest.mark.gpu


def _attention(q, kc, vc, ks, vs, table, n, scale):
    """fp64 out, lse of q [rows, D] over the n tokens of one sequence and head,
    and A = sum p |v| / sum p."""
    bs = kc.shape[1]
    p = torch.arange(n)
    blk = table[0, p // bs].long()
    k, v = (c[blk, p % bs, 0].double() * torch.exp2(s[blk, 0].double() - 127)[:, None]
            for c, s in ((kc, ks), (vc, vs)))
    x = scale * q.double() @ k.T
    lse = torch.logsumexp(x, -1)
    w = torch.exp(x - lse[:, None])
    return w @ v, lse, w @ v.abs()


@pytest.mark.parametrize("D,Hq,sq", [(64, 1, 1), (128, 4, 1), (128, 8, 1), (64, 16, 1), (128, 1, 40), (64, 4, 40)])
@pytest.mark.parametrize("low,high", [(-63, 63), (-63, 30), (-63, -7), (-40, 50)])
@pytest.mark.parametrize("below,cols", [(b, [0, 100, 257]) for b in (-6, 0, 4)] +
                         [(b, [c]) for b in (12, 20) for c in (7, 100, 257)])
def test_zero_blocks_beside_large_values(D, Hq, sq, low, high, below, cols):
    """Most tokens have V = 0 in blocks of the scale `low` (an append gives them
    -63), `below` binary orders below the others in score; the others' V is of
    one sign, in the blocks `cols` (of the first split and the second) of the scale
    `high`.  The zeros' weight must be in the sum.

    The bound: one bf16 rounding of the result and 2^-10 of A (fp16's 2^-11 and
    as much for fp32 noise); nothing else, since the tokens that make the output
    are the largest of their row.  lse: 2^-20 relative of the sum, and the score's
    own rounding: exponents of up to 2^7 in fp32, 2^-17 each side."""
    bs, n = 16, 4200
    gen = torch.Generator().manual_seed(D + Hq + low + high + below)
    table, blocks = Q.table_for([n], bs, gen)
    kc, vc = (torch.zeros(blocks, bs, 1, D, dtype=torch.float8_e4m3fn) for _ in "kv")
    ks = torch.full((blocks, 1), 127, dtype=torch.uint8)
    vs = torch.full((blocks, 1), 127 + low, dtype=torch.uint8)
    for c in cols:
        blk = int(table[0, c])
        vs[blk] = 127 + high
        vc[blk] = Q.to_e4m3(64 + 256 * torch.rand(bs, 1, D, generator=gen, dtype=torch.float64))
    for c in range(table.shape[1]):  # scores: log2 units, D = 64 .. 128 by one channel
        kc[int(table[0, c]), :, 0, 0] = float(0 if c in cols else -below)
    q = torch.zeros(1, sq, Hq, D, dtype=torch.bfloat16)
    q[..., 0] = 1
    scale = 0.6931471805599453
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = pkv.paged_prefill_attn_q8(q.cuda(), *Q.cuda_cache(kc, vc, ks, vs), table.cuda(),
                                         torch.tensor([n], dtype=torch.int32, device="cuda"), max_seqlen_k=n,
                                         scale=scale, causal=False, err=err)
    assert int(err) == 0
    ref, rl, mag = _attention(q[0].flatten(0, 1), kc, vc, ks, vs, table, n, scale)
    tol = ref.abs() * Q.BF16_HALF * 1.01 + 2.0 ** -10 * mag
    over = ((out.cpu().double()[0].flatten(0, 1) - ref).abs() / tol).max().item()
    assert over <= 1, f"out off by {over:.2f} times its bound"
    d = (lse.cpu().double()[0].T.flatten() - rl).abs().max().item()
    assert d <= 2.0 ** -16 + 2.0 ** -20, f"lse off by {d:.2e}"


@pytest.mark.parametrize("D,Hq,sq", [(128, 4, 1), (128, 8, 1), (64, 16, 1), (128, 4, 40)])
def test_any_scales_side_by_side(D, Hq, sq):
    """Every block's V scale drawn from -63 to 63: the output is that of the
    largest few, the sum that of all."""
    bs, n = 16, 5000
    gen = torch.Generator().manual_seed(D + Hq)
    table, blocks = Q.table_for([n], bs, gen)
    kc, vc, ks, vs = Q.make_cache8(blocks, bs, 1, D, gen, 0, interleaved=False)
    vs = (64 + torch.randint(0, 127, vs.shape, generator=gen)).to(torch.uint8)
    q = torch.randn(1, sq, Hq, D, generator=gen).to(torch.bfloat16)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = pkv.paged_prefill_attn_q8(q.cuda(), *Q.cuda_cache(kc, vc, ks, vs), table.cuda(),
                                         torch.tensor([n], dtype=torch.int32, device="cuda"), max_seqlen_k=n,
                                         causal=False, err=err)
    assert int(err) == 0
    ref, rl, mag = _attention(q[0].flatten(0, 1), kc, vc, ks, vs, table, n, D ** -0.5)
    tol = ref.abs() * Q.BF16_HALF * 1.01 + 2.0 ** -10 * mag
    assert ((out.cpu().double()[0].flatten(0, 1) - ref).abs() <= tol).all()
    assert (lse.cpu().double()[0].T.flatten() - rl).abs().max() <= 1e-4
