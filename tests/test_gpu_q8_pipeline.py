"""The new operators together, as a program uses them: serving over the 8-bit
cache (rotating append, then attention, chunk by chunk and token by token), and
a training step (rotating append, prefill, its backward, and the append's)."""
import pytest
import torch

import paged_kv_decode_31_b200 as pkv

import q8_helpers as Q

pytestmark = pytest.mark.gpu


def _bf16(shape, gen):
    return torch.randn(shape, generator=gen).to(torch.bfloat16)


@pytest.mark.parametrize("D,Hq,Hkv,bs,rot,il", [(128, 8, 2, 16, 128, False), (64, 4, 4, 64, 32, True)])
def test_serving_over_the_8_bit_cache(D, Hq, Hkv, bs, rot, il):
    """A packed prompt chunk, a second one, then single tokens, for three
    requests; after every append the attention equals the fp64 form over the
    cache as it then is, and the cache is within a rounding of the rotated
    keys and of the values."""
    gen = torch.Generator().manual_seed(D)
    B, chunks = 3, [[70, 1, 33], [20, 64, 5], [1, 1, 1], [1, 1, 1], [1, 0, 1]]
    total = [sum(c[b] for c in chunks) for b in range(B)]
    table, blocks = Q.table_for(total, bs, gen)
    kc, vc, ks, vs = Q.cuda_cache(*Q.make_cache8(blocks, bs, Hkv, D, gen, nan=True))
    f, m = pkv.rope_frequencies(rot, scaling="blend", factor=4.0, original_max=64)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    fd, td = f.cuda(), table.cuda()
    before = [0] * B
    new = [[], [], []]
    for c in chunks:
        n = sum(c)
        q, k, v = (_bf16((n, h, D), gen) for h in (Hq, Hkv, Hkv))
        cu = torch.tensor([0] + torch.tensor(c).cumsum(0).tolist(), dtype=torch.int32)
        sl = torch.tensor(before, dtype=torch.int32)
        qr = pkv.kv_append_q8(k.cuda(), v.cuda(), kc, vc, ks, vs, td, sl.cuda(), q=q.cuda(), inv_freq=fd,
                              cu_seqlens_new=cu.cuda(), interleaved=il, mscale=m, err=err)
        pos = torch.cat([before[b] + torch.arange(c[b]) for b in range(B)])
        kr = Q.rotate(k, pos, f, il, m)
        for b in range(B):
            new[b].append((kr[cu[b]:cu[b + 1]], v[cu[b]:cu[b + 1]].double()))
            before[b] += c[b]
        sl = torch.tensor(before, dtype=torch.int32)
        out, lse = pkv.paged_varlen_attn_q8(qr, kc, vc, ks, vs, td, sl.cuda(), cu.cuda(), max(c),
                                            max_seqlen_k=max(before), err=err)
        assert int(err) == 0
        host = [t.cpu() for t in (kc, vc)] + [t.cpu().view(torch.uint8) for t in (ks, vs)]
        for b in range(B):
            if not c[b]:
                continue
            a, e = int(cu[b]), int(cu[b + 1])
            ref = Q.attention(qr[a:e].cpu()[None], *host, table[b:b + 1], sl[b:b + 1], D ** -0.5, True)
            Q.check_attention(out[None, a:e], lse[None, :, a:e], *ref)
            # the cache: every value within half a step of its block's scale
            # (twice: a value that was requantised may have been rounded as a
            # subnormal of the smaller scale before)
            p = torch.arange(before[b])
            blk = table[b, p // bs].long()
            for i in (0, 1):
                scale = torch.exp2(host[2 + i][blk].double() - 127)[..., None]
                got = host[i][blk, p % bs].double() * scale
                want = torch.cat([x[i] for x in new[b]])
                tol = torch.maximum(want.abs() * Q.E4M3_HALF, scale * 2.0 ** -9) * (1 + 2.0 ** -9)
                assert torch.all((got - want).abs() <= tol)


def test_training_step_gradients():
    """q, k, v -> rotation and append -> causal prefill -> loss <out, w>: the
    chain of backward calls against fp64 autograd through the plain forms, and
    along a random direction against differences of the fp64 loss.  The
    prefill's backward holds its gradients to 1e-2 of the largest; the append's
    adds one bf16 rounding."""
    gen = torch.Generator().manual_seed(31)
    B, T, Hq, Hkv, D, bs, rot = 2, 150, 4, 2, 64, 16, 48
    f, _ = pkv.rope_frequencies(rot)
    table, blocks = Q.table_for([T, T], bs, gen)
    q, k, v = (_bf16((B, T, h, D), gen) for h in (Hq, Hkv, Hkv))
    w = _bf16((B, T, Hq, D), gen)
    td, fd, zero = table.cuda(), f.cuda(), torch.zeros(B, dtype=torch.int32, device="cuda")
    kc, vc = (torch.zeros(blocks, bs, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    sl = torch.full((B,), T, dtype=torch.int32, device="cuda")
    qr = pkv.kv_append_rope(k.cuda(), v.cuda(), kc, vc, td, zero, fd, q=q.cuda())
    out, lse = pkv.paged_prefill_attn(qr, kc, vc, td, sl, max_seqlen_k=T)
    dqr, dkc, dvc = pkv.paged_prefill_attn_bwd(qr, kc, vc, td, sl, out, lse, w.cuda(), max_seqlen_k=T)
    got = pkv.kv_append_rope_bwd(dqr, dkc, dvc, td, zero, fd)

    pos = torch.arange(T)

    def turn(x):  # differentiable, fp64, half layout
        theta = pos.double()[:, None, None] * f.double()
        a, b, rest = x[..., :rot // 2], x[..., rot // 2:rot], x[..., rot:]
        return torch.cat([a * theta.cos() - b * theta.sin(), b * theta.cos() + a * theta.sin(), rest], -1)

    def loss(q, k, v):
        kr, vr = (x.repeat_interleave(Hq // Hkv, 2) for x in (turn(k), v))
        s = torch.einsum("bihd,bjhd->bhij", turn(q), kr) * D ** -0.5
        s = s.masked_fill(pos[None, :] > pos[:, None], float("-inf"))
        return (torch.einsum("bhij,bjhd->bihd", s.softmax(-1), vr) * w.double()).sum()

    leaves = [x.double().requires_grad_() for x in (q, k, v)]
    loss(*leaves).backward()
    for g, x in zip(got, leaves):
        assert (g.cpu().double() - x.grad).abs().max() <= 1.4e-2 * x.grad.abs().max()
    step = [_bf16(x.shape, gen).double() * 1e-4 for x in (q, k, v)]
    base = [x.double() for x in (q, k, v)]
    diff = (loss(*[a + s for a, s in zip(base, step)]) - loss(*[a - s for a, s in zip(base, step)])) / 2
    along = sum((x.grad * s).sum() for x, s in zip(leaves, step))
    assert abs(diff - along) <= 1e-6 * sum((x.grad * s).abs().sum() for x, s in zip(leaves, step))
    mine = sum((g.cpu().double() * s).sum() for g, s in zip(got, step))
    assert abs(mine - diff) <= 1.4e-2 * sum(x.grad.abs().max() * s.abs().sum() for x, s in zip(leaves, step))
