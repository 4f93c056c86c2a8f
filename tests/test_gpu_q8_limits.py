"""The calls over the 8-bit cache, and the rotating append, at the ends of
their ranges: more units of work than the CTAs hold at once, batches without a
key, split counts far above the contexts, offsets past 32 bits, slices of wider
tensors, and streams given as handles."""
import pytest
import torch

import paged_kv_decode_31_b200 as pkv

import q8_helpers as Q

pytestmark = pytest.mark.gpu


def _bf16(shape, gen):
    return torch.randn(shape, generator=gen).to(torch.bfloat16)


@pytest.mark.parametrize("D,Hq,Hkv,sq,B", [(64, 16, 8, 1, 2400), (128, 128, 8, 1, 2400), (128, 32, 8, 5, 2400),
                                           (64, 48, 8, 3, 9000)])
def test_more_units_than_fit(D, Hq, Hkv, sq, B):
    """Above 128 units per CTA (18944 on 148 SMs, and past the schedule's
    scratch bytes): every request's bits are those of the request alone."""
    gen = torch.Generator().manual_seed(B + D)
    kc, vc, ks, vs = Q.make_cache8(8, 16, Hkv, D, gen, 3)
    dev = Q.cuda_cache(kc, vc, ks, vs)
    table = torch.randint(0, 8, (B, 4), generator=gen).to(torch.int32)
    lens = torch.randint(0, 65, (B,), generator=gen).to(torch.int32)
    q = _bf16((B, sq, Hq, D), gen)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = pkv.paged_prefill_attn_q8(q.cuda(), *dev, table.cuda(), lens.cuda(), max_seqlen_k=64, err=err)
    assert int(err) == 0
    for b in (0, 1, 700, B // 2, B - 2, B - 1):
        one = slice(b, b + 1)
        o1, l1 = pkv.paged_prefill_attn_q8(q[one].cuda(), *dev, table[one].cuda(), lens[one].cuda(), max_seqlen_k=64)
        assert torch.equal(o1[0], out[b]) and torch.equal(l1[0], lse[b])
        Q.check_attention(o1, l1, *Q.attention(q[one], kc, vc, ks, vs, table[one], lens[one], D ** -0.5, True))
    # in the packed call too, where requests without a token lie between
    cu = torch.zeros(2 * B + 1, dtype=torch.int32)
    cu[1::2] = sq * torch.arange(B)
    cu[2::2] = sq * torch.arange(1, B + 1)
    t2, l2 = table.repeat_interleave(2, 0), lens.repeat_interleave(2)
    po, pl = pkv.paged_varlen_attn_q8(q.view(B * sq, Hq, D).cuda(), *dev, t2.cuda(), l2.cuda(), cu.cuda(), sq,
                                      max_seqlen_k=64, err=err)
    assert int(err) == 0
    assert torch.equal(po.view(out.shape), out)
    assert torch.equal(pl.view(Hq, B, sq).transpose(0, 1), lse)


@pytest.mark.parametrize("sq", [1, 40])
def test_no_keys_and_long_limits(sq):
    """Contexts of length zero alone, and max_seqlen_k far above every context:
    out = 0 and lse = -inf without a key, else the bits of the tight limit."""
    gen = torch.Generator().manual_seed(3)
    Hq, Hkv, D = 8, 2, 128
    kc, vc, ks, vs = Q.make_cache8(8, 16, Hkv, D, gen, 3)
    dev = Q.cuda_cache(kc, vc, ks, vs)
    table = torch.randint(0, 8, (3, 4), generator=gen).to(torch.int32).cuda()
    q = _bf16((3, sq, Hq, D), gen).cuda()
    for msk in (0, 64, 50000):
        none = torch.zeros(3, dtype=torch.int32, device="cuda")
        out, lse = pkv.paged_prefill_attn_q8(q, *dev, table, none, max_seqlen_k=msk)
        assert torch.all(out == 0) and torch.all(torch.isneginf(lse))
    lens = torch.tensor([64, 0, 41], dtype=torch.int32, device="cuda")
    a = pkv.paged_prefill_attn_q8(q, *dev, table, lens, max_seqlen_k=64)
    b = pkv.paged_prefill_attn_q8(q, *dev, table, lens, max_seqlen_k=50000)
    c = pkv.paged_prefill_attn_q8(q, dev[0], dev[1], *(s.view(torch.uint8) for s in dev[2:]), table, lens)
    for x in (b, c):
        assert torch.equal(a[0], x[0]) and torch.equal(a[1], x[1])


def test_offsets_past_32_bits():
    """Caches of more than 2^32 bytes, the request in their last blocks."""
    gen = torch.Generator().manual_seed(9)
    Hkv, D, bs, n = 2, 128, 256, 300
    blocks = 2 ** 32 // (bs * Hkv * D) + 8
    table = torch.tensor([[blocks - 1, blocks - 3]], dtype=torch.int32)
    k, v, q = _bf16((1, n, Hkv, D), gen), _bf16((1, n, Hkv, D), gen), _bf16((1, n, 4, D), gen)
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    end = torch.full((1,), n, dtype=torch.int32, device="cuda")
    f = pkv.rope_frequencies(64)[0]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    caches = [torch.empty(blocks, bs, Hkv, D, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2)]
    scales = [torch.zeros(blocks, Hkv, dtype=torch.uint8, device="cuda") for _ in range(2)]
    qr = pkv.kv_append_q8(k.cuda(), v.cuda(), *caches, *scales, table.cuda(), zero, q=q.cuda(), inv_freq=f.cuda(),
                          err=err)
    small = [c[-8:].clone() for c in (*caches, *scales)]
    st = table - (blocks - 8)
    host = [c.cpu() for c in small]
    want = [torch.zeros(8, bs, Hkv, D).to(torch.float8_e4m3fn) for _ in range(2)]
    want += [torch.zeros(8, Hkv, dtype=torch.uint8) for _ in range(2)]
    Q.append_q8([Q.rotate(k[0], torch.arange(n), f)], [v[0].double()], *want, st, torch.zeros(1, dtype=torch.int32), bs)
    used = st[0].long()
    assert torch.equal(host[3][used], want[3][used])
    p = torch.arange(n)
    assert torch.equal(host[1].view(torch.uint8)[used[p // bs], p % bs],
                       want[1].view(torch.uint8)[used[p // bs], p % bs])
    for rows in (slice(n - 1, n), slice(0, n)):
        a = pkv.paged_prefill_attn_q8(qr[:, rows].contiguous(), *caches, *scales, table.cuda(), end, max_seqlen_k=n,
                                      err=err)
        b = pkv.paged_prefill_attn_q8(qr[:, rows].contiguous(), *small, st.cuda(), end, max_seqlen_k=n)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        Q.check_attention(*b, *Q.attention(qr[:, rows].cpu(), *host, st, end.cpu(), D ** -0.5, True))
    del caches, a, b
    bf = [torch.empty(blocks, bs, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    pkv.kv_append_rope(k.cuda(), v.cuda(), *bf, table.cuda(), zero, f.cuda(), err=err)
    dq, dk, dv = pkv.kv_append_rope_bwd(None, *bf, table.cuda(), zero, f.cuda(), n_new=n, err=err)
    rows = bf[1][table[0, p // bs].long().cuda(), (p % bs).cuda()]
    assert torch.equal(rows.cpu(), v[0]) and torch.equal(dv.cpu(), v)
    kr = bf[0][table[0, p // bs].long().cuda(), (p % bs).cuda()]
    alone = pkv.rope(k.cuda(), torch.arange(n, dtype=torch.int32, device="cuda")[None], f.cuda())
    assert torch.equal(kr, alone[0])
    back = pkv.rope(alone, torch.arange(n, dtype=torch.int32, device="cuda")[None], f.cuda(), inverse=True)
    assert torch.equal(dk, back)
    assert int(err) == 0


def test_slices_of_one_projection_and_stream_handles():
    """q, k and v as slices of one [tokens, (Hq + 2 Hkv), D] tensor, rotated in
    place; the stream as a Stream, as its handle, and as the default's 0."""
    gen = torch.Generator().manual_seed(4)
    Hq, Hkv, D, bs = 6, 2, 64, 32
    cu = torch.tensor([0, 50, 50, 83], dtype=torch.int32).cuda()
    sl = torch.tensor([7, 3, 0], dtype=torch.int32).cuda()
    table, blocks = Q.table_for([57, 3, 33], bs, gen)
    table, f = table.cuda(), pkv.rope_frequencies(32)[0].cuda()
    proj = _bf16((83, Hq + 2 * Hkv, D), gen).cuda()
    cache = Q.make_cache8(blocks, bs, Hkv, D, gen)
    after = sl + (cu[1:] - cu[:-1])
    side = torch.cuda.Stream()
    got = []
    for stream in (None, side, side.cuda_stream, 0):
        dev, x = Q.cuda_cache(*cache), proj.clone()
        q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        torch.cuda.synchronize()
        r = pkv.kv_append_q8(k, v, *dev, table, sl, q=q, q_out=q, inv_freq=f, cu_seqlens_new=cu, stream=stream)
        assert r.data_ptr() == x.data_ptr()
        out, lse = pkv.paged_varlen_attn_q8(q, *dev, table, after, cu, 50, max_seqlen_k=57, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(x[:, Hq:], proj[:, Hq:])
        got.append((x, *(t.view(torch.uint8) for t in dev), out, lse))
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))


@pytest.mark.parametrize("D,Hq,Hkv,n", [(128, 8, 2, [3, 40, 1]), (64, 3, 1, [50, 2, 7])])
def test_unaligned_outputs(D, Hq, Hkv, n):
    """out and the final rows with strides that no 16-byte store fits: the same
    bits, in both kernels, with one split and two, and nothing beside them."""
    gen = torch.Generator().manual_seed(D)
    lens = [n[0] + 30, 4200, n[2]]
    table, blocks = Q.table_for(lens, 16, gen)
    dev = Q.cuda_cache(*Q.make_cache8(blocks, 16, Hkv, D, gen, 2))
    q = _bf16((sum(n), Hq, D), gen).cuda()
    cu = torch.tensor([0] + torch.tensor(n).cumsum(0).tolist(), dtype=torch.int32).cuda()
    a = (q, *dev, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), cu, max(n))
    for msk in (4200, 9000):
        want = pkv.paged_varlen_attn_q8(*a, max_seqlen_k=msk, final=True)
        wide = torch.full((sum(n), Hq, D + 3), 7.0, dtype=torch.bfloat16, device="cuda")
        last = torch.full((3, Hq, D + 1), 7.0, dtype=torch.bfloat16, device="cuda")
        got = pkv.paged_varlen_attn_q8(*a, max_seqlen_k=msk, out=wide[..., 1:D + 1], final_out=last[..., 1:])
        for x, y in zip(want, got):
            assert torch.equal(x, y)
        assert torch.all(wide[..., 0] == 7.0) and torch.all(wide[..., D + 1:] == 7.0) and torch.all(last[..., 0] == 7.0)


@pytest.mark.parametrize("sq", [2, 40])
def test_a_query_row_that_is_not_finite_leaves_the_others_alone(sq):
    gen = torch.Generator().manual_seed(sq)
    kc, vc, ks, vs = Q.make_cache8(8, 16, 2, 128, gen, 3)
    table = torch.randperm(8, generator=gen).to(torch.int32)[None].cuda()
    a = (*Q.cuda_cache(kc, vc, ks, vs), table, torch.tensor([100], dtype=torch.int32, device="cuda"))
    q = _bf16((1, sq, 8, 128), gen).cuda()
    want = pkv.paged_prefill_attn_q8(q, *a)
    bad = q.clone()
    bad[0, 1, 3, 5] = float("nan")
    bad[0, 0, 6, 9] = float("-inf")
    got = pkv.paged_prefill_attn_q8(bad, *a)
    same = torch.ones(1, sq, 8, dtype=torch.bool, device="cuda")
    same[0, 1, 3] = same[0, 0, 6] = False
    assert torch.equal(want[0][same], got[0][same])
    assert torch.equal(want[1].transpose(1, 2)[same], got[1].transpose(1, 2)[same])


@pytest.mark.parametrize("D,Hq,Hkv", [(128, 24, 1), (64, 32, 2), (128, 17, 1), (64, 40, 5)])
def test_packed_requests_of_many_heads(D, Hq, Hkv):
    """More than 16 query heads per KV head (every request in the row-major
    kernel), exactly 16, and 8: packed equals the request alone, both within the
    bounds of the exact result; a decode step among prompts."""
    gen = torch.Generator().manual_seed(Hq)
    n, lens = [1, 0, 2, 19, 1, 1], [300, 7, 2, 140, 0, 4100]
    table, blocks = Q.table_for(lens, 64, gen)
    kc, vc, ks, vs = Q.make_cache8(blocks, 64, Hkv, D, gen, 3)
    dev = Q.cuda_cache(kc, vc, ks, vs)
    q = _bf16((sum(n), Hq, D), gen)
    cu = torch.tensor([0] + torch.tensor(n).cumsum(0).tolist(), dtype=torch.int32)
    sl = torch.tensor(lens, dtype=torch.int32)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse, fo, fl = pkv.paged_varlen_attn_q8(q.cuda(), *dev, table.cuda(), sl.cuda(), cu.cuda(), max(n),
                                                max_seqlen_k=4100, final=True, err=err)
    assert int(err) == 0
    for b, k in enumerate(n):
        if not k:
            continue
        a, one = int(cu[b]), slice(b, b + 1)
        qb = q[a:a + k][None]
        o, l = pkv.paged_decode_attn_q8(qb.cuda(), *dev, table[one].cuda(), sl[one].cuda(), max_seqlen_k=4100,
                                        causal=True)
        assert torch.equal(o[0], out[a:a + k]) and torch.equal(l[0], lse[:, a:a + k])
        assert torch.equal(fo[b], out[a + k - 1]) and torch.equal(fl[b], lse[:, a + k - 1])
        Q.check_attention(o, l, *Q.attention(qb, kc, vc, ks, vs, table[one], sl[one], D ** -0.5, True))


def test_packed_calls_one_after_another_and_captured():
    """The two launches of a packed call overlap at their ends: an append before
    the call is seen by both, what follows sees both complete, and a captured
    sequence of steps replays to the same bits."""
    gen = torch.Generator().manual_seed(31)
    Hq, Hkv, D, bs = 16, 4, 128, 16
    n, before = [1, 1, 2, 200, 1, 90], [4000, 900, 50, 700, 5000, 0]
    table, blocks = Q.table_for([b + 4 * k for b, k in zip(before, n)], bs, gen)
    cache = Q.make_cache8(blocks, bs, Hkv, D, gen, 2)
    cu = torch.tensor([0] + torch.tensor(n).cumsum(0).tolist(), dtype=torch.int32).cuda()
    table, step = table.cuda(), (cu[1:] - cu[:-1]).contiguous()
    f = pkv.rope_frequencies(D, device="cuda")[0]
    new = [[_bf16((sum(n), h, D), gen).cuda() for h in (Hq, Hkv, Hkv)] for _ in range(4)]

    def steps(dev, sl, wait):
        outs = []
        for q, k, v in new:
            q = pkv.kv_append_q8(k, v, *dev, table, sl, q=q, inv_freq=f, cu_seqlens_new=cu)
            if wait:
                torch.cuda.synchronize()
            sl = sl + step
            o, l = pkv.paged_varlen_attn_q8(q, *dev, table, sl, cu, max(n), max_seqlen_k=6000)
            outs += [o.clone(), l.clone()]  # (reads both launches' rows at once)
            if wait:
                torch.cuda.synchronize()
        return outs

    start = torch.tensor(before, dtype=torch.int32).cuda()
    want = steps(Q.cuda_cache(*cache), start, True)
    got = steps(Q.cuda_cache(*cache), start, False)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    dev, fresh = Q.cuda_cache(*cache), Q.cuda_cache(*cache)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = steps(dev, start, False)
    for _ in range(2):
        for a, b in zip(dev, fresh):
            a.view(torch.uint8).copy_(b.view(torch.uint8))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
