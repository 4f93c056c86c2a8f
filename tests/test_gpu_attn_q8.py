"""Attention over the 8-bit paged cache on the GPU against the fp64 form
(bounds in q8_helpers.check_attention)."""
import pytest
import torch

import paged_kv_decode_31_b200 as pkv

import q8_helpers as Q

pytestmark = pytest.mark.gpu


def _bf16(shape, gen):
    return torch.randn(shape, generator=gen).to(torch.bfloat16)


def _case(lens, sq, Hq, Hkv, D, bs, seed, spread=3, interleaved=True, packed=None):
    """A cache whose unused slots and blocks hold NaN bytes and whose unused
    table columns hold -1; q dense [B, sq, Hq, D]."""
    gen = torch.Generator().manual_seed(seed)
    table, blocks = Q.table_for([max(n, 0) for n in lens], bs, gen)
    kc, vc, ks, vs = Q.make_cache8(blocks, bs, Hkv, D, gen, spread, interleaved)
    used = torch.zeros(blocks, bs, dtype=torch.bool)
    for b, n in enumerate(lens):
        p = torch.arange(max(n, 0))
        used[table[b, p // bs].long(), p % bs] = True
    for c in (kc, vc):
        c.view(torch.uint8)[~used] = 0x7F
    q = _bf16((len(lens), sq, Hq, D), gen)
    return q, kc, vc, ks, vs, table, torch.tensor(lens, dtype=torch.int32)


def _run(case, causal, scale=None, entry=None, **kw):
    q, kc, vc, ks, vs, table, sl = case
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    D = q.shape[-1]
    scale = D ** -0.5 if scale is None else scale
    out, lse = (entry or pkv.paged_decode_attn_q8)(
        q.cuda(), *Q.cuda_cache(kc, vc, ks, vs), table.cuda(), sl.cuda(),
        max_seqlen_k=max(int(sl.max()), 0), scale=scale, causal=causal, err=err, **kw)
    torch.cuda.synchronize()
    assert int(err) == 0, f"device error bits {int(err)}"
    return out, lse


def _check(case, causal, scale=None, **kw):
    out, lse = _run(case, causal, scale, **kw)
    q, kc, vc, ks, vs, table, sl = case
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    Q.check_attention(out, lse, *Q.attention(q, kc, vc, ks, vs, table, sl, scale, causal))
    return out, lse


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bs", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 2), (10, 2)])
def test_decode(D, bs, Hq, Hkv):
    lens = [1, 2, 15, 16, 17, 127, 128, 129, 300, 0]
    _check(_case(lens, 1, Hq, Hkv, D, bs, seed=D + bs + Hq), causal=False)


@pytest.mark.parametrize("D,Hq,Hkv,sq,causal", [(128, 8, 2, 4, True), (128, 8, 2, 4, False), (64, 4, 4, 3, True),
                                                (128, 16, 2, 2, True), (64, 20, 1, 1, False),
                                                (128, 24, 1, 5, True), (64, 7, 1, 9, True)])
def test_multi_token_decode(D, Hq, Hkv, sq, causal):
    """Up to 16 rows per KV head and more; causal rows that see no key."""
    lens = [1, 3, 9, 64, 130, 259]
    _check(_case(lens, sq, Hq, Hkv, D, 16, seed=sq * 10 + D), causal)


@pytest.mark.parametrize("D,Hq,Hkv,sq,lens", [(128, 8, 2, 40, [40, 57, 200]), (64, 6, 2, 77, [100, 77, 20]),
                                              (128, 4, 4, 130, [130, 300, 1]), (128, 3, 1, 150, [150, 171]),
                                              (64, 16, 2, 33, [33, 1000])])
@pytest.mark.parametrize("causal", [True, False])
def test_prefill(D, Hq, Hkv, sq, lens, causal):
    _check(_case(lens, sq, Hq, Hkv, D, 32, seed=sq), causal, entry=pkv.paged_prefill_attn_q8)


@pytest.mark.parametrize("D,Hq,Hkv,sq", [(128, 8, 2, 1), (64, 4, 1, 20), (128, 16, 1, 12)])
def test_several_splits(D, Hq, Hkv, sq):
    _check(_case([4096, 4097, 9000, 5], sq, Hq, Hkv, D, 64, seed=sq), causal=sq > 1)


def test_scales_far_apart():
    """Blocks whose scales differ by up to 2^20, K's too: every score and every
    V value counts at its own size."""
    for spread, scale in ((10, 2.0 ** -12), (3, None)):
        q, kc, vc, ks, vs, table, sl = _case([700, 129], 2, 8, 2, 128, 16, seed=spread, spread=0)
        gen = torch.Generator().manual_seed(1)
        ks += torch.randint(-3, 4, ks.shape, generator=gen).to(torch.uint8)
        vs += torch.randint(-spread, spread + 1, vs.shape, generator=gen).to(torch.uint8)
        _check((q, kc, vc, ks, vs, table, sl), True, scale)


def test_growing_keys_move_the_reference():
    """Keys that grow tile by tile raise the running reference, and rescale O,
    in every tile; a last large V scale does the same."""
    for D, Hq, sq in ((128, 4, 1), (64, 4, 10), (128, 2, 100)):
        q, kc, vc, ks, vs, table, sl = _case([1500], sq, Hq, 1, D, 16, seed=D, spread=0)
        for j in range(94):
            ks[int(table[0, j])] = 108 + j // 6
            vs[int(table[0, j])] = 110 + (j * 7) % 13
        _check((q, kc, vc, ks, vs, table, sl), True)


def test_one_token_dominates():
    """A sink: one key far above the rest, whose V is almost zero (small
    scale), so the output comes from the others."""
    q, kc, vc, ks, vs, table, sl = _case([600, 40], 1, 4, 1, 128, 16, seed=2, spread=0)
    for b in range(2):
        blk = int(table[b, 0])
        ks[blk] = 126
        vs[blk] = 90
    _check((q, kc, vc, ks, vs, table, sl), False)


def test_query_sizes():
    """Rows of very different size, zeros, and elements 2^20 below the largest."""
    gen = torch.Generator().manual_seed(8)
    case = list(_case([333] * 6, 1, 4, 1, 128, 16, seed=8))
    q = case[0]
    for b, e in enumerate((-40, -8, 0, 3, -20, 0)):
        q[b] = (q[b].float() * 2.0 ** e).to(torch.bfloat16)
    q[5, 0, 1] = 0
    q[4] = (q[4].float() * torch.exp2(torch.randint(0, 20, q[4].shape, generator=gen).float())).to(torch.bfloat16)
    case[0] = q
    _check(tuple(case), False)


def test_packed_requests_equal_the_dense_calls():
    gen = torch.Generator().manual_seed(12)
    n, lens = [1, 0, 4, 33, 1, 130, 17], [700, 5, 4, 33, 1, 4200, 16]
    for D, Hq, Hkv in ((128, 8, 2), (64, 3, 1)):
        case = _case(lens, max(n), Hq, Hkv, D, 16, seed=D)
        _, kc, vc, ks, vs, table, sl = case
        qs = [_bf16((k, Hq, D), gen) for k in n]
        extra = _bf16((3, Hq, D), gen)  # tokens behind the last sequence
        q = torch.cat(qs + [extra])
        cu = torch.tensor([0] + torch.tensor(n).cumsum(0).tolist(), dtype=torch.int32)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        dev = Q.cuda_cache(kc, vc, ks, vs)
        out = torch.full(q.shape, 3.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((Hq, q.shape[0]), 3.0, device="cuda")
        out, lse, fo, fl = pkv.paged_varlen_attn_q8(
            q.cuda(), *dev, table.cuda(), sl.cuda(), cu.cuda(), max(n), max_seqlen_k=max(lens), out=out,
            lse=lse, final=True, err=err)
        assert int(err) == 0
        assert torch.all(out[sum(n):] == 3.0) and torch.all(lse[:, sum(n):] == 3.0)
        for b, k in enumerate(n):
            if not k:
                continue
            a = int(cu[b])
            do, dl = pkv.paged_prefill_attn_q8(qs[b][None].cuda(), *dev, table[b:b + 1].cuda(),
                                               sl[b:b + 1].cuda(), max_seqlen_k=lens[b])
            assert torch.equal(do[0], out[a:a + k]) and torch.equal(dl[0], lse[:, a:a + k])
            assert torch.equal(fo[b], out[a + k - 1]) and torch.equal(fl[b], lse[:, a + k - 1])
            qd = qs[b][None]
            Q.check_attention(do, dl, *Q.attention(qd, kc, vc, ks, vs, table[b:b + 1], sl[b:b + 1],
                                                   D ** -0.5, True))


def test_bits_do_not_depend_on_batch_layout_or_entry():
    """A request alone, in a batch, from a contiguous or interleaved cache,
    through the decode or the prefill call: the same bits -- and a row of a
    decode-sized request (at most 16 rows per KV head) the same bits whatever
    the number of query tokens beside it."""
    for D, Hq, Hkv in ((128, 8, 2), (64, 4, 4)):
        n, L = 70, 333
        q, kc, vc, ks, vs, table, sl = _case([L, 90], n, Hq, Hkv, D, 16, seed=D + 1)
        out, lse = _run((q, kc, vc, ks, vs, table, sl), True, entry=pkv.paged_prefill_attn_q8)
        alone = (q[:1], kc, vc, ks, vs, table[:1], sl[:1])
        o1, l1 = _run(alone, True, entry=pkv.paged_prefill_attn_q8)
        assert torch.equal(o1[0], out[0]) and torch.equal(l1[0], lse[0])
        flat = tuple(x.contiguous() for x in (kc, vc, ks, vs))
        o2, l2 = _run((q[:1], *flat, table[:1], sl[:1]), True)
        assert torch.equal(o2[0], out[0]) and torch.equal(l2[0], lse[0])
        o4, l4 = _run((q[:1, :4], kc, vc, ks, vs, table[:1], torch.tensor([L - n + 4], dtype=torch.int32)), True)
        for i in range(4):  # rows of a four-token step, as decode steps at their own context lengths
            keep = torch.tensor([L - n + i + 1], dtype=torch.int32)
            od, ld = _run((q[:1, i:i + 1], kc, vc, ks, vs, table[:1], keep), False)
            assert torch.equal(od[0, 0], o4[0, i]) and torch.equal(ld[0, :, 0], l4[0, :, i])
            # the prefill kernel rounds elsewhere: both are within their bounds of the exact row
            assert (od[0, 0].double() - out[0, i].double()).abs().max() <= 2.0 ** -6 * od.double().abs().max()


def test_head_major_cache_and_strided_tensors():
    """[num_blocks, Hkv, bs, D] memory seen as [num_blocks, bs, Hkv, D], q a
    slice of a wider projection, out strided."""
    q, kc, vc, ks, vs, table, sl = _case([77, 200], 1, 8, 2, 128, 32, seed=5)
    want = _check((q, kc, vc, ks, vs, table, sl), False)
    hk, hv = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (kc, vc))
    wide = torch.zeros(2, 1, 12, 128, dtype=torch.bfloat16)
    wide[:, :, 2:10] = q
    out = torch.zeros(2, 1, 16, 128, dtype=torch.bfloat16, device="cuda")[:, :, ::2]
    dev = Q.cuda_cache(hk, hv, ks, vs)
    assert not dev[0].is_contiguous()
    o, l = pkv.paged_decode_attn_q8(wide.cuda()[:, :, 2:10], *dev, table.cuda(), sl.cuda(), max_seqlen_k=200,
                                    out=out)
    assert torch.equal(o, want[0]) and torch.equal(l, want[1]) and o.data_ptr() == out.data_ptr()


def test_device_errors():
    q, kc, vc, ks, vs, table, sl = _case([40, 200], 1, 4, 2, 64, 16, seed=4)
    dev = Q.cuda_cache(kc, vc, ks, vs)

    def bits(table, sl, msk, dev=dev):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        pkv.paged_decode_attn_q8(q.cuda(), *dev, table.cuda(), sl.cuda(), max_seqlen_k=msk, err=err)
        return int(err)

    assert bits(table, sl, 200) == 0
    bad = table.clone()
    bad[1, 3] = 1000
    assert bits(bad, sl, 200) == 1
    assert bits(table[:, :8].contiguous(), sl, 200) == 2
    assert bits(table, torch.tensor([40, 5000], dtype=torch.int32), 200) & 16
    s = ks.clone()
    s[table[1, 0].long(), 1] = 255
    assert bits(table, sl, 200, Q.cuda_cache(kc, vc, s, vs)) == 32


def test_streams_and_two_graphs():
    """Two captured graphs with workspaces of their own, replayed on two
    streams at once, and an eager call between."""
    cases = [_case([5000, 300], 1, 8, 2, 128, 16, seed=s) for s in (21, 22)]
    runs = []
    for q, kc, vc, ks, vs, table, sl in cases:
        a = (q.cuda(), *Q.cuda_cache(kc, vc, ks, vs), table.cuda(), sl.cuda())
        want = pkv.paged_decode_attn_q8(*a, max_seqlen_k=5000)
        ws = torch.empty(pkv.workspace_size(2, 1, 8, 128, 5000), dtype=torch.uint8, device="cuda")
        out, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pkv.paged_decode_attn_q8(*a, max_seqlen_k=5000, out=out, lse=lse, workspace=ws)
        runs.append((g, a, want, out, lse, torch.cuda.Stream(), ws))  # (a graph's workspace lives with it)
    for _ in range(3):
        for g, _, _, out, lse, s, _ in runs:
            with torch.cuda.stream(s):
                out.zero_()
                lse.zero_()
                g.replay()
        side = pkv.paged_decode_attn_q8(*runs[0][1], max_seqlen_k=5000, stream=runs[1][5])
        torch.cuda.synchronize()
        for _, _, want, out, lse, _, _ in runs:
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        assert torch.equal(side[0], runs[0][2][0])
