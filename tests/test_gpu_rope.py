"""Rotation, the rotating append and its backward, and the append into an
8-bit cache, on the GPU against their fp64 forms.

Tolerances: a rotated bf16 value is rounded once (2^-8 of it) from fp32
arithmetic whose sine and cosine are off by at most 2^-22 of a unit and whose
products and sum round three times (2^-24 each): 2^-21 of |x1| + |x2|, times
mscale.  An e4m3 value is rounded once from the same arithmetic (2^-4 of it, or
half the smallest step).  Copied and unrotated values are exact."""
import pytest
import torch

import paged_kv_decode_31_b200 as pkv

import q8_helpers as Q

pytestmark = pytest.mark.gpu


def _bf16(shape, gen):
    return torch.randn(shape, generator=gen).to(torch.bfloat16)


def _near(got, want, x, r, mscale):
    """got (bf16, device) against the fp64 rotation `want` of x."""
    got = got.cpu().double().flatten(0, -3)
    amp = x.double().flatten(0, -3).abs().amax(-1, keepdim=True) * 2 * mscale
    tol = want.abs() * Q.BF16_HALF * 1.001 + amp * 2.0 ** -21
    assert torch.all((got - want).abs()[..., :r] <= tol[..., :r])
    assert torch.equal(got[..., r:], want[..., r:])


@pytest.mark.parametrize("D,rot,interleaved", [(128, 128, False), (128, 128, True), (128, 96, False),
                                               (128, 16, True), (64, 64, False), (64, 48, True),
                                               (64, 16, False)])
@pytest.mark.parametrize("inverse", [False, True])
def test_rope(D, rot, interleaved, inverse):
    gen = torch.Generator().manual_seed(rot + D)
    T, Hq, Hk, m = 37, 7, 3, 1.1386
    q, k = _bf16((T, Hq, D), gen), _bf16((T, Hk, D), gen)
    pos = torch.randint(-5, 1 << 20, (T,), generator=gen, dtype=torch.int32)
    pos[0], pos[1] = 0, (1 << 31) - 1
    f, _ = pkv.rope_frequencies(rot)
    yq, yk = pkv.rope(q.cuda(), pos.cuda(), f.cuda(), k=k.cuda(), interleaved=interleaved, mscale=m,
                      inverse=inverse)
    for x, y in ((q, yq), (k, yk)):
        _near(y, Q.rotate(x, pos, f, interleaved, m, inverse), x, rot, m)


def test_rope_in_place_strided_dense_and_empty():
    gen = torch.Generator().manual_seed(9)
    f, _ = pkv.rope_frequencies(128)
    B, n, H, D = 3, 5, 4, 128
    pos = torch.randint(0, 4096, (B, n), generator=gen, dtype=torch.int32)
    qkv = _bf16((B, n, 3 * H, D), gen)                 # q, k, v side by side: strided views
    q, k = qkv[:, :, :H], qkv[:, :, H:2 * H]
    want = pkv.rope(q.cuda(), pos.cuda(), f.cuda())
    _near(want, Q.rotate(q.flatten(0, 1), pos.flatten(), f), q, D, 1.0)
    g = qkv.cuda()
    out, k_out = pkv.rope(g[:, :, :H], pos.cuda(), f.cuda(), k=g[:, :, H:2 * H], out=g[:, :, :H],
                          k_out=g[:, :, H:2 * H])
    assert torch.equal(out, want) and out.data_ptr() == g.data_ptr()
    _near(k_out, Q.rotate(k.flatten(0, 1), pos.flatten(), f), k, D, 1.0)
    assert torch.equal(g[:, :, 2 * H:].cpu(), qkv[:, :, 2 * H:])
    e = pkv.rope(g[:0, :, :H], pos[:0].cuda(), f.cuda())
    assert e.shape == (0, n, H, D)
    # heads before tokens in memory
    t = _bf16((B, H, n, D), gen)
    y = pkv.rope(t.cuda().transpose(1, 2), pos.cuda(), f.cuda())
    _near(y, Q.rotate(t.transpose(1, 2).flatten(0, 1), pos.flatten(), f), t.transpose(1, 2), D, 1.0)


def test_rope_gradient_matches_differences():
    """<dy, R x> = <R^T dy, x>: the inverse is the transpose of the forward, and
    a step along any direction changes <dy, y> by the gradient's component."""
    gen = torch.Generator().manual_seed(4)
    T, H, D = 9, 2, 64
    f, m = pkv.rope_frequencies(32, scaling="blend", factor=4.0, original_max=4096)
    pos = torch.randint(0, 8192, (T,), generator=gen, dtype=torch.int32)
    x, dy, step = _bf16((T, H, D), gen), _bf16((T, H, D), gen), _bf16((T, H, D), gen)
    kw = dict(interleaved=True, mscale=m)
    dx = pkv.rope(dy.cuda(), pos.cuda(), f.cuda(), inverse=True, **kw).cpu().double()
    up, down = (Q.rotate(x.double() + s * step.double(), pos, f, True, m) for s in (1e-3, -1e-3))
    diff = (dy.double() * (up - down)).sum() / 2e-3
    got = (dx * step.double()).sum()
    # every dx element is off by at most half a bf16 step of itself
    assert abs(got - diff) <= Q.BF16_HALF * 1.01 * (dx * step.double()).abs().sum()


def _setup(lens0, n, Hkv, D, bs, gen, Hq=6, packed=False, layout="interleaved"):
    """Contexts lens0 before the append, n new tokens each (a list)."""
    total = [a + b for a, b in zip(lens0, n)]
    table, blocks = Q.table_for(total, bs, gen)
    seqlens = torch.tensor(lens0, dtype=torch.int32)
    rows = [(_bf16((m, Hq, D), gen), _bf16((m, Hkv, D), gen), _bf16((m, Hkv, D), gen)) for m in n]
    q, k, v = (torch.cat([r[i] for r in rows]) if packed else torch.stack([r[i] for r in rows])
               for i in range(3))
    cu = torch.tensor([0] + torch.tensor(n).cumsum(0).tolist(), dtype=torch.int32) if packed else None
    pos = torch.cat([a + torch.arange(m) for a, m in zip(lens0, n)])
    return table, blocks, seqlens, q, k, v, cu, pos


CASES = [  # contexts before, new tokens, Hkv, D, bs, packed, rotated, interleaved pairs
    ([0], [1], 1, 64, 16, False, 64, False),
    ([15, 16, 17, 130], [1] * 4, 2, 128, 16, False, 128, False),
    ([0, 31, 5], [40] * 3, 2, 128, 32, False, 96, True),
    ([7, 0, 255, 256, 100], [3, 0, 300, 1, 17], 3, 64, 256, True, 64, False),
    ([63, 64, 0], [130, 1, 2], 8, 128, 64, True, 32, True),
    ([5, 0], [1000, 777], 1, 128, 128, True, 128, False),
]


@pytest.mark.parametrize("lens0,n,Hkv,D,bs,packed,rot,il", CASES)
def test_append_rope_and_backward(lens0, n, Hkv, D, bs, packed, rot, il):
    gen = torch.Generator().manual_seed(len(n) * 100 + D)
    table, blocks, sl, q, k, v, cu, pos = _setup(lens0, n, Hkv, D, bs, gen, packed=packed)
    f, _ = pkv.rope_frequencies(rot)
    m = 1.25
    kv = _bf16((blocks, 2, bs, Hkv, D), gen)
    g = kv.cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(interleaved=il, mscale=m, err=err, cu_seqlens_new=None if cu is None else cu.cuda())
    qo = pkv.kv_append_rope(k.cuda(), v.cuda(), g[:, 0], g[:, 1], table.cuda(), sl.cuda(), f.cuda(),
                            q=q.cuda(), **kw)
    assert int(err) == 0
    D3 = lambda x: x.reshape(-1, x.shape[-2], D)  # noqa: E731
    _near(qo, Q.rotate(D3(q), pos, f, il, m), D3(q), rot, m)
    seq = torch.cat([torch.full((c,), b) for b, c in enumerate(n)])
    blk, slot = table[seq, pos // bs].long(), pos % bs
    got = g.cpu()
    _near(got[blk, 0, slot], Q.rotate(D3(k), pos, f, il, m), D3(k), rot, m)
    assert torch.equal(got[blk, 1, slot], D3(v))
    rest = torch.ones(blocks, bs, dtype=torch.bool)
    rest[blk, slot] = False
    assert torch.equal(got.permute(0, 2, 1, 3, 4)[rest], kv.permute(0, 2, 1, 3, 4)[rest])
    # the same bits without queries, and with the outputs in place
    g2, q2 = kv.cuda(), q.cuda()
    assert pkv.kv_append_rope(k.cuda(), v.cuda(), g2[:, 0], g2[:, 1], table.cuda(), sl.cuda(), f.cuda(),
                              **kw) is None
    assert torch.equal(g2, g)
    pkv.kv_append_rope(k.cuda(), v.cuda(), g2[:, 0], g2[:, 1], table.cuda(), sl.cuda(), f.cuda(), q=q2,
                       q_out=q2, **kw)
    assert torch.equal(q2, qo) and torch.equal(g2, g)
    # backward: gradients of cache rows (random) back to the tokens
    grad = _bf16(kv.shape, gen)
    dq, dk, dv = pkv.kv_append_rope_bwd(q.cuda(), grad.cuda()[:, 0], grad.cuda()[:, 1], table.cuda(),
                                        sl.cuda(), f.cuda(), **kw)
    assert int(err) == 0
    assert dq.shape == q.shape and dk.shape == k.shape and dv.shape == v.shape
    _near(dq, Q.rotate(D3(q), pos, f, il, m, inverse=True), D3(q), rot, m)
    _near(dk, Q.rotate(grad[blk, 0, slot], pos, f, il, m, inverse=True), grad[blk, 0, slot], rot, m)
    assert torch.equal(D3(dv.cpu()), grad[blk, 1, slot])
    none, dk2, dv2 = pkv.kv_append_rope_bwd(
        None, grad.cuda()[:, 0], grad.cuda()[:, 1], table.cuda(), sl.cuda(), f.cuda(),
        **(dict(total_new=sum(n)) if packed else dict(n_new=n[0])), **kw)
    assert none is None and torch.equal(dk2, dk) and torch.equal(dv2, dv)


def _append8(kc, vc, ks, vs, k, v, table, sl, q=None, f=None, cu=None, **kw):
    dev = Q.cuda_cache(kc, vc, ks, vs)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    qo = pkv.kv_append_q8(k.cuda(), v.cuda(), *dev, table.cuda(), sl.cuda(),
                          q=None if q is None else q.cuda(), inv_freq=None if f is None else f.cuda(),
                          cu_seqlens_new=None if cu is None else cu.cuda(), err=err, **kw)
    assert int(err) == 0
    kc, vc, ks, vs = (t.cpu() for t in dev)
    return kc, vc, ks.view(torch.uint8), vs.view(torch.uint8), qo


def _lists(x, n, packed):
    return list(x.split(n)) if packed else list(x)


@pytest.mark.parametrize("lens0,n,Hkv,D,bs,packed,rot,il", CASES)
@pytest.mark.parametrize("rotated", [False, True])
def test_append_q8(lens0, n, Hkv, D, bs, packed, rot, il, rotated):
    gen = torch.Generator().manual_seed(len(n) * 100 + D + bs)
    table, blocks, sl, q, k, v, cu, pos = _setup(lens0, n, Hkv, D, bs, gen, packed=packed)
    f, _ = pkv.rope_frequencies(rot)
    cache = Q.make_cache8(blocks, bs, Hkv, D, gen, spread=8)
    size = torch.exp2(torch.randint(-9, 6, (1, Hkv, 1), generator=gen).float())  # some scales rise
    k, v = (k * size).to(torch.bfloat16), (v * size).to(torch.bfloat16)
    kw = dict(interleaved=il, mscale=1.25) if rotated else {}
    kc, vc, ks, vs, qo = _append8(*cache, k, v, table, sl, q=q if rotated else None,
                                  f=f if rotated else None, cu=cu, **kw)
    flat = k.reshape(-1, Hkv, D)
    k64 = Q.rotate(flat, pos, f, il, 1.25) if rotated else flat.double()
    want = [t.clone() for t in cache]
    Q.append_q8(list(k64.split(n)), [x.double() for x in _lists(v, n, packed)], *want, table, sl, bs)
    assert torch.equal(ks, want[2]) and torch.equal(vs, want[3])
    assert torch.equal(vc.view(torch.uint8), want[1].view(torch.uint8))
    if not rotated:
        assert torch.equal(kc.view(torch.uint8), want[0].view(torch.uint8))
        return
    _near(qo, Q.rotate(q.reshape(-1, q.shape[-2], D), pos, f, il, 1.25), q.reshape(-1, q.shape[-2], D),
          rot, 1.25)
    seq = torch.cat([torch.full((c,), b) for b, c in enumerate(n)])
    blk, slot = table[seq, pos // bs].long(), pos % bs
    new = torch.zeros(blocks, bs, dtype=torch.bool)
    new[blk, slot] = True
    assert torch.equal(kc.view(torch.uint8)[~new], want[0].view(torch.uint8)[~new])
    e = torch.exp2(ks[blk].double() - 127)[..., None]
    got = kc[blk, slot].double() * e
    amp = flat.double().abs().amax(-1, keepdim=True) * 2.5
    tol = torch.maximum(k64.abs() * Q.E4M3_HALF, e * 2.0 ** -10) * (1 + 2.0 ** -10) + amp * 2.0 ** -21
    assert torch.all((got - k64).abs() <= tol)


def test_append_q8_token_by_token_and_special_values():
    """A block filled one token at a time ends with the scale of the block
    filled at once, and every value within one rounding of the larger scale's
    subnormal step; zeros, infinities and NaN."""
    gen = torch.Generator().manual_seed(77)
    bs, Hkv, D, T = 16, 2, 64, 40
    table, blocks = Q.table_for([T], bs, gen)
    x = _bf16((1, T, Hkv, D), gen) * torch.exp2(torch.randint(-12, 3, (1, T, 1, 1), generator=gen).float())
    x = x.to(torch.bfloat16)
    x[0, 20] = 0
    x[0, 21, 0, 3] = float("inf")
    x[0, 22, 1, 4] = float("nan")
    x[0, 23, 1, 5] = float("-inf")
    empty = Q.make_cache8(blocks, bs, Hkv, D, gen, nan=True)
    once = _append8(*empty, x, x, table, torch.zeros(1, dtype=torch.int32))
    step = empty
    for t in range(T):
        step = _append8(*step[:4], x[:, t:t + 1], x[:, t:t + 1], table,
                        torch.full((1,), t, dtype=torch.int32))
    assert torch.equal(step[2], once[2]) and torch.equal(step[3], once[3])
    pos = torch.arange(T)
    blk, slot = table[0, pos // bs].long(), pos % bs
    for i in (0, 1):
        a, b = (c[i][blk, slot].double() * torch.exp2(c[2 + i][blk].double() - 127)[..., None]
                for c in (once, step))
        e = torch.exp2(once[2 + i][blk].double() - 127)[..., None]
        assert torch.equal(a.isnan(), x[0].isnan()) and torch.equal(b.isnan(), x[0].isnan())
        # (an infinity saturates at 448 times the scale its block has when it
        # comes, which a token-by-token fill may raise later: not compared)
        ok = torch.isfinite(x[0])
        assert torch.all((a - b).abs()[ok] <= (e * 2.0 ** -9).expand_as(a)[ok])
        assert torch.all((a - b)[ok & (a.abs() >= e * 2.0 ** -5)] == 0)
        assert a[21, 0, 3] == 448 * e[21, 0, 0] and a[23, 1, 5] == -448 * e[23, 1, 0]
    # slots behind the tokens are left as they were
    rest = torch.ones(blocks, bs, dtype=torch.bool)
    rest[blk, slot] = False
    assert torch.all(once[0].view(torch.uint8)[rest] == 0x7F)
    # zeros alone: the smallest scale
    z = _append8(*empty, x[:, :1] * 0, x[:, :1] * 0, table, torch.zeros(1, dtype=torch.int32))
    assert int(z[2][table[0, 0], 0]) == 64 and torch.all(z[0][table[0, 0], 0].float() == 0)


def test_bad_tables_lengths_and_ranges_are_reported():
    """Caller errors set their bit, write nothing outside the table, and leave
    the other sequences' results alone."""
    gen = torch.Generator().manual_seed(5)
    f, _ = pkv.rope_frequencies(64)
    f = f.cuda()
    bs, Hkv, D = 16, 2, 64
    k = _bf16((4, 2, Hkv, D), gen).cuda()
    table = torch.tensor([[0, 1], [99, 2], [3, 4], [5, -1]], dtype=torch.int32, device="cuda")
    sl = torch.tensor([0, 3, 31, 15], dtype=torch.int32, device="cuda")
    for call, make in ((pkv.kv_append_rope, lambda: (torch.zeros(8, bs, Hkv, D, dtype=torch.bfloat16, device="cuda"),) * 1),
                       (pkv.kv_append_q8, None)):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        if make:
            kc, vc = make()[0], torch.zeros(8, bs, Hkv, D, dtype=torch.bfloat16, device="cuda")
            qo = call(k, k, kc, vc, table, sl, f, q=k, err=err)
        else:
            kc, vc, ks, vs = Q.cuda_cache(*Q.make_cache8(8, bs, Hkv, D, gen, interleaved=False))
            before = kc.view(torch.uint8).clone()
            qo = call(k, k, kc, vc, ks, vs, table, sl, q=k, inv_freq=f, err=err)
        # block 99 (sequence 1), column 2 of 2 (sequence 2), block -1 (sequence 3)
        assert int(err) == 1 | 2
        pos = (sl[:, None] + torch.arange(2, device="cuda")).flatten().cpu()
        _near(qo, Q.rotate(k.cpu().flatten(0, 1), pos, f.cpu()), k.cpu(), 64, 1.0)  # queries all rotate
        wrote = torch.zeros(8, bs, dtype=torch.bool)
        wrote[0, 0] = wrote[0, 1] = wrote[4, 15] = wrote[5, 15] = True
        if make:
            assert torch.equal((kc != 0).any(-1).any(-1).cpu(), wrote)
        else:
            same = (kc.view(torch.uint8) == before).all(-1).all(-1).cpu()
            assert torch.all(same[~wrote][:16])  # block 0 behind its two tokens
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kc = torch.zeros(8, bs, Hkv, D, dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, 3, 2, 2, 9], dtype=torch.int32, device="cuda")  # decreases; leaves [0, 8]
    kp = k.reshape(8, Hkv, D)
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(4, 2)
    pkv.kv_append_rope(kp, kp, kc, kc.clone(), table, torch.zeros_like(sl), f, cu_seqlens_new=cu, err=err)
    assert int(err) == 8
    assert torch.equal((kc != 0).any(-1).any(-1).any(-1).cpu(),
                       torch.tensor([1, 0, 0, 0, 0, 0, 0, 0], dtype=torch.bool))
    # tokens behind the last sequence: their query rows stay as they were
    cu = torch.tensor([0, 1, 1, 2, 5], dtype=torch.int32, device="cuda")
    err.zero_()
    qo = torch.full_like(kp, 7.0)
    pkv.kv_append_rope(kp, kp, kc, kc.clone(), table, torch.zeros_like(sl), f, cu_seqlens_new=cu, q=kp,
                       q_out=qo, err=err)
    assert int(err) == 0 and torch.all(qo[5:] == 7.0) and not torch.any(qo[:5] == 7.0)


def test_stream_and_graph():
    """On a side stream and captured: the graph's replay writes the same bits
    for new inputs in the same buffers."""
    gen = torch.Generator().manual_seed(6)
    f = pkv.rope_frequencies(64)[0].cuda()
    bs, Hkv, D = 16, 2, 64
    table, blocks = Q.table_for([40, 9], bs, gen)
    table, sl = table.cuda(), torch.tensor([20, 3], dtype=torch.int32, device="cuda")
    cache = Q.make_cache8(blocks, bs, Hkv, D, gen)
    xs = [_bf16((2, 3, Hkv, D), gen).cuda() for _ in range(3)]
    q = xs[0].clone()
    q_out = torch.empty_like(q)
    side = torch.cuda.Stream()
    a, b = Q.cuda_cache(*cache), Q.cuda_cache(*cache)
    torch.cuda.synchronize()
    first = pkv.kv_append_q8(xs[0], xs[0], *a, table, sl, q=q, inv_freq=f, stream=side)
    side.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        pkv.kv_append_q8(q, q, *b, table, sl, q=q, inv_freq=f, q_out=q_out)
    gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, q_out)
    for s, t in zip(a, b):
        assert torch.equal(s.view(torch.uint8), t.view(torch.uint8))
    for x in xs[1:]:
        q.copy_(x)
        gr.replay()
        want = pkv.kv_append_q8(x, x, *a, table, sl, q=x, inv_freq=f)
        torch.cuda.synchronize()
        assert torch.equal(want, q_out)
        for s, t in zip(a, b):
            assert torch.equal(s.view(torch.uint8), t.view(torch.uint8))
