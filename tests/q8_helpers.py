"""Plain fp64 forms of the rotary and 8-bit-cache operators, on the CPU, and
the inputs of their tests."""
import math

import torch

# Half a step relative to the value: bf16 keeps 8 significant bits, so the step
# is at most 2^-7 of the value (a power of two's) and half of it 2^-8; e4m3
# keeps 4: 2^-4.
BF16_HALF = 2.0 ** -8
E4M3_HALF = 2.0 ** -4


def rotate(x, pos, inv_freq, interleaved=False, mscale=1.0, inverse=False):
    """x [T, H, D] at pos [T], fp64."""
    x = x.double().clone()
    r = 2 * inv_freq.numel()
    theta = pos.double()[:, None, None] * inv_freq.double()
    c, s = mscale * torch.cos(theta), mscale * torch.sin(theta)
    if inverse:
        s = -s
    i = torch.arange(0, r, 2) if interleaved else torch.arange(r // 2)
    j = i + 1 if interleaved else i + r // 2
    a, b = x[..., i], x[..., j]
    x[..., i], x[..., j] = a * c - b * s, b * c + a * s
    return x


def need_exp(amax):
    """Least e in [-63, 63] with amax <= 448 * 2^e (scalar)."""
    if amax == 0:
        return -63
    e = math.frexp(amax)[1] - 9
    while amax > math.ldexp(448.0, e):
        e += 1
    while amax <= math.ldexp(448.0, e - 1):
        e -= 1
    return max(-63, min(63, e))


def to_e4m3(x):
    """Nearest e4m3 (ties to even), saturating, of fp64 values; NaN stays."""
    y = x.abs().clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(y.clamp(min=2.0 ** -6))) - 3)
    y = torch.copysign(torch.round(y / step) * step, x)
    return y.to(torch.float32).to(torch.float8_e4m3fn)


def append_q8(k_new, v_new, kc, vc, ks, vs, table, seqlens, bs):
    """Sequences' new tokens (lists of [n, Hkv, D] fp64, K already rotated)
    into a cache of e4m3 tensors and uint8 scale bytes, in place."""
    for b, n0 in enumerate(seqlens.tolist()):
        for new, cache, sc in ((k_new[b], kc, ks), (v_new[b], vc, vs)):
            n = new.shape[0]
            for col in range(n0 // bs, (n0 + n - 1) // bs + 1 if n else 0):
                blk = int(table[b, col])
                lo, hi = max(n0, col * bs), min(n0 + n, (col + 1) * bs)
                for h in range(new.shape[1]):
                    x = new[lo - n0:hi - n0, h]
                    fin = x[torch.isfinite(x)]
                    e = need_exp(float(fin.abs().max()) if fin.numel() else 0.0)
                    first = lo - col * bs
                    if first > 0:
                        old = int(sc[blk, h]) - 127
                        e = max(e, old)
                        held = cache[blk, :first, h].double() * 2.0 ** (old - e)
                        cache[blk, :first, h] = to_e4m3(held)
                    cache[blk, first:first + hi - lo, h] = to_e4m3(x * 2.0 ** -e)
                    sc[blk, h] = e + 127


def attention(q, kc, vc, ks, vs, table, seqlens, scale, causal, nq=None):
    """fp64 attention of dense q [B, sq, Hq, D] over an 8-bit cache; returns
    out, lse [B, Hq, sq] and the part of out's bound that P's rounding gives:
    2^-10 of A = sum p |v| / sum p (fp16's 2^-11, and as much for fp32 noise),
    and the step that small probabilities keep.  That is 2^-18 (half of the
    smallest step of the third operand, 2^-9 / 2^8) where the largest p of a
    row, with its token's V scale 2^ev folded in, is at least 2^2: 2^-20 2^ev
    |v8| of the result per token, ev at most the largest.
    nq: the query counts of a padded batch."""
    B, sq, Hq, D = q.shape
    bs, Hkv = kc.shape[1], kc.shape[2]
    out = torch.zeros(B, sq, Hq, D, dtype=torch.float64)
    mag = torch.zeros_like(out)
    lse = torch.full((B, Hq, sq), -math.inf, dtype=torch.float64)
    for b in range(B):
        n, L = sq if nq is None else nq[b], int(seqlens[b])
        if L <= 0 or n == 0:
            continue
        p = torch.arange(L)
        blk = table[b].long()[p // bs]
        k = kc[blk, p % bs].double() * torch.exp2(ks.double()[blk] - 127)[..., None]
        v8, ev = vc[blk, p % bs].double(), torch.exp2(vs.double()[blk] - 127)
        v = v8 * ev[..., None]
        tail = 2.0 ** -20 * v8.abs().sum(0) * ev.amax(0)[:, None]  # [Hkv, D]
        k, v = (x.repeat_interleave(Hq // Hkv, 1) for x in (k, v))
        s = scale * torch.einsum("ihd,jhd->hij", q[b, :n].double(), k)
        if causal:
            s = s.masked_fill(p[None, None] > L - n + torch.arange(n)[None, :, None], -math.inf)
        l = torch.logsumexp(s, -1)
        w = torch.exp(s - l[..., None].clamp(min=-1e300))
        w = torch.where(torch.isneginf(l)[..., None], 0.0, w)
        lse[b, :, :n] = l
        out[b, :n] = torch.einsum("hij,jhd->ihd", w, v)
        mag[b, :n] = 2.0 ** -10 * torch.einsum("hij,jhd->ihd", w, v.abs())
        mag[b, :n] += tail.repeat_interleave(Hq // Hkv, 0)
    return out, lse, mag


def check_attention(out, lse, ref, rlse, mag):
    """out: one bf16 rounding of the result (2^-8) and `mag`, what P's rounding
    may do (see attention).  lse: scores off by fp32 rounding and by 2^-21 of
    the row's largest |q| per term (under 6e-5 at these sizes), exp and sums by
    2^-20 relative."""
    out, lse = out.cpu().double(), lse.cpu().double()
    empty = torch.isneginf(rlse)
    assert torch.equal(torch.isneginf(lse), empty)
    assert torch.all(out.permute(0, 2, 1, 3)[empty] == 0)
    tol = ref.abs() * BF16_HALF * 1.01 + mag + 1e-30
    over = ((out - ref).abs() / tol).max().item()
    assert over <= 1, f"out off by {over:.2f} times its bound"
    if (~empty).any():
        d = (lse - rlse)[~empty].abs().max().item()
        assert d <= 1e-4, f"lse off by {d:.2e}"


def make_cache8(blocks, bs, Hkv, D, gen, spread=0, interleaved=True, nan=False):
    """A random cache: values, scale bytes within `spread` of 120; NaN bytes
    everywhere if `nan` (fill what is used)."""
    shape = (blocks, 2, bs, Hkv, D)
    kv = to_e4m3((torch.randn(shape, generator=gen, dtype=torch.float64) * 60).clamp(-448, 448))
    if nan:
        kv.view(torch.uint8).fill_(0x7F)
    sc = 120 + torch.randint(-spread, spread + 1, (blocks, 2, Hkv), generator=gen).to(torch.uint8)
    if interleaved:
        return kv[:, 0], kv[:, 1], sc[:, 0], sc[:, 1]
    return tuple(x.contiguous() for x in (kv[:, 0], kv[:, 1], sc[:, 0], sc[:, 1]))


def cuda_cache(kc, vc, ks, vs):
    """Device copies with the same strides (interleaved views stay such)."""
    def up(t):
        g = torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device="cuda")
        g.view(torch.uint8).copy_(t.view(torch.uint8))
        return g
    return up(kc), up(vc), up(ks).view(torch.float8_e8m0fnu), up(vs).view(torch.float8_e8m0fnu)


def table_for(lens, bs, gen, spare=3, width=None):
    """A shuffled block table for sequences of `lens` tokens; unused columns -1."""
    need = [max(1, -(-n // bs)) for n in lens]
    blocks = sum(need) + spare
    perm = torch.randperm(blocks, generator=gen).to(torch.int32)
    t = torch.full((len(lens), width or max(need)), -1, dtype=torch.int32)
    at = 0
    for b, k in enumerate(need):
        t[b, :k] = perm[at:at + k]
        at += k
    return t, blocks
