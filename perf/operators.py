"""Cases and plain forms of the rotary, appending and 8-bit-cache operators.

Four operators: the rotation of queries and keys (`rope`), the append to a
paged bf16 cache with the rotation applied on the way (`append_rope`, forward
and backward), the same append into a paged cache held in 8 bits with a
power-of-two scale for each block of tokens and KV head (`append_q8`), and
attention over that cache (`attn_q8`: decode, multi-token decode, prefill
chunks, packed requests).  `own` selects the framework's calls; otherwise
`run` computes the same results with elementary torch operations in fp32
(angles in fp64).
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
EXP_MIN, EXP_MAX = -63, 63  # exponents a block's scale may take


def listed():
    return [
        # one decode step of a batch of 64 requests at far positions: latency
        dict(name="rope decode", op="rope", tokens=64, Hq=32, Hkv=8, D=128, rot=128,
             interleaved=False, inverse=False, factor=1.0, mscale=1.0, max_pos=131072),
        # the gradient of a prompt batch's rotation: neighbouring pairs, half
        # of the head, frequencies stretched for a long context
        dict(name="rope gradient", op="rope", tokens=8 * 2048 + 5, Hq=16, Hkv=4, D=128, rot=64,
             interleaved=True, inverse=True, factor=4.0, mscale=1.1386, max_pos=32768),
        # the append of one decode step, 64 requests
        dict(name="append decode", op="append_rope", B=64, n=1, packed=False, ctx=4096, Hq=32,
             Hkv=8, D=128, bs=16, rot=128, interleaved=False, factor=1.0, mscale=1.0, grad=False),
        # a packed batch of prompt chunks of mixed lengths
        dict(name="append chunks", op="append_rope", B=24, n=1024, packed=True, ctx=2048, Hq=16,
             Hkv=4, D=128, bs=16, rot=128, interleaved=False, factor=1.0, mscale=1.0, grad=False),
        # the backward of the append of whole prompts (training)
        dict(name="append gradient", op="append_rope", B=8, n=2048, packed=False, ctx=0, Hq=16,
             Hkv=4, D=128, bs=16, rot=128, interleaved=False, factor=1.0, mscale=1.0, grad=True),
        # the 8-bit cache: one decode step, and a packed batch of prompt chunks
        dict(name="append q8 decode", op="append_q8", B=64, n=1, packed=False, ctx=4096, Hq=32,
             Hkv=8, D=128, bs=16, rot=128, interleaved=False, factor=1.0, mscale=1.0),
        dict(name="append q8 chunks", op="append_q8", B=24, n=1024, packed=True, ctx=2048, Hq=16,
             Hkv=4, D=128, bs=64, rot=96, interleaved=False, factor=4.0, mscale=1.1386),
        # attention over the 8-bit cache: the smallest decode call (two short
        # requests) ...
        dict(name="attn q8 tiny", op="attn_q8", form="dense", B=2, nq=1, ctx=339, mixed=True, Hq=4,
             Hkv=2, D=64, bs=16, causal=False),
        # ... long-context decode (the framework's headline batch) ...
        dict(name="attn q8 long", op="attn_q8", form="dense", B=4, nq=1, ctx=131072, mixed=False,
             Hq=32, Hkv=8, D=128, bs=16, causal=False),
        # ... a ragged decode batch with large pages ...
        dict(name="attn q8 ragged", op="attn_q8", form="dense", B=64, nq=1, ctx=32768, mixed=True,
             Hq=16, Hkv=4, D=128, bs=256, causal=False),
        # ... the last chunk of a chunked prefill ...
        dict(name="attn q8 chunk", op="attn_q8", form="dense", B=8, nq=512, ctx=2048, mixed=False,
             Hq=16, Hkv=4, D=128, bs=16, causal=True),
        # ... and packed requests: decode steps, multi-token steps and chunks
        dict(name="attn q8 packed", op="attn_q8", form="packed", B=32, nq=512, ctx=4096,
             mixed=True, Hq=32, Hkv=8, D=128, bs=16, causal=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["rope", "append_rope", "append_q8", "attn_q8", "attn_q8"])
    D = rng.choice([64, 128])
    Hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8])
    G = min(G, 32 // Hkv)
    heads = dict(Hq=Hkv * G, Hkv=Hkv, D=D)
    bs = rng.choice([16, 32, 64, 128, 256])
    far = rng.random() < 0.5
    rot = dict(rot=16 * rng.randint(1, D // 16), interleaved=rng.random() < 0.5,
               factor=4.0 if far else 1.0, mscale=1.1386 if far else 1.0)
    if op == "rope":
        return dict(op=op, tokens=_log(rng, 1, 16384), max_pos=rng.choice([4096, 131072, 1 << 20]),
                    inverse=rng.random() < 0.5, **heads, **rot)
    if op in ("append_rope", "append_q8"):
        n = 1 if rng.random() < 0.4 else _log(rng, 2, 1024)
        B = _log(rng, 1, max(1, min(64, 16384 // n)))
        c = dict(op=op, B=B, n=n, packed=rng.random() < 0.5, ctx=_log(rng, 1, 8192), bs=bs, **heads,
                 **rot)
        if op == "append_rope":
            c["grad"] = rng.random() < 0.4
        return c
    form = rng.choice(["decode", "decode", "steps", "chunk", "packed"])
    causal = form in ("chunk", "packed") or rng.random() < 0.5
    if form == "decode":
        B = _log(rng, 1, 64)
        nq, ctx = 1, _log(rng, 1, min(131072, (4 * 131072 * 8 * 128) // (B * Hkv * D)))
    elif form == "steps":
        B, nq = _log(rng, 1, 32), rng.randint(2, 17)
        ctx = _log(rng, nq, 16384)
    else:
        B, nq = _log(rng, 1, 8), _log(rng, 18, 512)
        ctx = _log(rng, nq, 2048)
    return dict(op=op, form="packed" if form == "packed" else "dense", B=B, nq=nq, ctx=ctx,
                mixed=rng.random() < 0.5, bs=bs, causal=causal, **heads)


# ---------------------------------------------------------------------------
# the lengths of a case (the same for every seed)
# ---------------------------------------------------------------------------

def _lengths(c):
    """Per request: (query or new tokens, context length before the append or
    with the queries)."""
    rng = random.Random(c["B"] * 7919 + c["ctx"])
    if c["op"] == "attn_q8":
        ctx = [rng.randint(1, c["ctx"]) if c["mixed"] and i else c["ctx"] for i in range(c["B"])]
        if c["form"] == "dense":
            return [c["nq"]] * c["B"], ctx
        nq = [c["nq"] if i == 0 else rng.choice([1, 1, 4, rng.randint(1, c["nq"])])
              for i in range(c["B"])]
        return [min(n, k) for n, k in zip(nq, ctx)], ctx
    n = [rng.randint(1, c["n"]) if c["packed"] and i else c["n"] for i in range(c["B"])]
    return n, [rng.randint(0, c["ctx"]) for _ in range(c["B"])]


def work(c):
    if c["op"] == "rope":
        e = c["tokens"] * (c["Hq"] + c["Hkv"]) * c["D"]
        return {"bytes": 4 * e + 4 * c["tokens"] + 2 * c["rot"], "flops": 3 * e * c["rot"] / c["D"]}
    n, ctx = _lengths(c)
    if c["op"] != "attn_q8":
        t = sum(n)
        q, kv = t * c["Hq"] * c["D"], 2 * t * c["Hkv"] * c["D"]
        wide = 4 * q + (4 if c["op"] == "append_rope" else 3) * kv
        if c["op"] == "append_q8":
            wide += sum(-(-k // c["bs"]) + 1 for k in n) * 2 * c["Hkv"]
        return {"bytes": wide + 4 * len(n), "flops": 3 * (q + kv / 2) * c["rot"] / c["D"]}
    kv = sum(ctx) * c["Hkv"] * c["D"] * 2 + sum(-(-k // c["bs"]) for k in ctx) * 2 * c["Hkv"]
    rows = sum(n) * c["Hq"]
    pairs = sum(sum(max(0, k - a + i + 1) for i in range(a)) if c["causal"] else a * k
                for a, k in zip(n, ctx))
    return {"bytes": kv + rows * (4 * c["D"] + 4), "flops": 4 * c["D"] * pairs * c["Hq"]}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _frequencies(c):
    """Inverse frequencies (fp32): base 10000, the slow ones stretched by
    `factor`, with a ramp between."""
    half = c["rot"] // 2
    i = torch.arange(half, dtype=torch.float64)
    f = 10000.0 ** (-i / half)
    ramp = ((i - half * 0.25) / (half * 0.5)).clamp(0, 1)
    return (f * (1 - ramp) + f / c["factor"] * ramp).to(torch.float32).cuda()


def _cache_q8(blocks, bs, Hkv, D, gen):
    """K and V of `blocks` blocks: normal values, heads and channels of
    different size, in e4m3 with the scale's exponent of each block and head.
    [blocks, 2, bs, Hkv, D] and [blocks, 2, Hkv]."""
    kv = torch.empty(blocks, 2, bs, Hkv, D, dtype=torch.float8_e4m3fn, device="cuda")
    sc = torch.empty(blocks, 2, Hkv, dtype=torch.uint8, device="cuda")
    size = 0.5 + 1.5 * torch.rand(2, 1, Hkv, D, generator=gen, device="cuda")
    step = max(1, (1 << 27) // (2 * bs * Hkv * D))
    for a in range(0, blocks, step):
        x = torch.randn(kv[a:a + step].shape, generator=gen, device="cuda") * size
        x *= 0.25 + 2 * torch.rand(x.shape[0], 1, 1, Hkv, 1, generator=gen, device="cuda")
        e = _need(x.abs().amax(dim=(2, 4)))
        kv[a:a + step] = torch.ldexp(x, -e[:, :, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(kv.dtype)
        sc[a:a + step] = (e + 127).to(torch.uint8)
    return kv, sc.view(torch.float8_e8m0fnu)


def _need(amax):
    """The least exponent e with amax <= 448 * 2^e, within the scale's range."""
    m, e = torch.frexp(amax / E4M3_MAX)
    e = torch.where(m == 0.5, e - 1, e)
    return torch.where(amax > 0, e, EXP_MIN).clamp(EXP_MIN, EXP_MAX)


def _normal(shape, gen):
    return torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)


def prepare(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(c)
    D, Hq, Hkv = c["D"], c["Hq"], c["Hkv"]
    if c["op"] == "rope":
        s["q"], s["k"] = (_normal((c["tokens"], h, D), gen) for h in (Hq, Hkv))
        s["pos"] = torch.randint(0, c["max_pos"], (c["tokens"],), generator=gen, device="cuda",
                                 dtype=torch.int32)
        s["freq"] = _frequencies(c)
        return s
    n, ctx = _lengths(c)
    bs = c["bs"]
    total = ctx if c["op"] == "attn_q8" else [a + b for a, b in zip(n, ctx)]
    need = [max(1, -(-k // bs)) for k in total]
    blocks = sum(need) + 3
    perm = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((c["B"], max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = perm[at:at + k]
        at += k
    s["table"] = table
    s["seqlens"] = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    packed = c["packed"] if c["op"] != "attn_q8" else c["form"] == "packed"
    cu = torch.tensor([sum(n[:b]) for b in range(c["B"] + 1)], dtype=torch.int32, device="cuda")
    s["cu"] = cu if packed else None
    lead = (sum(n),) if packed else (c["B"], n[0])
    s["max_n"], s["max_len"] = max(n), max(total)
    if c["op"] == "attn_q8":
        s["q"] = _normal((*lead, Hq, D), gen)
        s["kv"], s["sc"] = _cache_q8(blocks, bs, Hkv, D, gen)
        s["scale"] = 1.0 / math.sqrt(D)
        return s
    s["freq"] = _frequencies(c)
    s["q"], s["k"], s["v"] = (_normal((*lead, h, D), gen) for h in (Hq, Hkv, Hkv))
    if c["op"] == "append_rope":
        s["kv"] = _normal((blocks, 2, bs, Hkv, D), gen)  # the cache, or its gradient
    else:
        s["kv"], s["sc"] = _cache_q8(blocks, bs, Hkv, D, gen)
        s["k"] = (s["k"] * (0.5 + torch.rand(D, generator=gen, device="cuda"))).to(torch.bfloat16)
    # the places that the append writes: block and slot of each (8 bits: from
    # the start of the first block on, which a larger scale rewrites)
    rows = []
    for b in range(c["B"]):
        first = ctx[b] if c["op"] == "append_rope" else ctx[b] // bs * bs
        p = torch.arange(first, total[b], device="cuda")
        rows.append(torch.stack([table[b, p // bs].long(), p % bs]))
    s["blk"], s["slot"] = torch.cat(rows, 1)
    return s


# ---------------------------------------------------------------------------
# the operators
# ---------------------------------------------------------------------------

def _rotate(x, angle, rot, interleaved, mscale, inverse):
    """x [T, H, D] in fp32, angle [T, rot / 2] in fp64."""
    c = (angle.cos() * mscale).to(x.dtype)[:, None]
    s = (angle.sin() * (-mscale if inverse else mscale)).to(x.dtype)[:, None]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * c - b * s, b * c + a * s], dim=-1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * c - b * s, b * c + a * s], dim=-1)
    return torch.cat([turned, x[..., rot:]], dim=-1)


def _turn(s, x, pos, inverse=False):
    """The rotation of x [..., H, D] at the flat positions `pos`, in fp32."""
    angle = pos.double()[:, None] * s["freq"].double()
    y = _rotate(x.flatten(0, -3).float(), angle, s["rot"], s["interleaved"], s["mscale"], inverse)
    return y.view(x.shape)


def _new_places(s):
    """Sequence and position of every new token, flat."""
    if s["cu"] is not None:
        t = torch.arange(s["k"].shape[0], device="cuda")
        b = torch.searchsorted(s["cu"].long(), t, right=True) - 1
        return b, s["seqlens"][b] + t - s["cu"][b]
    b = torch.arange(s["B"], device="cuda").repeat_interleave(s["n"])
    return b, s["seqlens"][b] + torch.arange(s["n"], device="cuda").repeat(s["B"])


def _values(s):
    """The values that the 8-bit cache holds at the places written."""
    return s["kv"][s["blk"], :, s["slot"]].to(torch.bfloat16) * s["sc"][s["blk"]].to(torch.bfloat16)[..., None]


def _plain_append(s):
    b, pos = _new_places(s)
    blk, slot = s["table"][b, pos // s["bs"]].long(), pos.long() % s["bs"]
    if s.get("grad"):
        g = s["kv"][blk, :, slot]
        dk = _turn(s, g[:, 0], pos, inverse=True).to(torch.bfloat16)
        dq = _turn(s, s["q"], pos, inverse=True).to(torch.bfloat16)
        return dq, dk.view(s["k"].shape), g[:, 1].clone().view(s["v"].shape)
    q = _turn(s, s["q"], pos).to(torch.bfloat16)
    k, v = _turn(s, s["k"], pos).flatten(0, -3), s["v"].flatten(0, -3)
    if s["op"] == "append_rope":
        s["kv"][blk, 0, slot], s["kv"][blk, 1, slot] = k.to(torch.bfloat16), v
        return q, s["kv"][s["blk"], :, s["slot"]]
    x = torch.stack([k, v.float()], 1)  # [T, 2, Hkv, D]
    amax = torch.zeros(s["kv"].shape[0], 2, s["Hkv"], device="cuda")
    amax.index_reduce_(0, blk, x.abs().amax(-1), "amax")
    wrote = torch.zeros(s["kv"].shape[0], dtype=torch.bool, device="cuda")
    wrote[blk] = True
    begun = torch.zeros_like(wrote)  # blocks with earlier tokens
    first = (s["seqlens"] // s["bs"]).clamp(max=s["table"].shape[1] - 1).long()
    start = s["table"].gather(1, first[:, None])[:, 0].long()
    begun[start[s["seqlens"] % s["bs"] > 0]] = True
    old = s["sc"].view(torch.uint8).int() - 127
    e = torch.where(begun[:, None, None], torch.maximum(old, _need(amax)), _need(amax))
    e = torch.where(wrote[:, None, None], e, old)
    up = (begun & wrote).nonzero()[:, 0]
    held = torch.ldexp(s["kv"][up].float(), (old - e)[up][:, :, None, :, None])
    s["kv"][up] = held.to(s["kv"].dtype)
    x = torch.ldexp(x, -e[blk][..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(s["kv"].dtype)
    bits = s["kv"].view(torch.uint8)
    bits[blk, 0, slot], bits[blk, 1, slot] = x[:, 0].view(torch.uint8), x[:, 1].view(torch.uint8)
    s["sc"].view(torch.uint8).copy_(e + 127)
    return q, _values(s)


def _plain_attention(s):
    B, Hkv, D = s["B"], s["Hkv"], s["D"]
    G, n, L = s["Hq"] // Hkv, s["max_n"], s["max_len"]
    key = torch.arange(L, device="cuda")
    held = key < s["seqlens"][:, None]  # [B, L]
    blk = s["table"][:, key // s["bs"]].long().clamp(min=0)
    bits = s["kv"].view(torch.uint8)

    def read(which):
        x = bits[blk, which, key % s["bs"]].view(s["kv"].dtype).float()
        x = x * s["sc"][blk, which].float()[..., None]
        return torch.where(held[..., None, None], x, 0.0).permute(0, 2, 1, 3)  # [B, Hkv, L, D]

    if s["cu"] is not None:
        i = torch.arange(n, device="cuda")
        count = (s["cu"][1:] - s["cu"][:-1])[:, None]
        token = (s["cu"][:-1, None] + i).clamp(max=s["q"].shape[0] - 1).long()
        q = s["q"][token]
        own_row = i < count
    else:
        q, count = s["q"], torch.full((B, 1), n, device="cuda")
        i = torch.arange(n, device="cuda")
    q = q.float().view(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D)
    score = (q @ read(0).transpose(-1, -2)).view(B, Hkv, G, n, L) * s["scale"]
    seen = held[:, None]
    if s["causal"]:
        seen = seen & (key <= (s["seqlens"][:, None] - count + i)[..., None])
    score = torch.where(seen[:, None, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top > -math.inf, top, 0.0))
    total = p.sum(-1, keepdim=True)
    lse = (torch.log(total) + torch.where(top > -math.inf, top, 0.0))[..., 0]
    out = (p.view(B, Hkv, G * n, L) @ read(1)).view(B, Hkv, G, n, D)
    out = torch.where(total > 0, out / total, 0.0).permute(0, 3, 1, 2, 4).reshape(B, n, s["Hq"], D)
    lse = lse.reshape(B, s["Hq"], n)
    if s["cu"] is not None:
        out, lse = out[own_row], lse.permute(0, 2, 1)[own_row].transpose(0, 1).contiguous()
    return out.to(torch.bfloat16), lse


def _own(s):
    import paged_kv_decode_31_b200 as pkv
    turn = {k: s[k] for k in ("interleaved", "mscale") if k in s}
    if s["op"] == "rope":
        return pkv.rope(s["q"], s["pos"], s["freq"], k=s["k"], inverse=s["inverse"], **turn)
    k, v = s["kv"][:, 0], s["kv"][:, 1]
    if s["op"] == "append_rope" and s["grad"]:
        return pkv.kv_append_rope_bwd(s["q"], k, v, s["table"], s["seqlens"], s["freq"],
                                      cu_seqlens_new=s["cu"], **turn)
    if s["op"] == "append_rope":
        q = pkv.kv_append_rope(s["k"], s["v"], k, v, s["table"], s["seqlens"], s["freq"], q=s["q"],
                               cu_seqlens_new=s["cu"], **turn)
        return q, s["kv"][s["blk"], :, s["slot"]]
    ks, vs = s["sc"][:, 0], s["sc"][:, 1]
    if s["op"] == "append_q8":
        q = pkv.kv_append_q8(s["k"], s["v"], k, v, ks, vs, s["table"], s["seqlens"], q=s["q"],
                             inv_freq=s["freq"], cu_seqlens_new=s["cu"], **turn)
        return q, _values(s)
    if s["cu"] is not None:
        return pkv.paged_varlen_attn_q8(s["q"], k, v, ks, vs, s["table"], s["seqlens"], s["cu"],
                                        s["max_n"], max_seqlen_k=s["max_len"], scale=s["scale"],
                                        causal=s["causal"])
    call = pkv.paged_prefill_attn_q8 if s["max_n"] > 17 else pkv.paged_decode_attn_q8
    return call(s["q"], k, v, ks, vs, s["table"], s["seqlens"], max_seqlen_k=s["max_len"],
                scale=s["scale"], causal=s["causal"])


def run(s):
    if own:
        return _own(s)
    if s["op"] == "rope":
        return tuple(_turn(s, x, s["pos"], s["inverse"]).to(torch.bfloat16) for x in (s["q"], s["k"]))
    if s["op"] == "attn_q8":
        return _plain_attention(s)
    return _plain_append(s)


# ---------------------------------------------------------------------------
# the same results from the definitions, in fp64
# ---------------------------------------------------------------------------

def _spin(x, pos, s, sign):
    """Each pair of the rotated part as a complex number times m e^(i theta)."""
    x = x.double()
    r, h = s["rot"], s["rot"] // 2
    first = torch.arange(0, r, 2) if s["interleaved"] else torch.arange(h)
    second = first + (1 if s["interleaved"] else h)
    theta = torch.outer(pos.double(), s["freq"].double())
    z = torch.complex(x[..., first], x[..., second])
    z = z * torch.polar(torch.full_like(theta, s["mscale"]), sign * theta)[:, None]
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "rope":
        return tuple(_spin(x, s["pos"], s, -1 if c["inverse"] else 1) for x in (s["q"], s["k"]))
    n, ctx = _lengths(c)
    bs, D = c["bs"], c["D"]
    if c["op"] == "attn_q8":
        outs, lses, at = [], [], 0
        for b in range(c["B"]):
            p = torch.arange(ctx[b], device="cuda")
            blk = s["table"][b].long()[p // bs]
            k, v = (s["kv"][:, w][blk, p % bs].double() * s["sc"][:, w][blk].double()[..., None]
                    for w in (0, 1))
            q = (s["q"][at:at + n[b]] if s["cu"] is not None else s["q"][b]).double()
            at += n[b]
            bad = p > ctx[b] - n[b] + torch.arange(n[b], device="cuda")[:, None]
            ob, lb = torch.zeros_like(q), torch.empty(c["Hq"], n[b], device="cuda", dtype=q.dtype)
            for h in range(c["Hq"]):
                kv = h * c["Hkv"] // c["Hq"]
                x = s["scale"] * torch.einsum("qd,td->qt", q[:, h], k[:, kv])
                if c["causal"]:
                    x.masked_fill_(bad, -math.inf)
                lb[h] = torch.logsumexp(x, -1)
                some = lb[h] > -math.inf
                ob[some, h] = torch.exp(x[some] - lb[h][some, None]) @ v[:, kv]
            outs.append(ob)
            lses.append(lb)
        if s["cu"] is not None:
            return torch.cat(outs), torch.cat(lses, 1)
        return torch.stack(outs), torch.stack(lses)
    pos = torch.cat([ctx[b] + torch.arange(n[b], device="cuda") for b in range(c["B"])])
    seq = torch.cat([torch.full((n[b],), b, device="cuda") for b in range(c["B"])])
    blk, slot = s["table"][seq, pos // bs].long(), pos % bs
    q, k, v = (s[x].reshape(len(pos), -1, D) for x in "qkv")
    if c["op"] == "append_rope" and c["grad"]:
        dk, dv = s["kv"][blk, 0, slot], s["kv"][blk, 1, slot].double()
        back = [_spin(q, pos, s, -1), _spin(dk, pos, s, -1), dv]
        return tuple(x.view(like.shape) for x, like in zip(back, (s["q"], s["k"], s["v"])))
    new = torch.stack([_spin(k, pos, s, 1), v.double()], 1)
    q = _spin(q, pos, s, 1).view(s["q"].shape)
    if c["op"] == "append_rope":
        return q, new
    got, at = [], 0

    def held(x, e):  # the nearest e4m3 value times 2^e, in fp64
        y = (x / 2.0 ** e).abs().clamp(max=E4M3_MAX)
        step = 2.0 ** (torch.floor(torch.log2(y.clamp(min=2.0 ** -6))) - 3)
        return torch.sign(x) * torch.round(y / step) * step * 2.0 ** e

    for b in range(c["B"]):
        base = ctx[b] // bs * bs
        x = torch.zeros(-(-(ctx[b] + n[b] - base) // bs) * bs, 2, c["Hkv"], D, device="cuda",
                        dtype=torch.float64)
        x[ctx[b] - base:ctx[b] - base + n[b]] = new[at:at + n[b]]
        at += n[b]
        x = x.view(-1, bs, 2, c["Hkv"], D)
        amax = x.abs().amax(dim=(1, 4))
        e = torch.ceil(torch.log2(amax / E4M3_MAX)).clamp(EXP_MIN, EXP_MAX)  # [blocks, 2, Hkv]
        if ctx[b] > base:
            old = s["table"][b, base // bs].long()
            was = s["sc"][old].double()  # [2, Hkv]
            e[0] = torch.maximum(e[0], torch.log2(was))
            x[0, :ctx[b] - base] = (s["kv"][old, :, :ctx[b] - base].double() *
                                    was[:, None, :, None]).transpose(0, 1)
        y = held(x, e[:, None, :, :, None]).flatten(0, 1)
        got.append(y[:ctx[b] + n[b] - base])
    return q, torch.cat(got)
