"""The rotary and 8-bit-cache calls without a GPU: refusals before any launch,
the frequency table, and the plain forms used by the GPU tests."""
import ctypes
import math

import pytest
import torch

import paged_kv_decode_31_b200 as pkv
from paged_kv_decode_31_b200 import binding, cache8, rotary
from paged_kv_decode_31_b200 import build as pkv_build

import q8_helpers as Q

ERR_ARG, ERR_WORKSPACE = 1, 2


@pytest.fixture(scope="module")
def lib():
    pkv_build.build()
    return binding.lib()


def _params(rotary_dim=128, mscale=1.0, inv_freq=0x1000, interleaved=0):
    return rotary._RopeParams(inv_freq, rotary_dim, interleaved, mscale)


def _call(fn, types, args):
    fn.argtypes = types  # (as the binding sets them)
    fn.restype = ctypes.c_int
    return fn(*args)


P, I, I64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
ROPE = [P, P, P, P, I, P, P, P, P, I, P, I, I, I, P, I, P]
APPEND = [P, P, P, P, I, P, P, P, P, P, I, P, P, P, P, I64, P, I64, I, P, I, I, I, I, I, P, P, P]
APPEND8 = APPEND[:15] + [P, P, P, P] + APPEND[15:]
ATTN8 = [P] * 10 + [I64, P, I64, I, P, I, I, I, I, I, I, I, ctypes.c_float, I, P, P, P, P,
                    ctypes.c_size_t, P, P]


def _st(*s):
    return (ctypes.c_int64 * len(s))(*s)


TOK, CACHE, SC = _st(1024, 1024, 128), _st(16 * 8 * 128, 8 * 128, 128), _st(8, 1)


@pytest.mark.parametrize("over", [dict(q=None), dict(q=0x10004), dict(out=None), dict(pos=None),
                                  dict(Hq=0), dict(D=96), dict(rot=24), dict(rot=0), dict(rot=144),
                                  dict(mscale=0.0), dict(mscale=math.nan), dict(freq=None),
                                  dict(st=_st(1024, 1020, 128)), dict(st=_st(1024, 0, 128)),
                                  dict(k=0x9000), dict(batch=-1)])
def test_rope_refusals(lib, over):
    a = dict(q=0x10000, out=0x20000, pos=0x30000, Hq=8, D=128, rot=128, mscale=1.0, freq=0x1000, st=TOK,
             k=None, batch=2)
    a.update(over)
    par = _params(a["rot"], a["mscale"], a["freq"])
    args = [a["q"], a["st"], a["out"], TOK, a["Hq"], a["k"], None, None, None, 0, a["pos"], a["batch"],
            1, a["D"], ctypes.addressof(par), 0, None]
    assert _call(lib.pkv_rope, ROPE, args) == ERR_ARG


def _append_args(**over):
    a = dict(q=None, kn=0x10000, vn=0x20000, cu=None, total=0, kc=0x30000, vc=0x40000, cst=CACHE,
             ks=0x50000, sst=SC, nb=64, bt=0x60000, bts=16, w=16, sl=0x70000, B=2, n=1, Hkv=8, D=128,
             bs=16, rot=128, par=True)
    a.update(over)
    par = _params(a["rot"])
    keep = ctypes.addressof(par) if a["par"] else None
    head = [a["q"], TOK if a["q"] else None, a["q"], TOK if a["q"] else None, 8, a["kn"], TOK, a["vn"],
            TOK, a["cu"], a["total"], a["kc"], a["cst"], a["vc"], CACHE]
    tail = [a["nb"], a["bt"], a["bts"], a["w"], a["sl"], a["B"], a["n"], a["Hkv"], a["D"], a["bs"], keep,
            None, None]
    return head, [a["ks"], a["sst"], a["ks"], SC], tail, par


BAD = [dict(kn=None), dict(vn=0x20008), dict(kc=None), dict(vc=0x40004), dict(nb=0), dict(bt=None),
       dict(bts=8), dict(w=0), dict(sl=None), dict(B=0), dict(n=-1), dict(Hkv=0), dict(D=80), dict(bs=8),
       dict(bs=48), dict(rot=20), dict(cu=0x99000, total=-1), dict(cst=_st(16 * 8 * 128, 8 * 128, 4)),
       dict(B=1 << 20, n=1 << 20)]


@pytest.mark.parametrize("over", BAD)
def test_append_refusals(lib, over):
    head, sc, tail, par = _append_args(**over)
    assert _call(lib.pkv_kv_append_rope, APPEND, head + tail) == ERR_ARG
    assert _call(lib.pkv_kv_append_q8, APPEND8, head + sc + tail) == ERR_ARG


def test_append_rope_needs_frequencies_and_q8_does_not(lib):
    head, sc, tail, par = _append_args(par=False)
    assert _call(lib.pkv_kv_append_rope, APPEND, head + tail) == ERR_ARG
    head, sc, tail, par = _append_args(par=False, q=0x80000)       # queries are rotated: refused
    assert _call(lib.pkv_kv_append_q8, APPEND8, head + sc + tail) == ERR_ARG
    head, sc, tail, par = _append_args(par=False, n=0)              # nothing to append
    assert _call(lib.pkv_kv_append_q8, APPEND8, head + sc + tail) == 0
    for over in (dict(ks=None), dict(sst=_st(8, 0)), dict(cst=_st(16 * 8 * 128, 8 * 128, 8))):
        head, sc, tail, par = _append_args(**over)
        assert _call(lib.pkv_kv_append_q8, APPEND8, head + sc + tail) == ERR_ARG


@pytest.mark.parametrize("over", [dict(q=None), dict(kc=None), dict(ks=None), dict(D=96), dict(Hq=30),
                                  dict(bs=24), dict(scale=0.0), dict(scale=9.0), dict(scale=math.nan),
                                  dict(kst=_st(16 * 8 * 128, 8 * 128, 8)), dict(sst=_st(0, 1)),
                                  dict(kc=0x20008), dict(msk=-1), dict(B=0)])
def test_attention_q8_refusals(lib, over):
    a = dict(q=0x10000, kc=0x20000, ks=0x30000, kst=CACHE, sst=SC, D=128, Hq=32, bs=16, scale=0.1, msk=256,
             B=2, ws=0x90000, wsb=1 << 30)
    a.update(over)

    def call(fn):
        return _call(fn, ATTN8, [a["q"], _st(4096, 4096, 128), a["kc"], a["kst"], a["kc"], CACHE, a["ks"],
                                 a["sst"], a["ks"], SC, 64, 0x40000, 16, 16, 0x50000, a["msk"], a["B"], 1,
                                 a["Hq"], 8, a["D"], a["bs"], a["scale"], 0, 0x60000,
                                 _st(4096, 4096, 128), 0x70000, a["ws"], a["wsb"], None, None])
    assert call(lib.pkv_paged_decode_attn_q8) == ERR_ARG
    assert call(lib.pkv_paged_prefill_attn_q8) == ERR_ARG
    a.update(dict(q=0x10000, kc=0x20000, ks=0x30000, kst=CACHE, sst=SC, D=128, Hq=32, bs=16, scale=0.1,
                  msk=256, B=2, wsb=64))
    assert call(lib.pkv_paged_decode_attn_q8) == ERR_WORKSPACE


def test_error_bit_agrees_with_the_header():
    import re
    text = open(pkv_build.ROOT + "/include/pagedkv.h").read()
    assert int(re.search(r"#define PKV_DEVERR_SCALE (\d+)", text)[1]) == cache8.DEVERR_SCALE


def test_host_tensors_are_rejected():
    x, cu = torch.zeros(2, 1, 4, 128, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    c8 = torch.zeros(8, 16, 4, 128).to(torch.float8_e4m3fn)
    sc = torch.zeros(8, 4, dtype=torch.uint8)
    c, t, sl = torch.zeros(8, 16, 4, 128, dtype=torch.bfloat16), torch.zeros(2, 4, dtype=torch.int32), cu[:2]
    f = torch.ones(64)
    for call in (lambda: pkv.rope(x, cu[:2, None], f), lambda: pkv.kv_append_rope(x, x, c, c, t, sl, f),
                 lambda: pkv.kv_append_rope_bwd(x, c, c, t, sl, f),
                 lambda: pkv.kv_append_q8(x, x, c8, c8, sc, sc, t, sl),
                 lambda: pkv.paged_decode_attn_q8(x, c8, c8, sc, sc, t, sl, max_seqlen_k=4),
                 lambda: pkv.paged_prefill_attn_q8(x, c8, c8, sc, sc, t, sl, max_seqlen_k=4),
                 lambda: pkv.paged_varlen_attn_q8(x[0], c8, c8, sc, sc, t, sl, cu, 1, max_seqlen_k=4)):
        with pytest.raises(TypeError):
            call()


def test_frequency_tables():
    f, m = pkv.rope_frequencies(128)
    assert m == 1.0 and f.dtype == torch.float32 and f.shape == (64,)
    want = torch.tensor([10000.0 ** (-i / 64) for i in range(64)], dtype=torch.float64)
    assert torch.equal(f, want.float())
    lin, _ = pkv.rope_frequencies(128, scaling="linear", factor=4.0)
    assert torch.equal(lin, (want / 4).float())
    base, _ = pkv.rope_frequencies(128, scaling="base", factor=4.0)
    assert base[0] == 1 and abs(float(base[-1]) * 4 / float(want[-1]) - 1) < 1e-6
    for kind in ("blend", "bands"):
        g, m = pkv.rope_frequencies(128, scaling=kind, factor=8.0, original_max=4096)
        turns = 4096 * want / (2 * math.pi)
        assert torch.equal(g[turns >= 34], want.float()[turns >= 34])
        assert torch.equal(g[turns <= 0.9], (want / 8).float()[turns <= 0.9])
        assert torch.all(g[1:] < g[:-1])
        assert m == (0.1 * math.log(8.0) + 1 if kind == "blend" else 1.0)
        same, _ = pkv.rope_frequencies(128, scaling=kind, factor=1.0, original_max=4096)
        assert torch.allclose(same.double(), want, rtol=2.0 ** -23)
    for bad in (dict(rotary_dim=24), dict(rotary_dim=0), dict(rotary_dim=64, base=1.0),
                dict(rotary_dim=64, factor=0.5), dict(rotary_dim=64, scaling="other"),
                dict(rotary_dim=64, scaling="blend", factor=2.0)):
        with pytest.raises(ValueError):
            pkv.rope_frequencies(**bad)


def test_plain_forms():
    """The references themselves: the rotation against complex numbers and its
    transpose, the rounding against torch's, the scale's border cases."""
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(5, 2, 64, generator=gen, dtype=torch.float64)
    pos, f = torch.tensor([0, 1, 7, 100000, -3]), pkv.rope_frequencies(32)[0]
    for il in (False, True):
        y = Q.rotate(x, pos, f, il, 1.25)
        a = x[..., 0:32:2] if il else x[..., :16]
        b = x[..., 1:32:2] if il else x[..., 16:32]
        z = torch.complex(a, b) * torch.exp(1j * pos.double()[:, None, None] * f.double()) * 1.25
        re = y[..., 0:32:2] if il else y[..., :16]
        assert torch.allclose(re, z.real, atol=1e-12) and torch.equal(y[..., 32:], x[..., 32:])
        back = Q.rotate(y, pos, f, il, 1.25, inverse=True)
        assert torch.allclose(back[..., :32], 1.25 ** 2 * x[..., :32], atol=1e-12)
    v = torch.randn(4096, generator=gen, dtype=torch.float64) * 100
    v = torch.cat([v, torch.tensor([0.0, 448.0, -448.0, 2.0 ** -9, 2.0 ** -10, 17.0, 0.0009765625])])
    v = v.float().double()
    assert torch.equal(Q.to_e4m3(v).view(torch.uint8), v.float().clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
    assert [Q.need_exp(a) for a in (0.0, 448.0, 449.0, 224.0, 1.75, 1.76, 2.0 ** 100, 2.0 ** -100)] == \
        [-63, 0, 1, -1, -8, -7, 63, -63]
