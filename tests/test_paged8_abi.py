"""Refusals and host logic of the windowed attention, the rotary append, the
cache read-back and the e4m3 cache.  Runs without a GPU: every argument check
precedes the first CUDA call."""
from __future__ import annotations

import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import paged8


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_verification_attn_gb300 import binding, build
    build.build()
    return binding.load()


def vp(x):
    return ctypes.c_void_p(x) if x else None


def _err(lib, rc, code, needle):
    assert rc == code
    assert needle in lib.spec_last_error().decode()


@pytest.mark.parametrize("bad,needle", [
    (dict(window=0), "window must be"),
    (dict(window=-5), "window must be"),
    (dict(sinks=-1), "num_sinks"),
    (dict(mask=16, window=3), "tree"),
    (dict(k=0), "num_draft"),
    (dict(k=65), "num_draft"),
    (dict(Hq=6, Hkv=4), "multiple"),
    (dict(D=100), "head_dim"),
    (dict(kvdt=2), "kv_dtype"),
    (dict(kvdt=6), "kv_dtype"),
    (dict(kvdt=5), "E4M3"),
    (dict(kvdt=5, ks=16, vs=18), "4-byte"),
    (dict(q=0), "null"),
    (dict(out=24), "aligned"),
    (dict(scale=float("nan")), "NaN"),
])
def test_window_refusals(lib, bad, needle):
    a = dict(q=16, kc=16, vc=16, ks=None, vs=None, bt=16, ctx=16, mask=None, B=1, k=4, Hq=8,
             Hkv=2, D=128, P=16, NP=8, MP=4, qdt=1, kvdt=1, scale=0.088, window=64, sinks=4,
             out=16)
    a.update(bad)
    rc = lib.spec_verify_attn_window(
        vp(a["q"]), vp(a["kc"]), vp(a["vc"]), vp(a["ks"]), vp(a["vs"]), vp(a["bt"]), vp(a["ctx"]),
        vp(a["mask"]), a["B"], a["k"], a["Hq"], a["Hkv"], a["D"], a["P"], a["NP"], a["MP"],
        a["qdt"], a["kvdt"], a["scale"], a["window"], a["sinks"], vp(a["out"]), None, None)
    _err(lib, rc, -1, needle)


@pytest.mark.parametrize("bad,code,needle", [
    (dict(n=0), -1, "num_new"),
    (dict(Hkv=0), -1, "num_kv_heads"),
    (dict(Hq=-1), -1, "num_q_heads"),
    (dict(D=48), -1, "head_dim"),
    (dict(rot=24), -1, "rotary_dim"),
    (dict(rot=144), -1, "rotary_dim"),
    (dict(rot=-16), -1, "rotary_dim"),
    (dict(src=5), -1, "src_dtype"),
    (dict(cdt=2), -1, "cache_dtype"),
    (dict(cdt=6), -1, "cache_dtype"),
    (dict(amp=math.inf), -1, "amplitude"),
    (dict(amp=math.nan), -1, "amplitude"),
    (dict(kst=255), -1, "stride is shorter"),
    (dict(qst=1000), -1, "stride is shorter"),
    (dict(kst=260), -1, "aligned"),
    (dict(q=0), -1, "null"),
    (dict(table=0), -1, "null"),
    (dict(vc=0), -1, "null"),
    (dict(ks=0), -1, "E4M3"),
    (dict(kn=24), -1, "aligned"),
    (dict(vc=24), -1, "aligned"),
    (dict(table=20), -1, "8-byte"),
    (dict(cdt=3, ks=0), -1, "I8"),
    (dict(B=1 << 20, n=1 << 10), -2, "too many"),
])
def test_rope_append_refusals(lib, bad, code, needle):
    a = dict(q=16, kn=16, vn=16, qo=16, qst=1024, kst=256, vst=256, ost=1024, src=1, kc=16, vc=16,
             ks=16, vs=16, cdt=5, bt=16, ctx=16, table=16, rot=64, amp=1.0, B=2, n=4, Hq=8, Hkv=2,
             D=128, P=16, NP=8, MP=4)
    a.update(bad)
    rc = lib.spec_rope_append(
        vp(a["q"]), vp(a["kn"]), vp(a["vn"]), vp(a["qo"]), a["qst"], a["kst"], a["vst"], a["ost"],
        a["src"], vp(a["kc"]), vp(a["vc"]), vp(a["ks"]), vp(a["vs"]), a["cdt"], vp(a["bt"]),
        vp(a["ctx"]), None, None, vp(a["table"]), a["rot"], 0, a["amp"], a["B"], a["n"], a["Hq"],
        a["Hkv"], a["D"], a["P"], a["NP"], a["MP"], None)
    _err(lib, rc, code, needle)


@pytest.mark.parametrize("bad,code,needle", [
    (dict(n=-1), -1, "max_len"),
    (dict(D=40), -1, "head_dim"),
    (dict(P=0), -1, "page_size"),
    (dict(odt=5), -1, "out_dtype"),
    (dict(cdt=4), -1, "cache_dtype"),
    (dict(lens=0), -1, "null"),
    (dict(vo=0), -1, "null"),
    (dict(vs=0), -1, "E4M3"),
    (dict(ko=24), -1, "aligned"),
    (dict(B=70000), -2, "too many"),
    (dict(n=1 << 30), -2, "too many"),
])
def test_gather_refusals(lib, bad, code, needle):
    a = dict(kc=16, vc=16, ks=16, vs=16, cdt=5, bt=16, lens=16, B=2, n=40, Hkv=2, D=128, P=16,
             NP=8, MP=4, odt=1, ko=16, vo=16)
    a.update(bad)
    rc = lib.spec_kv_gather(vp(a["kc"]), vp(a["vc"]), vp(a["ks"]), vp(a["vs"]), a["cdt"],
                            vp(a["bt"]), None, vp(a["lens"]), a["B"], a["n"], a["Hkv"], a["D"],
                            a["P"], a["NP"], a["MP"], a["odt"], vp(a["ko"]), vp(a["vo"]), None)
    _err(lib, rc, code, needle)


def test_kv_append_e4m3_refusals(lib):
    def call(kn=16, ks=16):
        return lib.spec_kv_append(vp(kn), vp(16), 1, vp(16), vp(16), vp(ks), vp(16), 5, vp(16),
                                  vp(16), 2, 4, 2, 128, 16, 8, 4, None)
    _err(lib, call(ks=0), -1, "E4M3")
    _err(lib, call(kn=24), -1, "aligned")


def test_empty_calls_are_no_ops(lib):
    assert lib.spec_verify_attn_window(*[None] * 8, 0, 4, 8, 2, 128, 16, 8, 4, 1, 5, 0.1, 7, 0,
                                       None, None, None) == 0
    assert lib.spec_kv_gather(None, None, None, None, 5, None, None, None, 3, 0, 2, 128, 16, 8, 4,
                              1, None, None, None) == 0


@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 4.0), ("ntk", 8.0),
                                            ("yarn", 16.0)])
@pytest.mark.parametrize("rot", [32, 96, 128])
def test_rope_table(lib, rot, scaling, factor):
    from speculative_decoding_verification_attn_gb300 import binding
    table, amp = binding.spec_rope_table(rot, 500000.0, scaling, factor, 8192, device="cpu")
    f, amp64 = paged8.freqs64(rot, 500000.0, scaling, factor, 8192)
    assert table.shape == (rot // 2,) and abs(amp - amp64) <= 2.0 ** -24 * amp64
    # the angle of a far position, reduced in whole arithmetic, against the
    # 64-bit product: f and 2 pi are each off by 2^-53, pow by a few of them
    pos = 1_000_003
    for j in range(rot // 2):
        got = Fraction((pos * (int(table[j]) % (1 << 64))) % (1 << 64), 1 << 64)
        want = Fraction(float(f[j])) * pos / Fraction(2 * math.pi)
        off = abs(got - want % 1)
        off = min(off, 1 - off)
        assert off <= float(want) * 2.0 ** -49 + pos * 2.0 ** -64


def test_rope_table_refusals(lib):
    buf = (ctypes.c_uint64 * 128)()
    amp = ctypes.c_float()
    ok = dict(rot=64, theta=1e4, how=0, factor=1.0, orig=0.0, fast=32.0, slow=1.0)
    for bad, needle in [(dict(rot=3), "rotary_dim"), (dict(rot=258), "rotary_dim"),
                        (dict(theta=1.0), "theta"), (dict(theta=math.nan), "theta"),
                        (dict(how=4), "scaling"), (dict(how=1, factor=0.5), "factor"),
                        (dict(how=2, factor=2.0, rot=2), "NTK"),
                        (dict(how=3, factor=2.0, orig=0.0), "original_len"),
                        (dict(how=3, factor=2.0, orig=10.0, fast=1.0, slow=1.0), "slow_turns")]:
        a = dict(ok, **bad)
        rc = lib.spec_rope_table(a["rot"], a["theta"], a["how"], a["factor"], a["orig"], a["fast"],
                                 a["slow"], buf, ctypes.byref(amp))
        _err(lib, rc, -1, needle)
    assert lib.spec_rope_table(64, 1e4, 0, 1.0, 0.0, 0.0, 0.0, None, None) == -1


def test_binding_refuses_mismatched_tensors(lib):
    from speculative_decoding_verification_attn_gb300 import binding
    B, k, Hq, Hkv, D, P, NP = 2, 4, 8, 2, 128, 16, 8
    q = torch.zeros(B, k, Hq, D, dtype=torch.bfloat16)
    kc = torch.zeros(NP, Hkv, P, D, dtype=torch.bfloat16)
    k8 = torch.zeros(NP, Hkv, P, D, dtype=torch.uint8).view(paged8.E4M3)
    bt, ctx = torch.zeros(B, 4, dtype=torch.int32), torch.zeros(B, dtype=torch.int32)
    s = torch.ones(NP, Hkv)
    W = binding.spec_verify_attn_window
    for args, kw in [((q, kc, k8, bt, ctx, k, 0.1, 8, 0, q), {}),
                     ((q, k8, k8, bt, ctx, k, 0.1, 8, 0, q), dict(k_scale=s.half(), v_scale=s)),
                     ((q, k8, k8, bt, ctx, k, 0.1, 8, 0, q), dict(k_scale=s[:3], v_scale=s)),
                     ((q, kc, kc, bt.long(), ctx, k, 0.1, 8, 0, q), {}),
                     ((q, kc, kc, bt[:1], ctx, k, 0.1, 8, 0, q), {}),
                     ((q, kc, kc, bt, ctx, 3, 0.1, 8, 0, q), {}),
                     ((q, kc, kc, bt, ctx, k, 0.1, 8, 0, q.float()), {}),
                     ((q, kc, kc, bt, ctx, k, 0.1, 8, 0, q), {}),  # not on a CUDA device
                     ]:
        with pytest.raises(ValueError):
            W(*args, **kw)
    with pytest.raises(ValueError):
        binding.spec_verify_attn(q, k8, k8, bt, ctx, k, 0.1, q, k_scale=s.half(), v_scale=s)
    kn = torch.zeros(B, k, Hkv, D, dtype=torch.bfloat16)
    R = binding.spec_rope_append
    table = torch.zeros(32, dtype=torch.int64)
    for args, kw in [((q, kn, kn, None, kc, kc, bt, ctx, table), {}),
                     ((q, kn, kn[:, :3], q, kc, kc, bt, ctx, table), {}),
                     ((q.float(), kn, kn, q.float(), kc, kc, bt, ctx, table), {}),
                     ((q, kn.transpose(1, 2).contiguous().transpose(1, 2), kn, q, kc, kc, bt, ctx,
                       table), {}),
                     ((q, kn, kn, q, kc, kc, bt, ctx, table), dict(new_lens=ctx.long())),
                     ((q, kn, kn, q, kc, kc, bt, ctx, table), dict(positions=bt[:, :3])),
                     ((q, kn, kn, q, kc, kc, bt, ctx, table.int()), {})]:
        with pytest.raises(ValueError):
            R(*args, **kw)
    with pytest.raises(ValueError):
        binding.spec_kv_gather(kc, kc, bt, ctx, kn, kn.float())
    with pytest.raises(ValueError):
        binding.spec_rope_table(64, scaling="other", device="cpu")


def test_plain_window_closed_forms():
    """The 64-bit reference itself: window 1 without sinks returns the query's
    own value row; an all-covering window equals no window."""
    g = torch.Generator().manual_seed(1)
    kc, _ = paged8.fill_cache(g, "f32", 4, 1, 8, 32)
    vc, _ = paged8.fill_cache(g, "f32", 4, 1, 8, 32)
    table, ctx = torch.tensor([[2, 0, 3]]), torch.tensor([11])
    q = torch.randn(1, 3, 2, 32, generator=g)
    out, lse, _, _ = paged8.attn64(q, kc, vc, None, None, table, ctx, 0.2, window=1)
    own = paged8.dense64(vc, None, table, 0, 14)[11:14, 0]
    assert torch.allclose(out[0], own[:, None].expand(3, 2, 32))
    a = paged8.attn64(q, kc, vc, None, None, table, ctx, 0.2)
    b = paged8.attn64(q, kc, vc, None, None, table, ctx, 0.2, window=14)
    assert torch.equal(a[0], b[0])
    assert paged8.visible(10, 3, 1, None, 4, 2) == [0, 1, 8, 9, 10, 11]
    assert paged8.visible(10, 3, 2, 0b101, 4, 0) == [8, 9, 10, 12]


def test_binding_checks_int8_scales(lib):
    """The windowed attention, the rotary append and the gather take an int8
    cache's scales as float16 [num_pages, Hkv, P] and nothing else (the library
    sees a bare pointer)."""
    from speculative_decoding_verification_attn_gb300 import binding
    B, k, Hq, Hkv, D, P, NP = 2, 4, 8, 2, 64, 16, 4
    q = torch.zeros(B, k, Hq, D, dtype=torch.bfloat16)
    kn = torch.zeros(B, k, Hkv, D, dtype=torch.bfloat16)
    c8 = torch.zeros(NP, Hkv, P, D, dtype=torch.int8)
    good = torch.zeros(NP, Hkv, P, dtype=torch.float16)
    bt = torch.zeros(B, 2, dtype=torch.int32)
    ctx = torch.zeros(B, dtype=torch.int32)
    for bad in (good.float(), good[:3], good[:, :, 0]):
        for pair in ((bad, good), (good, bad)):
            kw = dict(k_scale=pair[0], v_scale=pair[1])
            with pytest.raises(ValueError, match="int8 cache"):
                binding.spec_verify_attn_window(q, c8, c8, bt, ctx, k, 0.1, 8, 0, q, **kw)
            with pytest.raises(ValueError, match="int8 cache"):
                binding.spec_rope_append(q, kn, kn, q, c8, c8, bt, ctx, None, **kw)
            with pytest.raises(ValueError, match="int8 cache"):
                binding.spec_kv_gather(c8, c8, bt, ctx, kn, kn.clone(), **kw)
