"""GPU parity of the e4m3 cache (one scale per page and kv-head), windowed
attention, the rotary append and the cache read-back against plain 64-bit
implementations, and a run of them together."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import paged8
from paged8 import BF16_HALF_STEP, E4M3

pytestmark = pytest.mark.gpu


@pytest.fixture()
def binding():
    from speculative_decoding_verification_attn_gb300 import binding as m
    m.spec_set_option(m.SPEC_OPT_ATTN_PATH, 0)
    m.spec_device_error()
    yield m
    for opt in (m.SPEC_OPT_ATTN_PATH, m.SPEC_OPT_NUM_CTAS, m.SPEC_OPT_SIMT_CHUNK,
                m.SPEC_OPT_SPLIT_WEIGHT):
        m.spec_set_option(opt, 0)
    assert m.spec_device_error() == 0


def cuda(x):
    return None if x is None else x.cuda()


def random_tree(rng, B, k):
    mask = np.zeros((B, k), np.uint64)
    for b in range(B):
        for i in range(k):
            p = rng.integers(-1, i) if i else -1
            mask[b, i] = (1 << i) | (int(mask[b, p]) if p >= 0 else 0)
    return mask.view(np.int64)


def poison(cache, table, ctx, k, window, sinks):
    """NaN into every slot that no query sees, and page ids off the table."""
    if cache.dtype == torch.int8:
        return
    bad = torch.ones(cache.shape[0], cache.shape[2], dtype=torch.bool)
    for b, c in enumerate(ctx):
        for j in range(c + k):
            if not window or j < sinks or j > c - window:
                bad[int(table[b, j // cache.shape[2]]), j % cache.shape[2]] = False
    if cache.dtype == E4M3:
        raw = cache.view(torch.uint8)
        raw[bad[:, None, :, None].expand_as(raw)] = 0x7F
    else:
        cache[bad[:, None, :, None].expand_as(cache)] = float("nan")


def attn_case(seed, kind, qdt, B, k, Hq, Hkv, D, P, ctx, window=0, sinks=0, tree=False,
              qscale=1.5):
    rng = np.random.default_rng(seed)
    gen = torch.Generator().manual_seed(seed)
    table, NP = paged8.pool(rng, B, [c + k for c in ctx], Hkv, D, P)
    kc, ks = paged8.fill_cache(gen, kind, NP, Hkv, P, D)
    vc, vs = paged8.fill_cache(gen, kind, NP, Hkv, P, D)
    q = (qscale * torch.randn(B, k, Hq, D, generator=gen)).to(qdt)
    mask = random_tree(rng, B, k) if tree else None
    if window:
        # pages that no query sees have left the pool
        for b, c in enumerate(ctx):
            for g in range(table.shape[1]):
                lo, hi = g * P, (g + 1) * P - 1
                if hi <= c - window and lo >= sinks:
                    table[b, g] = -1
    safe = table.clamp(min=0)
    poison(kc, safe, ctx, k, window, sinks)
    poison(vc, safe, ctx, k, window, sinks)
    return dict(q=q, kc=kc, vc=vc, ks=ks, vs=vs, table=table, ctx=torch.tensor(ctx).int(),
                mask=None if mask is None else torch.from_numpy(mask), k=k, window=window,
                sinks=sinks, scale=D ** -0.5)


def check_attn(m, c, seed=None):
    d = {n: cuda(c[n]) for n in ("q", "kc", "vc", "ks", "vs", "table", "ctx", "mask")}
    out = torch.full_like(d["q"], float("nan"))
    lse = torch.full(out.shape[:3], float("nan"), device="cuda")
    if c["window"]:
        m.spec_verify_attn_window(d["q"], d["kc"], d["vc"], d["table"], d["ctx"], c["k"],
                                  c["scale"], c["window"], c["sinks"], out, lse, d["ks"], d["vs"],
                                  tree_mask=d["mask"])
    elif c["mask"] is not None:
        m.spec_verify_attn_tree(d["q"], d["kc"], d["vc"], d["table"], d["ctx"], d["mask"], c["k"],
                                c["scale"], out, lse, d["ks"], d["vs"])
    else:
        m.spec_verify_attn(d["q"], d["kc"], d["vc"], d["table"], d["ctx"], c["k"], c["scale"], out,
                           lse, d["ks"], d["vs"])
    ref, rl, mag, kn = paged8.attn64(c["q"], c["kc"], c["vc"], c["ks"], c["vs"], c["table"],
                                     c["ctx"], c["scale"], c["mask"], c["window"], c["sinks"])
    to, tl = paged8.attn_bounds(c["q"], ref, mag, kn, c["scale"], c["q"].dtype == torch.float32)
    off = (out.double().cpu() - ref).abs()
    assert torch.isfinite(off).all()
    assert (off <= to).all(), "out off by %g, %g allowed" % (off.max(), to[off > to].min())
    empty = torch.isinf(rl)
    got = lse.double().cpu()
    assert torch.equal(torch.isinf(got), empty)
    lo = torch.where(empty, torch.zeros(()).double(), (got - rl).abs())
    assert (lo <= tl).all(), "lse off by %g" % lo.max()
    assert m.spec_device_error() == 0
    return out, lse


# ---------------------------------------------------------------- e4m3 cache
SHAPES = [
    # B, k, Hq, Hkv, P, contexts
    (1, 1, 8, 2, 16, [0]),
    (1, 1, 32, 8, 16, [100]),
    (2, 4, 8, 2, 16, [127, 128]),
    (3, 4, 16, 4, 32, [1, 300, 129]),
    (2, 8, 64, 8, 16, [517, 40]),
    (1, 16, 28, 4, 32, [1000]),
    (2, 16, 16, 2, 64, [255, 700]),
    (1, 5, 10, 2, 128, [383]),
    (1, 3, 12, 2, 256, [511]),
    (4, 2, 4, 4, 16, [16, 15, 17, 260]),
]


@pytest.mark.parametrize("path", [0, 1])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_e4m3_attention(binding, shape, path):
    B, k, Hq, Hkv, P, ctx = SHAPES[shape]
    binding.spec_set_option(binding.SPEC_OPT_ATTN_PATH, path)
    check_attn(binding, attn_case(shape, "e4m3", torch.bfloat16, B, k, Hq, Hkv, 128, P, ctx))


@pytest.mark.parametrize("D,P,qdt,k,Hq,Hkv", [
    (64, 16, torch.bfloat16, 4, 8, 2), (128, 16, torch.float32, 4, 4, 2),
    (256, 16, torch.bfloat16, 3, 4, 1), (128, 3, torch.bfloat16, 4, 8, 2),
    (128, 24, torch.bfloat16, 2, 8, 8), (32, 1, torch.float32, 1, 2, 1),
    (128, 16, torch.bfloat16, 33, 4, 1), (96, 512, torch.bfloat16, 4, 6, 3)])
def test_e4m3_attention_other_shapes(binding, D, P, qdt, k, Hq, Hkv):
    """Shapes off the tensor-core kernel: head sizes, page sizes, fp32 queries,
    more than 128 query rows."""
    check_attn(binding, attn_case(7, "e4m3", qdt, 2, k, Hq, Hkv, D, P, [70, 233]))


@pytest.mark.parametrize("k,Hq,Hkv", [(16, 28, 4), (8, 8, 2), (5, 6, 6), (64, 2, 1)])
def test_e4m3_tree(binding, k, Hq, Hkv):
    check_attn(binding, attn_case(11, "e4m3", torch.bfloat16, 2, k, Hq, Hkv, 128, 16, [0, 203],
                                  tree=True))


@pytest.mark.parametrize("ctas", [1, 3, 40, 400])
def test_e4m3_forced_splits(binding, ctas):
    binding.spec_set_option(binding.SPEC_OPT_NUM_CTAS, ctas)
    check_attn(binding, attn_case(5, "e4m3", torch.bfloat16, 3, 4, 16, 4, 128, 16, [900, 3, 517]))


@pytest.mark.parametrize("ctas", [0, 1, 3, 40, 400])
@pytest.mark.parametrize("k,Hq,Hkv", [(4, 8, 2), (8, 16, 2), (16, 28, 4)])
def test_e4m3_cut_segments(binding, k, Hq, Hkv, ctas):
    """Tables too long for a CTA per segment: segments cut at every place, CTAs
    without a tile among the pieces, 16 to 112 rows."""
    binding.spec_set_option(binding.SPEC_OPT_NUM_CTAS, ctas)
    check_attn(binding, attn_case(6, "e4m3", torch.bfloat16, 3, k, Hq, Hkv, 128, 16,
                                  [2100, 3, 1300]))


def test_e4m3_scales(binding):
    """A page whose scale is zero counts as zero rows; a very large and a very
    small scale keep their rows' weight."""
    c = attn_case(3, "e4m3", torch.bfloat16, 1, 4, 8, 2, 128, 16, [300])
    c["ks"][int(c["table"][0, 2])] = 0.0
    c["vs"][int(c["table"][0, 3])] = 0.0
    c["vs"][int(c["table"][0, 5])] *= 2.0 ** 40
    c["vs"][int(c["table"][0, 7])] *= 2.0 ** -60
    check_attn(binding, c)


def test_e4m3_one_key_outweighs_the_rest(binding):
    """A first key 14 above all others in the exponent (an attention sink) holds
    most of the weight; the many light keys together still count."""
    c = attn_case(9, "e4m3", torch.bfloat16, 1, 2, 8, 2, 128, 32, [2047], qscale=0.0)
    q = torch.zeros_like(c["q"])
    q[..., 0] = 8.0
    c["q"] = q
    kc = torch.zeros(c["kc"].shape)
    page, vpage = int(c["table"][0, 0]), int(c["table"][0, 0])
    kc[page, :, 0, 0] = 20.0
    c["kc"], c["ks"] = kc.to(E4M3), torch.ones_like(c["ks"])
    v = torch.ones(c["vc"].shape)
    v[vpage, :, 0] = 0.0
    c["vc"], c["vs"] = v.to(E4M3), torch.ones_like(c["vs"])
    out, _ = check_attn(binding, c)
    assert out.float().min() > 1e-3  # 2048 keys of e^-14.1: the light keys' share


@pytest.mark.parametrize("qscale", [1e-30, 0.02, 20.0, 200.0])
@pytest.mark.parametrize("k,Hq,Hkv", [(4, 8, 2), (8, 16, 2), (16, 28, 4)])
def test_e4m3_score_ranges(binding, k, Hq, Hkv, qscale):
    """Scores that lie hundreds apart from tile to tile (every reference moves,
    both up and past the block scales' range) and scores that hardly differ."""
    check_attn(binding, attn_case(61, "e4m3", torch.bfloat16, 2, k, Hq, Hkv, 128, 16,
                                  [1500, 333], qscale=qscale))


@pytest.mark.parametrize("order", [1, -1])
@pytest.mark.parametrize("k,Hq,Hkv", [(2, 8, 2), (8, 16, 2), (16, 28, 4)])
def test_e4m3_rising_and_falling_scores(binding, k, Hq, Hkv, order):
    """Keys whose scores climb (or fall) by 30 in the exponent every 100 keys."""
    c = attn_case(62, "e4m3", torch.bfloat16, 1, k, Hq, Hkv, 128, 32, [1300])
    q = 0.3 * c["q"]
    q[..., 0] = 8.0
    c["q"] = q
    x = c["kc"].float() / 448.0
    for j in range(1300 + k):
        at = j if order > 0 else 1300 - j
        x[int(c["table"][0, j // 32]), :, j % 32, 0] = float(at // 100) * 40.0
    x = torch.nan_to_num(x)
    c["ks"] = x.abs().amax((2, 3)).clamp(min=0.01) / 448.0
    c["kc"] = (x / c["ks"][:, :, None, None]).to(E4M3)
    check_attn(binding, c)


def test_e4m3_descriptor_form(binding):
    c = attn_case(2, "e4m3", torch.bfloat16, 2, 4, 8, 2, 128, 16, [60, 200])
    out, lse = check_attn(binding, c)
    o2, l2 = torch.zeros_like(out), torch.zeros_like(lse)
    binding.spec_verify_attn_tensors(cuda(c["q"]), cuda(c["kc"]), cuda(c["vc"]), cuda(c["table"]),
                                     cuda(c["ctx"]), 4, c["scale"], o2, l2, cuda(c["ks"]),
                                     cuda(c["vs"]))
    assert torch.equal(out, o2) and torch.equal(lse, l2)


# ---------------------------------------------------------------- windows
WINDOWS = [(1, 0), (1, 3), (2, 1), (17, 0), (64, 4), (100, 16), (128, 129), (300, 0), (5000, 7),
           (2 ** 31 - 1, 2 ** 31 - 1)]


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "i8"])
@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_window(binding, kind, window, sinks):
    check_attn(binding, attn_case(21, kind, torch.bfloat16, 3, 4, 8, 2, 128, 16, [0, 257, 700],
                                  window, sinks))


@pytest.mark.parametrize("kind,P,k,Hq,Hkv", [("bf16", 64, 16, 28, 4), ("e4m3", 32, 16, 28, 4),
                                             ("e4m3", 128, 8, 64, 8), ("bf16", 256, 1, 8, 8),
                                             ("i8", 32, 8, 16, 2)])
@pytest.mark.parametrize("window,sinks", [(40, 4), (333, 0), (600, 200)])
def test_window_shapes(binding, kind, P, k, Hq, Hkv, window, sinks):
    check_attn(binding, attn_case(22, kind, torch.bfloat16, 2, k, Hq, Hkv, 128, P, [1500, 613],
                                  window, sinks))


@pytest.mark.parametrize("kind,qdt,D,P,k", [("f32", torch.float32, 64, 16, 4),
                                            ("bf16", torch.float32, 128, 16, 9),
                                            ("bf16", torch.bfloat16, 64, 5, 3),
                                            ("i8", torch.bfloat16, 96, 16, 2),
                                            ("e4m3", torch.bfloat16, 64, 16, 4)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (50, 4), (128, 40)])
@pytest.mark.parametrize("chunk", [0, 16, 48])
def test_window_other_shapes(binding, kind, qdt, D, P, k, window, sinks, chunk):
    binding.spec_set_option(binding.SPEC_OPT_SIMT_CHUNK, chunk)
    check_attn(binding, attn_case(23, kind, qdt, 2, k, 4, 2, D, P, [400, 31], window, sinks))


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "i8"])
def test_window_tree(binding, kind):
    check_attn(binding, attn_case(24, kind, torch.bfloat16, 2, 16, 14, 2, 128, 16, [0, 400], 64, 4,
                                  tree=True))


@pytest.mark.parametrize("kind,D", [("bf16", 128), ("e4m3", 128), ("i8", 128), ("f32", 64)])
@pytest.mark.parametrize("window", [0, 8])
def test_rows_that_see_nothing(binding, kind, D, window):
    """A tree row without bits over an empty context: out 0, lse -inf."""
    c = attn_case(25, kind, torch.float32 if kind == "f32" else torch.bfloat16, 2, 4, 4, 2, D, 16,
                  [0, 40], window, 0, tree=True)
    c["mask"][0, 1] = 0
    c["mask"][0, 3] = 0
    binding.spec_set_option(binding.SPEC_OPT_SIMT_CHUNK, 16)
    out, lse = check_attn(binding, c)
    assert (out[0, 1] == 0).all() and torch.isinf(lse[0, 3]).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "i8"])
@pytest.mark.parametrize("ctas", [1, 7, 300])
def test_window_forced_splits(binding, kind, ctas):
    binding.spec_set_option(binding.SPEC_OPT_NUM_CTAS, ctas)
    check_attn(binding, attn_case(26, kind, torch.bfloat16, 4, 3, 8, 2, 128, 16,
                                  [1300, 5, 900, 260], 400, 140))


@pytest.mark.parametrize("ctas", [0, 7, 400])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_window_cut_segments(binding, kind, ctas):
    """As above with a window of more tiles than a CTA takes whole."""
    binding.spec_set_option(binding.SPEC_OPT_NUM_CTAS, ctas)
    check_attn(binding, attn_case(29, kind, torch.bfloat16, 4, 3, 8, 2, 128, 16,
                                  [3100, 5, 2200, 260], 1600, 140))


@pytest.mark.parametrize("ctas", [1, 2, 5, 11, 23])
@pytest.mark.parametrize("kind,window", [("bf16", 200), ("e4m3", 200), ("e4m3", 0)])
def test_ranges_that_end_with_segments(binding, kind, window, ctas):
    """More short segments than CTAs, of very unequal lengths: no segment is cut,
    some CTAs take many and some none."""
    binding.spec_set_option(binding.SPEC_OPT_NUM_CTAS, ctas)
    ctx = [1300, 5, 900, 260, 0, 64] if window else [370, 5, 130, 260, 0, 64]
    check_attn(binding, attn_case(30, kind, torch.bfloat16, 6, 3, 16, 4, 128, 16, ctx, window,
                                  9 if window else 0))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_window_that_covers_all_equals_none(binding, kind):
    c = attn_case(27, kind, torch.bfloat16, 2, 4, 8, 2, 128, 16, [90, 300])
    a, _ = check_attn(binding, c)
    b, _ = check_attn(binding, dict(c, window=4096))
    assert (a.float() - b.float()).abs().max() <= 2 * BF16_HALF_STEP * a.float().abs().max()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_bad_tables_are_flagged(binding, kind):
    c = attn_case(28, kind, torch.bfloat16, 1, 4, 8, 2, 128, 16, [300], 64, 4)
    d = {n: cuda(c[n]) for n in ("q", "kc", "vc", "ks", "vs", "table", "ctx")}
    out = torch.zeros_like(d["q"])

    def call():
        binding.spec_verify_attn_window(d["q"], d["kc"], d["vc"], d["table"], d["ctx"], 4, 0.1, 64,
                                        4, out, None, d["ks"], d["vs"])
        return binding.spec_device_error()

    assert call() == 0
    last = int(d["table"][0, 18])
    d["table"][0, 18] = 10 ** 6
    assert call() == binding.SPEC_DEVERR_PAGE
    d["table"][0, 18] = last
    d["ctx"][0] = 10 ** 6
    d["table"].clamp_(min=0)
    assert call() == binding.SPEC_DEVERR_CTX


# ---------------------------------------------------------------- rotary append
def rope_case(seed, kind, dt, B, n, Hq, Hkv, D, P, ctx, lens=None):
    rng = np.random.default_rng(seed)
    gen = torch.Generator().manual_seed(seed)
    table, NP = paged8.pool(rng, B, [c + n for c in ctx], Hkv, D, P)
    kc, ks = paged8.fill_cache(gen, kind, NP, Hkv, P, D)
    vc, vs = paged8.fill_cache(gen, kind, NP, Hkv, P, D)
    qkv = torch.randn(B, n, Hq + 2 * Hkv, D, generator=gen)
    qkv *= torch.exp(torch.randn(B, n, 1, 1, generator=gen))
    return dict(qkv=qkv.to(dt), Hq=Hq, Hkv=Hkv, kc=kc, vc=vc, ks=ks, vs=vs, table=table,
                ctx=torch.tensor(ctx).int(),
                lens=None if lens is None else torch.tensor(lens).int())


def run_rope(m, c, rot, inter, amp, table, positions=None, in_place=False):
    d = {n: cuda(c[n]) for n in ("qkv", "kc", "vc", "ks", "vs", "table", "ctx", "lens")}
    Hq, Hkv = c["Hq"], c["Hkv"]
    q, k, v = d["qkv"][:, :, :Hq], d["qkv"][:, :, Hq:Hq + Hkv], d["qkv"][:, :, Hq + Hkv:]
    q_out = q if in_place else torch.full(q.shape, -7.0, dtype=q.dtype, device="cuda")
    m.spec_rope_append(q, k, v, q_out, d["kc"], d["vc"], d["table"], d["ctx"], table,
                       interleaved=inter, amplitude=amp, positions=cuda(positions),
                       new_lens=d["lens"], k_scale=d["ks"], v_scale=d["vs"])
    torch.cuda.synchronize()
    return dict(q=q_out.cpu(), **{x: None if d[x] is None else d[x].cpu()
                                  for x in ("kc", "vc", "ks", "vs")})


def check_rows(kind, cache, scale, old, old_scale, table, ctx, lens, x):
    """x [B, n, Hkv, D] fp64 rows at ctx ..; every other slot as it was, but
    for the kept codes of a page whose scale grew."""
    B, n, Hkv, D = x.shape
    P = cache.shape[2]
    raw, raw_old = ((t.view(torch.uint8) if t.dtype == E4M3 else t) for t in (cache, old))
    touched = torch.zeros(cache.shape[0], P, dtype=torch.bool)
    pages = set()
    for b in range(B):
        for t in range(lens[b]):
            pos = int(ctx[b]) + t
            page, slot = int(table[b, pos // P]), pos % P
            touched[page, slot] = True
            pages.add((b, pos // P))
            want = x[b, t]
            if kind == "f32":
                assert ((cache[page, :, slot].double() - want).abs() <=
                        3e-7 * want.abs().amax(-1, keepdim=True)).all()
            elif kind == "bf16":
                lim = BF16_HALF_STEP * 1.001 * want.abs() + 3e-7 * want.abs().amax(-1, keepdim=True)
                assert ((cache[page, :, slot].double() - want).abs() <= lim).all()
            elif kind == "i8":
                s = scale[page, :, slot].double()[:, None]
                top = want.abs().amax(-1, keepdim=True)
                # the code's half step, 127 of an fp16 scale half a step off
                lim = s * 0.5 * (1 + 1e-5) + top * 2.0 ** -11 * 1.01
                assert ((cache[page, :, slot].double() * s - want).abs() <= lim).all()
    if kind != "e4m3":
        keep = ~touched
        assert torch.equal(raw[keep[:, None, :].expand(-1, Hkv, -1)],
                           raw_old[keep[:, None, :].expand(-1, Hkv, -1)])
        return
    val, vold = paged8.value64(cache, scale), paged8.value64(old, old_scale)
    seen = torch.zeros(cache.shape[0], dtype=torch.bool)
    for b, g in pages:
        page = int(table[b, g])
        seen[page] = True
        lo, hi = max(int(ctx[b]), g * P), min(int(ctx[b]) + lens[b], (g + 1) * P)
        rows = x[b, lo - int(ctx[b]):hi - int(ctx[b])].transpose(0, 1)  # [Hkv, r, D]
        kept = lo - g * P
        s = rows.abs().amax((1, 2)) / 448.0
        if kept:
            s = torch.maximum(s, old_scale[page].double())
        assert ((scale[page].double() - s).abs() <= 1e-6 * s).all()
        # a new code: half a step of e4m3 (2^-4 of the value, 2^-10 of the
        # scale among its subnormals), and the fp32 rotation
        lim = (2.0 ** -4 * rows.abs()).clamp(min=0) + (2.0 ** -10 + 1e-4) * s[:, None, None]
        got = val[page, :, kept:kept + hi - lo]
        assert ((got - rows).abs() <= lim).all()
        grew = scale[page] > old_scale[page]
        before, after = vold[page, :, :kept], val[page, :, :kept]
        lim = 2.0 ** -4 * before.abs() + (2.0 ** -10 + 1e-6) * s[:, None, None]
        lim[~grew] = 0
        assert ((after - before).abs() <= lim).all()
        tail = slice(kept + hi - lo, P)
        assert torch.equal(raw[page, :, tail], raw_old[page, :, tail])
    assert torch.equal(raw[~seen], raw_old[~seen])
    assert torch.equal(scale[~seen], old_scale[~seen])


def check_rope(m, c, kind, rot, inter, scaling="none", factor=1.0, positions=None, in_place=False):
    B, n, _, D = c["qkv"].shape
    Hq, Hkv = c["Hq"], c["Hkv"]
    lens = [n] * B if c["lens"] is None else [max(0, min(n, int(v))) for v in c["lens"]]
    table, amp = (None, 1.0)
    f = torch.zeros(0, dtype=torch.float64)
    if rot:
        table, amp = m.spec_rope_table(rot, 10000.0, scaling, factor, 4096)
        f, _ = paged8.freqs64(rot, 10000.0, scaling, factor, 4096)
    got = run_rope(m, c, rot, inter, amp, table, positions, in_place)
    x = c["qkv"].double().clone()
    for b in range(B):
        pos = positions[b].double() if positions is not None else \
            int(c["ctx"][b]) + torch.arange(n).double()
        x[b, :, :Hq + Hkv] = paged8.rotate64(c["qkv"][b, :, :Hq + Hkv], pos, f, amp, inter)
        want = x[b, :lens[b], :Hq]
        lim = 3e-7 * want.abs().amax(-1, keepdim=True) if want.numel() else 0
        if c["qkv"].dtype == torch.bfloat16:
            lim = lim + BF16_HALF_STEP * 1.001 * want.abs()
        assert ((got["q"][b, :lens[b]].double() - want).abs() <= lim).all()
        rest = got["q"][b, lens[b]:]
        assert (rest == (c["qkv"][b, lens[b]:, :Hq] if in_place else -7.0)).all()
    for w, part in (("k", x[:, :, Hq:Hq + Hkv]), ("v", x[:, :, Hq + Hkv:])):
        check_rows(kind, got[w + "c"], got[w + "s"], c[w + "c"], c[w + "s"], c["table"], c["ctx"],
                   lens, part)
    assert m.spec_device_error() == 0
    return got


@pytest.mark.parametrize("kind", ["f32", "bf16", "i8", "e4m3"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rot,D", [(128, 128), (64, 128), (16, 32), (0, 64), (96, 96), (256, 256),
                                   (32, 160)])
def test_rope_append(binding, kind, inter, rot, D):
    c = rope_case(31, kind, torch.bfloat16, 3, 4, 6, 2, D, 16, [0, 13, 40])
    check_rope(binding, c, kind, rot, inter)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("scaling,factor", [("linear", 8.0), ("ntk", 4.0), ("yarn", 16.0)])
def test_rope_append_scaled_and_far(binding, kind, scaling, factor):
    """Far positions: fp32 holds the angle only because it is reduced first."""
    c = rope_case(32, kind, torch.bfloat16, 2, 3, 4, 2, 128, 16, [5, 8])
    pos = torch.tensor([[131071, 1000003, 16777217], [7, 99999999, 2147483647]]).int()
    check_rope(binding, c, kind, 128, False, scaling, factor, positions=pos)


@pytest.mark.parametrize("kind", ["bf16", "i8", "e4m3"])
@pytest.mark.parametrize("P", [1, 3, 16, 64, 256])
@pytest.mark.parametrize("n", [1, 5, 37, 300])
def test_rope_append_lengths_and_pages(binding, kind, P, n):
    c = rope_case(33, kind, torch.bfloat16, 2, n, 2, 3, 64, P, [3, 66])
    check_rope(binding, c, kind, 64, False)


@pytest.mark.parametrize("kind", ["f32", "e4m3"])
@pytest.mark.parametrize("D", [128, 256])
def test_rope_append_f32_source(binding, kind, D):
    c = rope_case(34, kind, torch.float32, 2, 20, 4, 9, D, 32, [30, 0])
    check_rope(binding, c, kind, 64, True)


@pytest.mark.parametrize("kind", ["bf16", "i8", "e4m3"])
def test_rope_append_padded_batch(binding, kind):
    """Sequences of unequal lengths, one of none, one past the padding."""
    c = rope_case(35, kind, torch.bfloat16, 5, 21, 4, 2, 128, 16, [0, 5, 100, 31, 16],
                  lens=[21, 0, 7, 1, 1000])
    check_rope(binding, c, kind, 128, True)


@pytest.mark.parametrize("P,n,inter,src", [
    (16, 1024, False, torch.bfloat16), (16, 1024, True, torch.float32),
    (64, 4096, False, torch.float32), (64, 4096, True, torch.bfloat16)])
def test_rope_append_many_pages(binding, P, n, inter, src):
    """A call of so many pages that a block takes several groups of heads writes
    what one call per sequence writes, bit for bit (partly filled pages, ragged
    lengths, a last group of its own)."""
    B, Hq, Hkv, D, rot = 8, 2, 12, 32, 32
    gen = torch.Generator(device="cuda").manual_seed(P)
    q, k, v = (torch.randn(B, n, H, D, device="cuda", generator=gen).to(src)
               for H in (Hq, Hkv, Hkv))
    k *= torch.rand(B, n, 1, 1, device="cuda", generator=gen).add(0.1).to(src)
    mp = (n + 2 * P - 1) // P + 1
    table = torch.randperm(B * mp, device="cuda", generator=gen).int().view(B, mp)
    ctx = torch.tensor([0, 1, P - 1, 5, P, 7, 3, 2], dtype=torch.int32, device="cuda")
    lens = torch.tensor([n, n - 1, n // 2, 0, 1, n, n - 17, 33], dtype=torch.int32, device="cuda")
    kc, vc = (torch.randint(0, 0x78, (B * mp, Hkv, P, D), device="cuda", generator=gen)
              .to(torch.uint8).view(paged8.E4M3) for _ in range(2))
    ks, vs = (torch.rand(B * mp, Hkv, device="cuda", generator=gen) * 0.02 for _ in range(2))
    rope, amp = binding.spec_rope_table(rot)
    one = [t.clone() for t in (kc, vc, ks, vs)]
    qo, qone = torch.zeros_like(q), torch.zeros_like(q)
    binding.spec_rope_append(q, k, v, qo, kc, vc, table, ctx, rope, inter, amp, new_lens=lens,
                             k_scale=ks, v_scale=vs)
    for b in range(B):
        s = slice(b, b + 1)
        binding.spec_rope_append(q[s], k[s], v[s], qone[s], one[0], one[1], table[s], ctx[s], rope,
                                 inter, amp, new_lens=lens[s], k_scale=one[2], v_scale=one[3])
    assert torch.equal(qo, qone)
    for got, want in zip((kc, vc), one[:2]):
        assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))
    assert torch.equal(ks, one[2]) and torch.equal(vs, one[3])


def test_rope_append_in_place(binding):
    c = rope_case(36, "e4m3", torch.bfloat16, 2, 6, 8, 2, 128, 16, [9, 64])
    check_rope(binding, c, "e4m3", 128, False, in_place=True)


def test_rope_append_without_queries_is_kv_append(binding):
    c = rope_case(37, "e4m3", torch.bfloat16, 2, 6, 4, 2, 128, 16, [9, 64])
    got = check_rope(binding, c, "e4m3", 0, False)
    d = {n: cuda(c[n]) for n in ("qkv", "kc", "vc", "ks", "vs", "table", "ctx")}
    k, v = d["qkv"][:, :, 4:6].contiguous(), d["qkv"][:, :, 6:].contiguous()
    binding.spec_kv_append(k, v, d["kc"], d["vc"], d["table"], d["ctx"], d["ks"], d["vs"])
    for n in ("kc", "vc"):
        assert torch.equal(d[n].cpu().view(torch.uint8), got[n].view(torch.uint8))
    assert torch.equal(d["ks"].cpu(), got["ks"]) and torch.equal(d["vs"].cpu(), got["vs"])


@pytest.mark.parametrize("kind", ["bf16", "i8"])
def test_rope_append_matches_kv_append_unrotated(binding, kind):
    """Nothing rotated: bit for bit what spec_kv_append writes."""
    c = rope_case(38, kind, torch.bfloat16, 3, 5, 4, 2, 128, 16, [9, 64, 0])
    got = check_rope(binding, c, kind, 0, False)
    d = {n: cuda(c[n]) for n in ("qkv", "kc", "vc", "ks", "vs", "table", "ctx")}
    k, v = d["qkv"][:, :, 4:6].contiguous(), d["qkv"][:, :, 6:].contiguous()
    binding.spec_kv_append(k, v, d["kc"], d["vc"], d["table"], d["ctx"], d["ks"], d["vs"])
    for n in ("kc", "vc", "ks", "vs"):
        if got[n] is not None:
            assert torch.equal(d[n].cpu(), got[n])


def test_page_scale_starts_afresh_and_grows(binding):
    """The first slot resets the page's scale, later rows only raise it, zero
    rows give scale 0 and code 0."""
    kc = torch.zeros(2, 1, 16, 64, dtype=torch.uint8, device="cuda").view(E4M3)
    vc, table = kc.clone(), torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    ks, vs = torch.full((2, 1), 5.0, device="cuda"), torch.full((2, 1), 5.0, device="cuda")
    seen = []
    for pos, mag in [(0, 0.0), (1, 448.0), (2, 4.48), (3, 896.0), (0, 44.8)]:
        ctx = torch.tensor([pos], dtype=torch.int32, device="cuda")
        x = torch.zeros(1, 1, 1, 64, device="cuda")
        x[..., 3] = mag
        binding.spec_kv_append(x, -x, kc, vc, table, ctx, ks, vs)
        seen.append((float(ks[0, 0]), float(kc.view(torch.uint8).view(E4M3).float()[0, 0, pos, 3])))
    one = float(torch.tensor(44.8) / 448)
    assert [s for s, _ in seen] == [0.0, 1.0, 1.0, 2.0, one]
    assert [c for _, c in seen] == [0.0, 448.0, 4.5, 448.0, 448.0]
    assert float(vs[0, 0]) == one and float(ks[1, 0]) == 5.0


@pytest.mark.parametrize("kind", ["bf16", "i8", "e4m3"])
def test_rope_append_flags_bad_positions(binding, kind):
    c = rope_case(39, kind, torch.bfloat16, 2, 4, 4, 2, 128, 16, [14, 40])
    table, _ = binding.spec_rope_table(128)

    def flags(**kw):
        d = dict(c, **kw)
        got = run_rope(binding, d, 128, False, 1.0, table)
        assert (got["q"] != -7.0).any(-1).all()  # q is rotated all the same
        return binding.spec_device_error(), got

    bad = c["table"].clone()
    bad[0, 1] = 10 ** 6
    code, got = flags(table=bad)
    assert code == binding.SPEC_DEVERR_PAGE
    code, _ = flags(ctx=torch.tensor([14, 10 ** 6]).int())
    assert code == binding.SPEC_DEVERR_CTX
    code, got = flags(ctx=torch.tensor([-9, -10 ** 6]).int())
    assert code == binding.SPEC_DEVERR_CTX
    for n in ("kc", "vc"):
        a, b = got[n], c[n]
        if kind == "e4m3":
            a, b = a.view(torch.uint8), b.view(torch.uint8)
        assert torch.equal(a, b)


# ---------------------------------------------------------------- read-back
@pytest.mark.parametrize("kind", ["f32", "bf16", "i8", "e4m3"])
@pytest.mark.parametrize("odt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("P,D,Hkv", [(16, 128, 8), (1, 32, 3), (24, 96, 1), (256, 256, 2)])
def test_gather(binding, kind, odt, P, D, Hkv):
    rng = np.random.default_rng(41)
    gen = torch.Generator().manual_seed(41)
    lens, starts = [0, 1, 130, 61], [4, 0, 17, 255]
    table, NP = paged8.pool(rng, 4, [a + b for a, b in zip(lens, starts)], Hkv, D, P)
    d = {}
    for w in "kv":
        d[w], d[w + "s"] = paged8.fill_cache(gen, kind, NP, Hkv, P, D)
    out = {w: torch.full((4, 130, Hkv, D), -3.0, dtype=odt, device="cuda") for w in "kv"}
    call = dict(starts=torch.tensor(starts).int().cuda(), k_scale=cuda(d["ks"]),
                v_scale=cuda(d["vs"]))
    binding.spec_kv_gather(cuda(d["k"]), cuda(d["v"]), table.cuda(),
                           torch.tensor(lens).int().cuda(), out["k"], out["v"], **call)
    for w in "kv":
        s = d[w + "s"]
        val = d[w].float()
        if s is not None:
            val = val * (s[:, :, None, None] if s.dim() == 2 else s.float()[..., None])
        for b in range(4):
            got = out[w][b].cpu()
            for t in range(lens[b]):
                pos = starts[b] + t
                want = val[int(table[b, pos // P]), :, pos % P].to(odt)
                assert torch.equal(got[t], want)
            assert (got[lens[b]:] == -3.0).all()
    assert binding.spec_device_error() == 0


def test_gather_flags_bad_tables(binding):
    gen = torch.Generator().manual_seed(42)
    k, s = paged8.fill_cache(gen, "e4m3", 4, 2, 16, 64)
    table = torch.tensor([[1, 7, -1, 2]]).int().cuda()
    o1, o2 = (torch.full((1, 80, 2, 64), -3.0, device="cuda") for _ in range(2))
    args = (cuda(k), cuda(k), table, torch.tensor([80]).int().cuda(), o1, o2)
    binding.spec_kv_gather(*args, k_scale=cuda(s), v_scale=cuda(s))
    assert binding.spec_device_error() == (binding.SPEC_DEVERR_PAGE | binding.SPEC_DEVERR_CTX)
    assert (o1[0, 16:48] == -3.0).all() and (o2[0, 64:] == -3.0).all()
    assert (o1[0, :16] != -3.0).any() and (o1[0, 48:64] != -3.0).any()
    binding.spec_kv_gather(*args, starts=torch.tensor([-5]).int().cuda(), k_scale=cuda(s),
                           v_scale=cuda(s))
    assert binding.spec_device_error() & binding.SPEC_DEVERR_CTX


# ---------------------------------------------------------------- together
class Engine:
    """A layer of a serving loop: prompts, then verification steps."""

    def __init__(self, m, kind, seed, B=3, Hq=8, Hkv=2, P=16, MP=24, window=0, sinks=0):
        self.m, self.kind, self.B, self.Hq, self.Hkv, self.P = m, kind, B, Hq, Hkv, P
        self.window, self.sinks = window, sinks
        self.gen = torch.Generator().manual_seed(seed)
        ids = torch.randperm(B * MP + 5, generator=self.gen)[:B * MP].int()
        self.table = ids.view(B, MP).cuda()
        NP = B * MP + 5
        kc, ks = paged8.fill_cache(self.gen, kind, NP, Hkv, P, 128)
        vc, vs = paged8.fill_cache(self.gen, kind, NP, Hkv, P, 128)
        self.kc, self.vc, self.ks, self.vs = kc.cuda(), vc.cuda(), cuda(ks), cuda(vs)
        self.ctx = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.rope, self.amp = m.spec_rope_table(128, 1e6, "yarn", 4.0, 64)

    def qkv(self, n):
        return torch.randn(self.B, n, self.Hq + 2 * self.Hkv, 128,
                           generator=self.gen).bfloat16().cuda()

    def append(self, qkv, lens=None, positions=None):
        H, K = self.Hq, self.Hkv
        q = torch.empty(qkv.shape[0], qkv.shape[1], H, 128, dtype=qkv.dtype, device="cuda")
        self.m.spec_rope_append(qkv[:, :, :H], qkv[:, :, H:H + K], qkv[:, :, H + K:], q, self.kc,
                                self.vc, self.table, self.ctx, self.rope, amplitude=self.amp,
                                positions=positions, new_lens=lens, k_scale=self.ks,
                                v_scale=self.vs)
        return q

    def attend(self, q, mask=None):
        out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
        args = (q, self.kc, self.vc, self.table, self.ctx, q.shape[1], 128 ** -0.5)
        if self.window:
            self.m.spec_verify_attn_window(*args, self.window, self.sinks, out, lse, self.ks,
                                           self.vs, tree_mask=mask)
        elif mask is not None:
            self.m.spec_verify_attn_tree(*args[:5], mask, *args[5:], out, lse, self.ks, self.vs)
        else:
            self.m.spec_verify_attn(*args, out, lse, self.ks, self.vs)
        return out, lse


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "i8"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (48, 4)])
def test_serving_run(binding, kind, window, sinks):
    """Prompts of unequal lengths, then steps of drafts: append, verify, accept,
    commit; the cache read back holds every accepted row."""
    m = binding
    e = Engine(m, kind, 51, window=window, sinks=sinks)
    lens = torch.tensor([70, 1, 33], dtype=torch.int32)
    prompt = e.qkv(70)
    e.append(prompt, lens.cuda())
    e.ctx += lens.cuda()
    kept = [[prompt[b, :int(lens[b])].cpu()] for b in range(3)]
    k = 4
    for step in range(6):
        x = e.qkv(k)
        q = e.append(x)
        out, lse = e.attend(q)
        host = {n: None if getattr(e, n) is None else getattr(e, n).cpu()
                for n in ("kc", "vc", "ks", "vs", "table", "ctx")}
        ref, rl, mag, kn = paged8.attn64(q.cpu(), host["kc"], host["vc"], host["ks"], host["vs"],
                                         host["table"], host["ctx"], 128 ** -0.5, None, window,
                                         sinks)
        to, tl = paged8.attn_bounds(q.cpu(), ref, mag, kn, 128 ** -0.5)
        assert ((out.double().cpu() - ref).abs() <= to).all()
        assert ((lse.double().cpu() - rl).abs() <= tl).all()
        logits = torch.randn(3, k + 1, 50, generator=e.gen).cuda()
        drafts = logits[:, :k].argmax(-1).int()
        drafts[step % 3, step % k] = 49 - drafts[step % 3, step % k]  # one miss
        acc, nxt = (torch.zeros(3, dtype=torch.int32, device="cuda") for _ in range(2))
        m.spec_accept_greedy(logits, drafts, k, acc, nxt)
        m.spec_commit(e.ctx, acc, 0)
        for b in range(3):
            kept[b].append(x[b, :int(acc[b])].cpu())
    n = int(e.ctx.max())
    ko, vo = (torch.zeros(3, n, e.Hkv, 128, device="cuda") for _ in range(2))
    m.spec_kv_gather(e.kc, e.vc, e.table, e.ctx, ko, vo, k_scale=e.ks, v_scale=e.vs)
    f, amp = paged8.freqs64(128, 1e6, "yarn", 4.0, 64)
    for b in range(3):
        rows = torch.cat(kept[b])
        assert rows.shape[0] == int(e.ctx[b])
        pos = torch.arange(rows.shape[0]).double()
        kw = paged8.rotate64(rows[:, e.Hq:e.Hq + e.Hkv], pos, f, amp, False)
        for got, want in ((ko, kw), (vo, rows[:, e.Hq + e.Hkv:].double())):
            off = (got[b, :rows.shape[0]].double().cpu() - want).abs()
            # bf16: half a step; e4m3: half a step when written and at most
            # once more for each of the few growths of its page's scale
            top = want.abs().max()
            lim = {"bf16": BF16_HALF_STEP * 1.01 * want.abs() + 1e-6 * top,
                   "i8": (0.5 / 127 + 2.0 ** -10) * top + 0 * want,
                   "e4m3": 6 * (2.0 ** -4 * want.abs() + 2.0 ** -10 * top / 448) + 1e-5 * top}[kind]
            assert (off <= lim).all()
    assert m.spec_device_error() == 0


def test_tree_step_with_depth_positions(binding):
    """A tree's nodes rotate by their depth; siblings share a position."""
    m = binding
    e = Engine(m, "e4m3", 52, B=2)
    e.append(e.qkv(40))
    e.ctx += 40
    mask = torch.tensor([[1, 3, 5, 11], [1, 3, 7, 15]], dtype=torch.int64)
    depth = torch.tensor([[0, 1, 1, 2], [0, 1, 2, 3]], dtype=torch.int32)
    x = e.qkv(4)
    q = e.append(x, positions=(e.ctx[:, None] + depth.cuda()).int().contiguous())
    f, amp = paged8.freqs64(128, 1e6, "yarn", 4.0, 64)
    for b in range(2):
        want = paged8.rotate64(x[b, :, :e.Hq].cpu(), 40 + depth[b].double(), f, amp, False)
        assert ((q[b].double().cpu() - want).abs() <= BF16_HALF_STEP * 1.001 * want.abs() +
                3e-7 * want.abs().amax(-1, keepdim=True)).all()
    out, lse = e.attend(q, mask.cuda())
    ref, rl, mag, kn = paged8.attn64(q.cpu(), e.kc.cpu(), e.vc.cpu(), e.ks.cpu(), e.vs.cpu(),
                                     e.table.cpu(), e.ctx.cpu(), 128 ** -0.5, mask)
    to, _ = paged8.attn_bounds(q.cpu(), ref, mag, kn, 128 ** -0.5)
    assert ((out.double().cpu() - ref).abs() <= to).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_captured_step_replays(binding, kind):
    """A step captured on a side stream and replayed with new inputs, also after
    the library's workspace has grown, equals the eager step."""
    m = binding
    e = Engine(m, kind, 53, window=40, sinks=2)
    e.append(e.qkv(60))
    e.ctx += 60
    x, side = e.qkv(4), torch.cuda.Stream()
    ko, vo = (torch.zeros(3, 80, e.Hkv, 128, dtype=torch.bfloat16, device="cuda")
              for _ in range(2))

    def step():
        q = e.append(x)
        o = e.attend(q)
        m.spec_kv_gather(e.kc, e.vc, e.table, e.ctx, ko, vo, k_scale=e.ks, v_scale=e.vs)
        return q, *o

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = step()
    for round_ in range(3):
        x.copy_(e.qkv(4))
        e.ctx += 2
        if round_ == 1:  # a call that needs a larger workspace than the step's
            V = 128256
            lg = torch.zeros(64, 17, V, dtype=torch.bfloat16, device="cuda")
            dr, r = torch.zeros(64, 16, dtype=torch.int32, device="cuda"), \
                torch.zeros(2, 64, dtype=torch.int32, device="cuda")
            m.spec_accept_rejection(lg, lg[:, :16].contiguous(), dr, 16, 1.0, 1, r[0], r[1])
            c = attn_case(54, "bf16", torch.float32, 2, 16, 16, 1, 256, 16, [3000, 2000])
            m.spec_set_option(m.SPEC_OPT_SIMT_CHUNK, 16)
            check_attn(m, c)
            m.spec_set_option(m.SPEC_OPT_SIMT_CHUNK, 0)
        saved = [None if t is None else t.clone() for t in (e.kc, e.vc, e.ks, e.vs)]
        graph.replay()
        torch.cuda.synchronize()
        first = [t.clone() for t in got] + [ko.clone(), vo.clone()]
        for t, s in zip((e.kc, e.vc, e.ks, e.vs), saved):
            if t is not None:
                (t.view(torch.uint8) if t.dtype == E4M3 else t).copy_(
                    s.view(torch.uint8) if t.dtype == E4M3 else s)
        eager = list(step()) + [ko, vo]
        for a, b in zip(first, eager):
            assert torch.equal(a, b)
    assert m.spec_device_error() == 0


def test_capture_refuses_to_grow_the_workspace(binding):
    m = binding
    m.spec_release()
    c = attn_case(55, "e4m3", torch.bfloat16, 1, 4, 8, 2, 128, 16, [40], 16, 0)
    d = {n: cuda(c[n]) for n in ("q", "kc", "vc", "ks", "vs", "table", "ctx")}
    out = torch.empty_like(d["q"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    keep = torch.zeros(1, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        keep += 1
        with pytest.raises(m.SpecError) as err:
            m.spec_verify_attn_window(d["q"], d["kc"], d["vc"], d["table"], d["ctx"], 4, 0.1, 16,
                                      0, out, None, d["ks"], d["vs"])
        assert err.value.code == m.SPEC_ERR_UNSUPPORTED
    check_attn(m, c)
    graph.replay()
    torch.cuda.synchronize()


def test_calls_on_another_stream(binding):
    m = binding
    c = attn_case(56, "e4m3", torch.bfloat16, 2, 4, 8, 2, 128, 16, [200, 90], 64, 4)
    want, _ = check_attn(m, c)
    d = {n: cuda(c[n]) for n in ("q", "kc", "vc", "ks", "vs", "table", "ctx")}
    out = torch.zeros_like(want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    m.spec_verify_attn_window(d["q"], d["kc"], d["vc"], d["table"], d["ctx"], 4, c["scale"], 64, 4,
                              out, None, d["ks"], d["vs"], stream=s)
    s.synchronize()
    assert torch.equal(out, want)


def test_results_do_not_vary(binding):
    """The same call twice gives the same bits (no order of atomics in it)."""
    c = attn_case(57, "e4m3", torch.bfloat16, 4, 8, 16, 2, 128, 16, [2000, 30, 900, 1500])
    a = check_attn(binding, c)
    for _ in range(5):
        b = check_attn(binding, c)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
