"""Edges of the windowed attention, the e4m3 cache and the rotary append."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from paged8 import E4M3
from test_gpu_paged8 import attn_case, binding, check_attn, cuda, rope_case, run_rope  # noqa: F401

pytestmark = pytest.mark.gpu


def window_call(m, c, window, sinks, mask=None):
    d = {n: cuda(c[n]) for n in ("q", "kc", "vc", "ks", "vs", "table", "ctx")}
    out = torch.full_like(d["q"], float("nan"))
    lse = torch.full(out.shape[:3], float("nan"), device="cuda")
    m.spec_verify_attn_window(d["q"], d["kc"], d["vc"], d["table"], d["ctx"], c["k"], c["scale"],
                              window, sinks, out, lse, d["ks"], d["vs"], tree_mask=cuda(mask))
    return out, lse


# ---------------------------------------------------------------- mask bits
@pytest.mark.parametrize("kind,qdt,D,path", [
    ("bf16", torch.bfloat16, 128, 0), ("i8", torch.bfloat16, 128, 0),
    ("e4m3", torch.bfloat16, 128, 0), ("e4m3", torch.bfloat16, 128, 1),
    ("f32", torch.float32, 64, 0)])
@pytest.mark.parametrize("k,window", [(4, 4), (4, 30), (63, 63)])
def test_window_tree_bits_past_the_drafts(binding, kind, qdt, D, path, k, window):
    """Bits t >= num_draft name no draft: they neither show a key nor move the
    query's position (a row of ones stood up to 63 positions too far)."""
    binding.spec_set_option(binding.SPEC_OPT_ATTN_PATH, path)
    c = attn_case(71, kind, qdt, 2, k, 2, 1, D, 16, [90, 7], window, 2, tree=True)
    want, lse = check_attn(binding, c)
    high = np.int64(-1) << k
    got = window_call(binding, c, window, 2, c["mask"] | int(high))
    assert torch.equal(got[0], want) and torch.equal(got[1], lse)


# ---------------------------------------------------------------- host checks
@pytest.mark.parametrize("kind,D", [("bf16", 128), ("e4m3", 128), ("f32", 64)])
def test_validation_knows_the_window(binding, kind, D):
    """SPEC_OPT_VALIDATE looks at the entries of pages that some query sees and at
    no others (pages behind the window may have left the pool)."""
    m = binding
    qdt = torch.float32 if kind == "f32" else torch.bfloat16
    c = attn_case(72, kind, qdt, 2, 4, 4, 2, D, 16, [300, 11], 64, 20)
    assert int(c["table"][0, 2]) == -1  # freed
    m.spec_set_option(m.SPEC_OPT_VALIDATE, 1)
    try:
        check_attn(m, c)
        first = (300 - 64 + 1) // 16  # page of the first key in the window
        for page in (0, 1, first, 18):  # sinks, window, drafts
            table = c["table"].clone()
            assert int(table[0, page]) >= 0
            table[0, page] = 10 ** 6
            with pytest.raises(m.SpecError) as err:
                window_call(m, dict(c, table=table), 64, 20)
            assert err.value.code == m.SPEC_ERR_INVALID
        assert int(c["table"][0, first - 1]) == -1
        full = c["table"].clamp(min=0)
        with pytest.raises(m.SpecError):  # without a window every page counts
            window_call(m, c, 400, 0)
        window_call(m, dict(c, table=full), 400, 0)
    finally:
        m.spec_set_option(m.SPEC_OPT_VALIDATE, 0)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("window,sinks", [(2 ** 31, 0), (2 ** 32 + 5, 3), (2 ** 40, 2 ** 33),
                                          (7, 2 ** 32 + 1)])
def test_windows_past_32_bits(binding, kind, window, sinks):
    """A window (or a number of sinks) longer than any context sees all of it."""
    c = attn_case(73, kind, torch.bfloat16, 2, 4, 8, 2, 128, 16, [90, 300])
    want = window_call(binding, c, 2 ** 31 - 1, 0)
    got = window_call(binding, c, window, sinks)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    with pytest.raises(binding.SpecError):
        window_call(binding, c, -2 ** 32 + 5, 0)
    with pytest.raises(binding.SpecError):
        window_call(binding, c, 5, -2 ** 32 + 5)


# ---------------------------------------------------------------- append
@pytest.mark.parametrize("kind", ["f32", "bf16", "i8", "e4m3"])
def test_rope_append_negative_context(binding, kind):
    """A sequence whose context is negative writes nothing, also where ctx + t is
    a position again; the others go on."""
    c = rope_case(74, kind, torch.bfloat16, 2, 6, 4, 2, 128, 16, [14, 40])
    bad = dict(c, ctx=torch.tensor([-2, 40]).int())
    table, _ = binding.spec_rope_table(128)
    good = run_rope(binding, c, 128, False, 1.0, table)
    assert binding.spec_device_error() == 0
    got = run_rope(binding, bad, 128, False, 1.0, table)
    assert binding.spec_device_error() == binding.SPEC_DEVERR_CTX
    assert (got["q"] != -7.0).any(-1).all()  # q is rotated all the same
    mine = torch.zeros(c["kc"].shape[0], dtype=torch.bool)
    mine[c["table"][1].clamp(min=0).long()] = c["table"][1] >= 0
    for n in ("kc", "vc", "ks", "vs"):
        if got[n] is None:
            continue
        a, b, g = ((t.view(torch.uint8) if t.dtype == E4M3 else t)
                   for t in (got[n], c[n], good[n]))
        assert torch.equal(a[~mine], b[~mine])
        assert torch.equal(a[mine], g[mine])


@pytest.mark.parametrize("src", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("P,D,kept", [(16, 128, 5), (32, 64, 0), (64, 256, 40)])
def test_e4m3_append_bit_for_bit(binding, src, P, D, kept):
    """Unrotated rows: scales, new codes and the kept rows' codes are the formula's
    in fp32, bit for bit, signed zeros and subnormal codes among them."""
    B, n, Hkv = 4, 20, 3
    gen = torch.Generator().manual_seed(75)
    x = torch.randn(2, B, n, Hkv, D, generator=gen)
    x *= torch.exp(3 * torch.randn(2, B, 1, Hkv, 1, generator=gen))
    x *= torch.rand(x.shape, generator=gen) ** 6  # down to the subnormal codes
    zero = torch.rand(x.shape, generator=gen) < 0.2
    x[zero] = torch.copysign(torch.zeros(()), torch.randn(x.shape, generator=gen)[zero])
    x[0, 3] = torch.copysign(torch.zeros(()), x[0, 3])  # a page of zeros
    x = x.to(src)
    mp = (kept + n + P - 1) // P
    table = torch.randperm(B * mp, generator=gen).int().view(B, mp)
    codes = torch.randint(0, 256, (2, B * mp, Hkv, P, D), generator=gen).to(torch.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0x80  # no NaN
    scale = torch.rand(2, B * mp, Hkv, generator=gen) * 0.05
    old_codes, old_scale = codes.clone(), scale.clone()
    got = [codes[w].view(E4M3).cuda() for w in range(2)]
    gs = [scale[w].cuda() for w in range(2)]
    binding.spec_kv_append(x[0].cuda(), x[1].cuda(), *got, table.cuda(),
                           torch.full((B,), kept).int().cuda(), *gs)
    for w in range(2):
        for b in range(B):
            for g in range(mp):
                page = int(table[b, g])
                lo, hi = max(kept, g * P), min(kept + n, (g + 1) * P)
                if lo >= hi:
                    continue
                rows = x[w, b, lo - kept:hi - kept].float().transpose(0, 1)  # [Hkv, r, D]
                first = lo - g * P
                s = rows.abs().amax((1, 2)) / 448.0
                before = old_scale[w, page].clone()
                if first:
                    s = torch.maximum(s, before)
                old_scale[w, page] = s
                wide = s[:, None, None]
                new = torch.where(wide > 0, rows / wide, torch.zeros(())).to(E4M3)
                old_codes[w, page, :, first:first + hi - lo] = new.view(torch.uint8)
                for h in range(Hkv):
                    if first and s[h] > before[h]:
                        row = old_codes[w, page, h, :first].view(E4M3).float() * before[h]
                        old_codes[w, page, h, :first] = (row / s[h]).to(E4M3).view(torch.uint8)
        assert torch.equal(gs[w].cpu(), old_scale[w])
        off = (got[w].cpu().view(torch.uint8) != old_codes[w]).sum().item()
        assert off == 0, "%d codes differ" % off
