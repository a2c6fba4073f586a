"""Edges of the windowed attention, the e4m3 cache and the rotary append."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from test_gpu_paged8 import attn_case, binding, check_attn, cuda  # noqa: F401

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
