"""Refusals and host logic at the edges of the paged calls.  Runs without a GPU:
every argument check precedes the first CUDA call."""
from __future__ import annotations

import ctypes
import math
import subprocess

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_verification_attn_gb300 import binding, build
    build.build()
    return binding.load()


def vp(x):
    return ctypes.c_void_p(x) if x else None


def attn_args(**kw):
    a = dict(q=16, kc=16, vc=16, ks=None, vs=None, bt=16, ctx=16, mask=None, B=1, k=4, Hq=8, Hkv=2,
             D=128, P=16, NP=8, MP=4, qdt=1, kvdt=1, scale=0.088, window=64, sinks=4, out=16)
    a.update(kw)
    return a


def attend(lib, form, **kw):
    """The status of an attention call of the given form."""
    a = attn_args(**kw)
    head = [vp(a[n]) for n in ("q", "kc", "vc", "ks", "vs", "bt", "ctx")]
    if form != "chain":
        head.append(vp(a["mask"]))
    tail = [a[n] for n in ("B", "k", "Hq", "Hkv", "D", "P", "NP", "MP", "qdt", "kvdt", "scale")]
    if form == "window":
        tail += [a["window"], a["sinks"]]
    name = {"chain": "", "tree": "_tree", "window": "_window"}[form]
    return getattr(lib, "spec_verify_attn" + name)(*head, *tail, vp(a["out"]), None, None)


@pytest.mark.parametrize("form,mask", [("chain", None), ("tree", 16), ("window", None),
                                       ("window", 16)])
@pytest.mark.parametrize("kvdt", [1, 5])
@pytest.mark.parametrize("k,P,MP", [(64, 16, 1), (2, 1, 1), (33, 16, 2)])
def test_tables_too_short_for_the_drafts(lib, form, mask, kvdt, k, P, MP):
    """A block table that cannot hold the drafts' keys is refused: the kernels read
    an entry for each of them."""
    kw = dict(k=k, P=P, MP=MP, mask=mask, kvdt=kvdt, window=64, ks=16, vs=16)
    assert attend(lib, form, **kw) == -1
    assert "block table" in lib.spec_last_error().decode()
    assert attend(lib, form, **dict(kw, B=0)) == 0


GROWTH = r"""
#include <cstdio>
#include <cstdlib>
#include "workspace.h"
int main(int argc, char** argv) {  // need, have, free bytes
    const size_t need = strtoull(argv[1], 0, 10), have = strtoull(argv[2], 0, 10),
                 room = strtoull(argv[3], 0, 10);
    int tries = 0;
    const size_t got = specv::grow_buffer(need, have, [&](size_t n) { ++tries; return n <= room; });
    printf("%zu %d", got, tries);
}
"""


@pytest.fixture(scope="module")
def growth(tmp_path_factory):
    from speculative_decoding_verification_attn_gb300 import build
    d = tmp_path_factory.mktemp("growth")
    (d / "main.cpp").write_text(GROWTH)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I" + build.CSRC, "-o", str(d / "main"),
                    str(d / "main.cpp")], check=True)

    def run(*args):
        out = subprocess.run([str(d / "main"), *map(str, args)], check=True, capture_output=True)
        return tuple(map(int, out.stdout.split()))
    return run


def test_workspace_growth(growth):
    """The workspace doubles (64 MB at least); with less memory than that free it
    takes what the call needs, and nothing when that does not fit either."""
    MB, GB = 1 << 20, 1 << 30
    assert growth(1000, 0, GB) == (64 * MB, 1)
    assert growth(70 * MB, 64 * MB, GB) == (128 * MB, 1)
    assert growth(3 * GB, GB, 4 * GB) == (3 * GB, 1)
    assert growth(GB + GB // 10, GB, GB + GB // 2) == (GB + GB // 10, 2)
    assert growth(1000, 0, 5000) == (1000, 2)
    assert growth(GB + GB // 10, GB, GB) == (0, 2)
    assert growth(3 * GB, GB, GB) == (0, 1)  # the same size is not asked for twice


def paged_tensors(kind):
    """Tensors of a small call on the CPU: q, rows, cache, scale, table, context."""
    B, k, Hq, Hkv, D, P, NP = 2, 4, 8, 2, 64, 16, 4
    cache = torch.zeros(NP, Hkv, P, D, dtype=torch.uint8)
    cache = cache.view(torch.int8 if kind == "i8" else torch.float8_e4m3fn) if kind != "bf16" \
        else cache.bfloat16()
    scale = {"bf16": None, "i8": torch.zeros(NP, Hkv, P, dtype=torch.float16),
             "e4m3": torch.zeros(NP, Hkv)}[kind]
    return dict(q=torch.zeros(B, k, Hq, D, dtype=torch.bfloat16),
                rows=torch.zeros(B, k, Hkv, D, dtype=torch.bfloat16), cache=cache, scale=scale,
                table=torch.zeros(B, 2, dtype=torch.int32), ctx=torch.zeros(B, dtype=torch.int32),
                mask=torch.zeros(B, k, dtype=torch.int64))


def paged_call(binding, call, t, **kw):
    """spec_verify_attn, _tree or spec_kv_append over the tensors t, some replaced."""
    a = dict(v_cache=t["cache"], out=t["q"], lse=None, k_scale=t["scale"], v_scale=t["scale"],
             v_new=t["rows"], table=t["table"], ctx=t["ctx"])
    a.update(kw)
    scales = dict(k_scale=a["k_scale"], v_scale=a["v_scale"])
    if call == "append":
        return binding.spec_kv_append(t["rows"], a["v_new"], t["cache"], a["v_cache"], a["table"],
                                      a["ctx"], **scales)
    args = (t["q"], t["cache"], a["v_cache"], a["table"], a["ctx"])
    if call == "tree":
        args += (t["mask"],)
        return binding.spec_verify_attn_tree(*args, 4, 0.1, a["out"], a["lse"], **scales)
    return binding.spec_verify_attn(*args, 4, 0.1, a["out"], a["lse"], **scales)


@pytest.mark.parametrize("call", ["chain", "tree", "append"])
def test_binding_checks_what_the_library_cannot_see(lib, call):
    """Scales, tables, caches and outputs of another type or size than the pointers
    are taken for are refused by the older calls as well."""
    from speculative_decoding_verification_attn_gb300 import binding
    for kind in ("i8", "e4m3"):
        t = paged_tensors(kind)
        other = t["scale"].float() if kind == "i8" else t["scale"].half()
        for bad in (other, t["scale"][:3], t["scale"][..., 0]):
            for name in ("k_scale", "v_scale"):
                with pytest.raises(ValueError, match="scales of an"):
                    paged_call(binding, call, t, **{name: bad})
    t = paged_tensors("bf16")
    for name in ("table", "ctx"):
        for dt in (torch.int64, torch.int16):
            with pytest.raises(ValueError, match="int32"):
                paged_call(binding, call, t, **{name: t[name].to(dt)})
    for bad in (t["cache"].float(), t["cache"][:3]):
        with pytest.raises(ValueError, match="k_cache and v_cache"):
            paged_call(binding, call, t, v_cache=bad)
    if call == "append":
        with pytest.raises(ValueError, match="k_new and v_new"):
            paged_call(binding, call, t, v_new=t["rows"].float())
    else:
        for bad in (t["q"].float(), t["q"][:1]):
            with pytest.raises(ValueError, match="out must"):
                paged_call(binding, call, t, out=bad)
        with pytest.raises(ValueError, match="lse must"):
            paged_call(binding, call, t, lse=torch.zeros(2, 4, 8, dtype=torch.float64))


class Elsewhere:
    """A tensor that says it lies on another GPU."""

    def __init__(self, t):
        self.t = t

    def __getattr__(self, name):
        return getattr(self.t, name)

    def get_device(self):
        return 1


@pytest.mark.parametrize("call", ["chain", "tree", "append"])
def test_binding_refuses_memory_of_another_device(lib, call, monkeypatch):
    """Kernels launch on the current device: a tensor of another one is refused
    before its pointer reaches them."""
    from speculative_decoding_verification_attn_gb300 import binding
    monkeypatch.setattr(binding, "_get_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 2)
    monkeypatch.setattr(binding, "_gpus", 0)
    t = paged_tensors("bf16")
    for name in ("table", "ctx", "v_new" if call == "append" else "out"):
        where = t["rows"] if name == "v_new" else t["q"] if name == "out" else t[name]
        with pytest.raises(ValueError, match="current device"):
            paged_call(binding, call, t, **{name: Elsewhere(where)})


@pytest.mark.parametrize("B,n,Hq,Hkv", [
    (1, 1, 8, 1 << 30),                # 2 * Hkv is 2^31
    (1 << 16, 1 << 16, 1 << 31 >> 1, 1 << 30),
    (1, 1, (1 << 31) - 1, (1 << 31) - 1), (1 << 30, 1, 0, 1), (1, 1 << 30, 0, 1)])
def test_append_limits_do_not_overflow(lib, B, n, Hq, Hkv):
    """Rows past 2^31 are refused however their number is made up."""
    row = 32 * max(Hq, Hkv)
    q = vp(16 if Hq else 0)
    rc = lib.spec_rope_append(q, vp(16), vp(16), q, row, row, row, row, 1, vp(16), vp(16), vp(16),
                              vp(16), 5, vp(16), vp(16), None, None, vp(16), 0, 0, 1.0, B, n, Hq,
                              Hkv, 32, 16, 8, 4, None)
    assert rc == -2 and "too many" in lib.spec_last_error().decode()


@pytest.mark.parametrize("n,Hkv,D", [(1 << 30, 1 << 30, 256), ((1 << 31) - 1, (1 << 31) - 1, 64),
                                     (1 << 27, 1, 256), (1 << 28, 1, 128)])
def test_gather_limits_do_not_overflow(lib, n, Hkv, D):
    rc = lib.spec_kv_gather(vp(16), vp(16), vp(16), vp(16), 5, vp(16), None, vp(16), 1, n, Hkv, D,
                            16, 8, 4, 1, vp(16), vp(16), None)
    assert rc == -2 and "too many" in lib.spec_last_error().decode()


def test_attention_limits_do_not_overflow(lib):
    big = (1 << 31) - 1
    for NP, Hkv, P in ((big, 1 << 22, big), (1 << 30, 1 << 13, 1 << 30), (1 << 13, 1, 1 << 20)):
        assert attend(lib, "chain", NP=NP, Hkv=Hkv, Hq=Hkv, P=P) == -1
        assert "cache too large" in lib.spec_last_error().decode()
    assert lib.spec_kv_append(vp(16), vp(16), 1, vp(16), vp(16), None, None, 1, vp(16), vp(16),
                              1 << 21, 1 << 21, 1 << 21, 32, 16, 8, 4, None) == -2
    assert "too many" in lib.spec_last_error().decode()


@pytest.mark.parametrize("rot,theta,factor,original", [
    (128, 10000.0, 16.0, 4096), (128, 500000.0, 4.0, 8192), (64, 1e6, 8.0, 32768), (32, 1e4, 2.0, 50)])
def test_rope_table_ramp_by_index(lib, rot, theta, factor, original):
    """The ramp over the pair's index: the table is the formula's in 64 bits (pow, the
    ramp, the sum and the division by 2 pi are off by less than 2^-49 together)."""
    from speculative_decoding_verification_attn_gb300 import binding
    table, amp = binding.spec_rope_table(rot, theta, "yarn-index", factor, original, device="cpu")
    assert abs(amp - (0.1 * math.log(factor) + 1)) <= 2.0 ** -24 * amp

    def border(turns):
        return rot / 2 * math.log(original / (2 * math.pi * turns)) / math.log(theta)
    first = max(0, math.floor(border(32.0)))
    last = max(first + 0.001, min(rot - 1, math.ceil(border(1.0))))
    for j in range(rot // 2):
        f = theta ** (-2 * j / rot)
        keep = 1 - min(1.0, max(0.0, (j - first) / (last - first)))
        want = (keep * f + (1 - keep) * f / factor) / (2 * math.pi) * 2.0 ** 64
        assert abs(int(table[j]) - want) <= 2.0 ** -49 * want + 1


def test_rope_table_ramp_by_index_borders(lib):
    """rot 128, theta 10000, 4096 positions: 64 ln(4096 / 64 pi) / ln 10000 = 20.9 and
    64 ln(4096 / 2 pi) / ln 10000 = 45.03, so pairs up to 20 are kept, pairs from 46 on
    scaled whole and pair 33 half; the other ramp has its own values between."""
    from speculative_decoding_verification_attn_gb300 import binding
    plain, _ = binding.spec_rope_table(128, 10000.0, device="cpu")
    by = {s: binding.spec_rope_table(128, 10000.0, s, 4.0, 4096, device="cpu")[0].double() /
          plain.double() for s in ("yarn", "yarn-index")}
    got = by["yarn-index"]
    assert (got[:21] - 1).abs().max() < 1e-12 and got[21] < 1
    assert (got[46:] - 0.25).abs().max() < 1e-12 and got[45] > 0.25
    assert abs(got[33] - 0.625) < 1e-12
    assert (by["yarn"] / got - 1).abs().max() > 0.2


def test_rope_table_ramp_flag_needs_yarn(lib):
    buf, amp = (ctypes.c_uint64 * 64)(), ctypes.c_float()
    for how in (16, 17, 18, 20, 35):
        assert lib.spec_rope_table(64, 1e4, how, 2.0, 4096.0, 32.0, 1.0, buf,
                                   ctypes.byref(amp)) == -1
        assert "scaling" in lib.spec_last_error().decode()
    assert lib.spec_rope_table(64, 1e4, 19, 2.0, 4096.0, 32.0, 0.0, buf, ctypes.byref(amp)) == 0
    assert lib.spec_rope_table(64, 1e4, 19, 2.0, 0.0, 32.0, 1.0, buf, ctypes.byref(amp)) == -1
