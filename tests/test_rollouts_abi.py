"""Refusals and host logic of the shared-prefix attention, the forking, releasing
and compacting of a paged cache and the token log probabilities.  Runs without
a GPU: every argument check precedes the first CUDA call."""
from __future__ import annotations

import ctypes
import math

import pytest
import torch

import paged8
import rollouts


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


CACHE = dict(kc=16, vc=16, ks=None, vs=None, cdt=1, bt=16, ctx=16, Hkv=2, D=128, P=16, NP=8, MP=4)
BAD_CACHE = [
    (dict(Hkv=0), -1, "num_kv_heads"),
    (dict(D=48), -1, "head_dim"),
    (dict(D=288), -1, "head_dim"),
    (dict(P=0), -1, "page_size"),
    (dict(NP=0), -1, "num_pages"),
    (dict(MP=0), -1, "max_pages"),
    (dict(cdt=2), -1, "cache_dtype"),
    (dict(cdt=3), -1, "I8"),
    (dict(cdt=5), -1, "E4M3"),
    (dict(cdt=5, ks=16, vs=18), -1, "4-byte"),
    (dict(kc=24), -1, "aligned"),
    (dict(vc=None), -1, "null"),
    (dict(bt=None), -1, "null"),
    (dict(ctx=None), -1, "null"),
    (dict(NP=2 ** 31 - 1, P=2 ** 20), -1, "too large"),
    (dict(NP=1, P=2 ** 24), -2, "page too large"),
]


@pytest.mark.parametrize("bad,code,needle", BAD_CACHE + [
    (dict(B=-1), -1, "batch"),
    (dict(B=65536), -2, "batch"),
    (dict(k=0), -1, "num_draft"),
    (dict(k=65), -1, "num_draft"),
    (dict(path=None), -1, "null"),
    (dict(acc=None), -1, "null"),
])
def test_compact_refusals(lib, bad, code, needle):
    a = dict(CACHE, path=16, acc=16, B=1, k=4)
    a.update(bad)
    rc = lib.spec_kv_compact(vp(a["kc"]), vp(a["vc"]), vp(a["ks"]), vp(a["vs"]), a["cdt"],
                             vp(a["bt"]), vp(a["ctx"]), vp(a["path"]), vp(a["acc"]), a["B"], a["k"],
                             a["Hkv"], a["D"], a["P"], a["NP"], a["MP"], None)
    _err(lib, rc, code, needle)


@pytest.mark.parametrize("bad,code,needle", BAD_CACHE + [
    (dict(n=-1), -1, "num_pairs"),
    (dict(n=1 << 24), -2, "num_pairs"),
    (dict(room=-1), -1, "room"),
    (dict(rows=0), -1, "num_rows"),
    (dict(par=None), -1, "null"),
    (dict(kid=None), -1, "null"),
    (dict(refs=None), -1, "null"),
])
def test_fork_refusals(lib, bad, code, needle):
    a = dict(CACHE, refs=16, par=16, kid=16, n=1, room=4, rows=2)
    a.update(bad)
    rc = lib.spec_kv_fork(vp(a["kc"]), vp(a["vc"]), vp(a["ks"]), vp(a["vs"]), a["cdt"], vp(a["bt"]),
                          vp(a["ctx"]), vp(a["refs"]), vp(a["par"]), vp(a["kid"]), a["n"], a["room"],
                          a["rows"], a["Hkv"], a["D"], a["P"], a["NP"], a["MP"], None)
    _err(lib, rc, code, needle)


@pytest.mark.parametrize("bad,code,needle", [
    (dict(n=-1), -1, "num < 0"),
    (dict(rows=0), -1, "num_rows"),
    (dict(P=0), -1, "page_size"),
    (dict(NP=0), -1, "num_pages"),
    (dict(bt=None), -1, "null"),
    (dict(refs=None), -1, "null"),
    (dict(which=None), -1, "null"),
])
def test_release_refusals(lib, bad, code, needle):
    a = dict(bt=16, ctx=16, refs=16, which=16, keep=None, n=1, rows=2, P=16, NP=8, MP=4)
    a.update(bad)
    rc = lib.spec_kv_release(vp(a["bt"]), vp(a["ctx"]), vp(a["refs"]), vp(a["which"]),
                             vp(a["keep"]), a["n"], a["rows"], a["P"], a["NP"], a["MP"], None)
    _err(lib, rc, code, needle)


@pytest.mark.parametrize("bad,code,needle", [
    (dict(B=-1), -1, "batch"),
    (dict(n=0), -1, "num_rows"),
    (dict(V=0), -1, "vocab"),
    (dict(V=2 ** 31 - 1), -1, "vocab"),
    (dict(dt=2), -1, "logits_dtype"),
    (dict(T=0.0), -1, "temperature"),
    (dict(T=-1.0), -1, "temperature"),
    (dict(T=math.nan), -1, "temperature"),
    (dict(T=math.inf), -1, "temperature"),
    (dict(T=1e-32), -1, "temperature"),
    (dict(K=-1), -1, "num_top"),
    (dict(K=33), -1, "num_top"),
    (dict(ids=None), -1, "num_top > 0"),
    (dict(x=24), -1, "aligned"),
    (dict(tok=None), -1, "null"),
    (dict(lp=None), -1, "null"),
    (dict(B=2 ** 20, n=2 ** 10), -2, "too many rows"),
])
def test_logprob_refusals(lib, bad, code, needle):
    a = dict(x=16, dt=1, tok=16, lens=None, B=2, n=3, V=1000, T=1.0, K=4, lp=16, ent=None, ids=16,
             top=None)
    a.update(bad)
    rc = lib.spec_token_logprobs(vp(a["x"]), a["dt"], vp(a["tok"]), vp(a["lens"]), a["B"], a["n"],
                                 a["V"], a["T"], a["K"], vp(a["lp"]), vp(a["ent"]), vp(a["ids"]),
                                 vp(a["top"]), None)
    _err(lib, rc, code, needle)


@pytest.mark.parametrize("bad,code,needle", [
    (dict(groups=-1), -1, "num_groups"),
    (dict(starts=None), -1, "group_starts"),
    (dict(lens=None), -1, "shared_lens"),
    (dict(k=65), -1, "num_draft"),
    (dict(Hq=6, Hkv=4), -1, "multiple"),
    (dict(D=100), -1, "head_dim"),
    (dict(kvdt=2), -1, "kv_dtype"),
    (dict(kvdt=3), -1, "I8"),
    (dict(q=None), -1, "null"),
    (dict(out=24), -1, "aligned"),
    (dict(k=64, P=16, MP=3), -1, "do not hold"),
    (dict(scale=math.nan), -1, "NaN"),
])
def test_shared_refusals(lib, bad, code, needle):
    a = dict(q=16, kc=16, vc=16, ks=None, vs=None, bt=16, ctx=16, mask=None, starts=16, lens=16,
             groups=1, B=2, k=4, Hq=8, Hkv=2, D=128, P=16, NP=8, MP=4, qdt=1, kvdt=1, scale=0.088,
             out=16)
    a.update(bad)
    rc = lib.spec_verify_attn_shared(
        vp(a["q"]), vp(a["kc"]), vp(a["vc"]), vp(a["ks"]), vp(a["vs"]), vp(a["bt"]), vp(a["ctx"]),
        vp(a["mask"]), vp(a["starts"]), vp(a["lens"]), a["groups"], a["B"], a["k"], a["Hq"],
        a["Hkv"], a["D"], a["P"], a["NP"], a["MP"], a["qdt"], a["kvdt"], a["scale"], vp(a["out"]),
        None, None)
    _err(lib, rc, code, needle)


@pytest.mark.parametrize("call", ["compact", "fork", "release", "logprob", "shared"])
def test_empty_calls(lib, call):
    """No sequences, pairs or rows: nothing is looked at."""
    n = None
    rc = {"compact": lambda: lib.spec_kv_compact(n, n, n, n, 1, n, n, n, n, 0, 4, 2, 128, 16, 8, 4, n),
          "fork": lambda: lib.spec_kv_fork(n, n, n, n, 1, n, n, n, n, n, 0, 0, 2, 2, 128, 16, 8, 4, n),
          "release": lambda: lib.spec_kv_release(n, n, n, n, n, 0, 2, 16, 8, 4, n),
          "logprob": lambda: lib.spec_token_logprobs(n, 1, n, n, 0, 3, 10, 1.0, 0, n, n, n, n, n),
          "shared": lambda: lib.spec_verify_attn_shared(n, n, n, n, n, n, n, n, n, n, 3, 0, 4, 8, 2,
                                                        128, 16, 8, 4, 1, 1, 0.1, n, n, n)}[call]()
    assert rc == 0


# ------------------------------------------------------------------ the binding's checks

def _state():
    s = rollouts.pool_state(0, "e4m3", [20, 0], 2, 64, 16)
    s["one"] = torch.zeros(1, dtype=torch.int32)
    return s


@pytest.mark.parametrize("bad", [
    dict(vc=lambda s: s["vc"].float()), dict(table=lambda s: s["table"].long()),
    dict(ctx=lambda s: s["ctx"][:1]), dict(refs=lambda s: s["refs"][1:]),
    dict(refs=lambda s: s["refs"].long()), dict(ks=lambda s: s["ks"].half()),
    dict(kid=lambda s: s["one"].long()), dict(kid=lambda s: torch.zeros(2, dtype=torch.int32)),
    dict()])
def test_binding_fork(bad):
    """Wrong types and shapes, and (last) tensors off the GPU."""
    from speculative_decoding_verification_attn_gb300 import binding
    s = _state()
    s["kid"] = s["one"]
    for n, f in bad.items():
        s[n] = f(s)
    with pytest.raises((ValueError, RuntimeError)):
        binding.spec_kv_fork(s["kc"], s["vc"], s["table"], s["ctx"], s["refs"], s["one"], s["kid"],
                             0, s["ks"], s["vs"])


@pytest.mark.parametrize("bad", [
    dict(path=torch.zeros(1, 4, dtype=torch.int32)), dict(path=torch.zeros(2, 4)),
    dict(n=torch.zeros(3, dtype=torch.int32)), dict(n=torch.zeros(2)), dict()])
def test_binding_compact(bad):
    from speculative_decoding_verification_attn_gb300 import binding
    s = _state()
    a = dict(path=torch.zeros(2, 4, dtype=torch.int32), n=torch.zeros(2, dtype=torch.int32))
    a.update(bad)
    with pytest.raises((ValueError, RuntimeError)):
        binding.spec_kv_compact(s["kc"], s["vc"], s["table"], s["ctx"], a["path"], a["n"], s["ks"],
                                s["vs"])


@pytest.mark.parametrize("bad", [
    dict(tok=torch.zeros(2, 3)), dict(tok=torch.zeros(3, dtype=torch.int32)),
    dict(lp=torch.zeros(2, 4)), dict(ent=torch.zeros(2, 3).double()),
    dict(ids=torch.zeros(2, 3, 5)), dict(top=torch.zeros(2, 3)),
    dict(ids=torch.zeros(2, 3, 5, dtype=torch.int32), top=torch.zeros(2, 3, 4)),
    dict(lens=torch.zeros(3, dtype=torch.int32)), dict()])
def test_binding_logprobs(bad):
    from speculative_decoding_verification_attn_gb300 import binding
    a = dict(tok=torch.zeros(2, 3, dtype=torch.int32), lp=torch.zeros(2, 3), ent=None, ids=None,
             top=None, lens=None)
    a.update(bad)
    with pytest.raises((ValueError, RuntimeError)):
        binding.spec_token_logprobs(torch.zeros(2, 3, 10), a["tok"], a["lp"], a["ent"], a["ids"],
                                    a["top"], a["lens"])


# ------------------------------------------------------------------ the plain forms themselves

def test_plain_fork_keeps_count():
    """Every page's count is the number of rows that list it, whatever is forked
    and released."""
    s = rollouts.pool_state(2, "bf16", [70, 0, 0, 33, 0, 0], 1, 32, 16, MP=8, spare=30)

    def check():
        want = torch.zeros_like(s["refs"])
        for e in s["table"].reshape(-1).tolist():
            if e >= 0:
                want[e] += 1
        assert torch.equal(want, s["refs"])

    check()
    assert rollouts.fork(s, [0, 0, 3, 0], [1, 2, 4, 0], 20) == 0
    check()
    assert rollouts.fork(s, [1, 2], [1, 2], 40) == 0
    check()
    rollouts.release(s, [0, 1, 4], [40, 0, 16])
    check()
    assert rollouts.fork(s, [0, 2], [0, 5], 10) == 0
    check()
    rollouts.release(s, list(range(6)))
    assert int(s["refs"].sum()) == 0


def test_plain_compact_keeps_rows():
    """The kept nodes' rows, read through the table, are the path's rows."""
    s = rollouts.pool_state(3, "f32", [13, 30], 2, 32, 8, hold_more=12)
    before = [paged8.dense64(s["kc"], None, s["table"], b, int(s["ctx"][b]) + 12)
              for b in range(2)]
    path = torch.tensor([[0, 3, 7, 11] + [-1] * 8, [2, 5] + [-1] * 10], dtype=torch.int32)
    n = torch.tensor([4, 2], dtype=torch.int32)
    assert rollouts.compact(s, path, n) == 0
    for b in range(2):
        c, m = int(s["ctx"][b]), int(n[b])
        after = paged8.dense64(s["kc"], None, s["table"], b, c + m)
        want = torch.cat([before[b][:c], before[b][c + path[b, :m].long()]])
        assert torch.equal(after, want)
