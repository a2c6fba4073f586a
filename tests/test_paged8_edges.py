"""Refusals and host logic at the edges of the paged calls.  Runs without a GPU:
every argument check precedes the first CUDA call."""
from __future__ import annotations

import ctypes
import subprocess

import pytest


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
