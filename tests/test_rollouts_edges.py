"""Index arithmetic of the paged calls of several continuations at the ends of its types,
compiled for the host, and their refusals.  Runs without a GPU."""
from __future__ import annotations

import ctypes
import subprocess

import pytest
import torch

PLACES = r"""
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include "places.h"
int main(int argc, char** argv) {
    auto n = [&](int i) { return (int32_t)strtoll(argv[i], 0, 10); };
    if (!strcmp(argv[1], "in_table")) printf("%d", (int)specv::in_table(n(2), n(3), n(4)));
    if (!strcmp(argv[1], "row_pieces")) printf("%d", specv::row_pieces(n(2), n(3), n(4)));
    if (!strcmp(argv[1], "entries_kept")) printf("%d", specv::entries_kept(n(2), n(3), n(4)));
}
"""


@pytest.fixture(scope="module")
def places(tmp_path_factory):
    from speculative_decoding_verification_attn_gb300 import build
    d = tmp_path_factory.mktemp("places")
    (d / "main.cpp").write_text(PLACES)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-fsanitize=signed-integer-overflow",
                    "-fno-sanitize-recover", "-I" + build.CSRC, "-o", str(d / "main"),
                    str(d / "main.cpp")], check=True)

    def run(*args):
        out = subprocess.run([str(d / "main"), *map(str, args)], check=True, capture_output=True)
        return int(out.stdout)
    return run


BIG = 2 ** 31 - 1


@pytest.mark.parametrize("first,g,width", [
    (0, 0, 1), (0, 1, 1), (3, 4, 8), (3, 4, 7), (BIG, 0, BIG), (BIG - 5, 63, 4), (BIG, 64, BIG),
    (BIG - 1, 0, BIG), (BIG - 63, 62, BIG)])
def test_entries_of_a_table(places, first, g, width):
    """Contexts at the end of 31 bits over pages of one token: no entry is taken for one
    of the table that is not."""
    assert places("in_table", first, g, width) == (first + g < width)


@pytest.mark.parametrize("keep,P,width", [
    (0, 16, 4), (1, 16, 4), (16, 16, 4), (17, 16, 4), (64, 16, 4), (65, 16, 4), (BIG, 1, 4),
    (BIG, 16, 4), (BIG - 254, 1, 100), (BIG, 1, BIG), (BIG, BIG, 4), (5, BIG, 4)])
def test_entries_that_a_release_keeps(places, keep, P, width):
    """Every token kept, as the largest number: no entry behind the table is counted, so a
    thread's place behind the first one stays within its type."""
    assert places("entries_kept", keep, P, width) == min(-(-keep // P), width)


@pytest.mark.parametrize("rows,dim,elem", [
    (0, 32, 4), (3, 32, 1), (15, 128, 2), (2 ** 22 + 15, 128, 4), (2 ** 23 - 1, 128, 4),
    (2 ** 25 - 1, 32, 4), (2 ** 22 - 1, 256, 4), (2 ** 25 - 1, 32, 1)])
def test_pieces_of_a_copied_page(places, rows, dim, elem):
    """Pages of up to 2^30 elements, 2^32 bytes."""
    assert rows * dim < 2 ** 30
    assert places("row_pieces", rows, dim, elem) == rows * dim * elem // 16


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_verification_attn_gb300 import binding, build
    build.build()
    return binding.load()


@pytest.mark.parametrize("call", ["fork", "release"])
@pytest.mark.parametrize("n,width,needle", [(1, 2 ** 30 + 1, "max_pages"), (1, BIG, "max_pages"),
                                            (1 << 24, 4, "2^24"), (BIG, 4, "2^24")])
def test_widest_tables_and_most_rows(lib, call, n, width, needle):
    """What a block's 32-bit walk over a row, and every row's look at all others, would not end
    for is refused; nothing was launched."""
    p = ctypes.c_void_p(16)
    if call == "fork":
        rc = lib.spec_kv_fork(p, p, None, None, 1, p, p, p, p, p, n, 4, 2, 2, 128, 16, 8, width, None)
    else:
        rc = lib.spec_kv_release(p, p, p, p, None, n, 2, 16, 8, width, None)
    assert rc == -2
    assert needle in lib.spec_last_error().decode()


@pytest.mark.parametrize("page_size,seen", [(16, 16), (2 ** 32 + 16, BIG), (-(2 ** 32) + 16, -1), (2 ** 31, BIG)])
def test_binding_release_page_size(monkeypatch, page_size, seen):
    """A page size past 32 bits keeps its sign and its size: none of its bits are dropped."""
    from speculative_decoding_verification_attn_gb300 import binding
    got = []

    class Library:
        def spec_kv_release(self, *args):
            got.append(args)
            return 0

    monkeypatch.setattr(binding, "load", lambda: Library())
    monkeypatch.setattr(binding, "_device_of", lambda t: -1)
    monkeypatch.setattr(binding, "_stream_on", lambda stream, dev: 0)
    row = torch.zeros(2, dtype=torch.int32)
    binding.spec_kv_release(torch.zeros(2, 3, dtype=torch.int32), row, row, row, page_size)
    assert got[0][7] == seen
