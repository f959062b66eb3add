"""The whole-number arithmetic by which the operators around a paged cache find
where they read and write, on the CPU, at the ends of what they accept."""
import ctypes
import itertools
import os
import shutil
import subprocess

import pytest

import entropy_bounded_softmax_gb300 as cs
from conftest import ROOT

CSRC = os.path.join(ROOT, "entropy_bounded_softmax_gb300", "csrc")
MOST = 1 << 30       # tokens of a table's row, and new tokens of a sequence

SHIM = """
#include "cs_pages.h"
extern "C" void claim(const int32_t* in, int32_t* out) {
    const cs::Claim c = cs::claim_of(in[0], in[1], in[2] != 0, in[3], in[4], in[5], in[6]);
    out[0] = c.len; out[1] = c.fresh; out[2] = c.held; out[3] = c.need; out[4] = c.bad;
}
extern "C" void start(const int32_t* in, int32_t* out) {
    const cs::TreeStart x = cs::tree_start_of(in, in[4], in[5], in[6], in[7]);
    out[0] = x.b; out[1] = x.base; out[2] = x.n.len; out[3] = x.n.fresh;
}
"""


@pytest.fixture(scope="module")
def library(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    folder = tmp_path_factory.mktemp("pages")
    source, library = folder / "shim.cpp", folder / "shim.so"
    source.write_text(SHIM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared",
                    "-fPIC", "-I", CSRC, str(source), "-o", str(library)],
                   check=True)
    return ctypes.CDLL(str(library))


def call(function, given, results):
    out = (ctypes.c_int32 * results)()
    function((ctypes.c_int32 * len(given))(*given), out)
    return list(out)


@pytest.mark.parametrize("page,max_pages", [
    (1, MOST), (1, MOST - 1), (2, MOST // 2), (16, MOST // 16), (3, 1000),
    (MOST, 1), (1 << 20, 1024), (7, 0), (2 ** 31 - 1, 0)])
def test_claims(library, page, max_pages):
    """The pages that a sequence is short of: never past its row."""
    ends = [-2 ** 31, -1, 0, 1, 2, 15, 16, 17, MOST - 1, MOST, MOST + 1,
            2 ** 31 - 1]
    pages = sorted({-2 ** 31, -1, 0, 1, max_pages - 1, max_pages,
                    max_pages + 1, 2 ** 31 - 1})
    for n, w, held, max_new in itertools.product(
            ends, ends, [None, *pages], (0, 16, MOST)):
        got = call(library.claim, (n, w, held is not None, held or 0, max_new,
                                   max_pages, page), 5)
        have = held if held is not None else -(-max(n, 0) // page)
        out = (n < 0 or w < 0 or w > max_new or not 0 <= have <= max_pages
               or have * page < n)
        want = 0 if out else -(-(n + w) // page)
        need = 0 if out else max(0, min(want, max_pages) - have)
        assert got == [n, 0 if out else w, have, need,
                       int(out or want > max_pages)], (n, w, held, max_new)
        assert out or 0 <= have + need <= max_pages


@pytest.mark.parametrize("batch,most,T", [(33, 1280, 5), (65535, MOST, 1 << 20),
                                          (513, 0, 4), (1, 16, 64)])
def test_where_a_share_begins(library, batch, most, T):
    """What paged_tree_attention's walk over the lengths left, which may be any
    numbers where they were changed under it, in range; as it is where it is."""
    ends = [-2 ** 31, -1, 0, 1, 2 ** 31 - 1]
    for b, base, n, w, g0 in itertools.product(
            [*ends, batch - 1, batch], [*ends, 1000], [*ends, most - 1, most],
            [*ends, T, T + 1], (0, 1, 1000, MOST)):
        got = call(library.start, (b, base, n, w, g0, batch, most, T), 4)
        assert 0 <= got[0] < batch and 0 <= got[1] <= g0
        assert 0 <= got[2] <= most and 0 <= got[3] <= min(T, got[2])
        if (0 <= b < batch and 0 <= base <= g0 and 0 <= n <= most
                and 0 <= w <= min(T, n)):
            assert got == [b, base, n, w]


@pytest.mark.parametrize("D", [64, 128, 136])
@pytest.mark.parametrize("T,H,Hk", [(1, 1, 1), (5, 8, 2), (32, 32, 8),
                                    (33, 32, 8), (65, 32, 8), (100, 6, 3)])
def test_what_needs_no_workspace(D, T, H, Hk):
    """The header's rule: units of the batch against the tokens of a row."""
    rows = T * (H // Hk)
    size = 256 if rows > 128 and D <= 128 else 128
    strides = (ctypes.c_int64 * 3)(T * H * D, H * D, D)
    full = 512 if D <= 128 else 256
    for B, most in itertools.product(
            (1, 2, 3, 13, 18, 19, 37, 38, 56, 57, 76, 77, 113, 114, 152, 153,
             300),
            (1, full // 16, full // 16 + 1, full // 8, full // 8 + 1, 1000)):
        units = B * Hk * -(-rows // size)
        shape = cs.cs_tree_shape(B, T, H, Hk, D, 16, 100, most, 0, 0.125,
                                 strides, strides, strides, strides, most,
                                 (0, T))
        whole = units <= 152 and 16 * most <= (2 * full if units >= 114
                                               else full)
        assert (cs.cs_paged_tree_attention_workspace(shape) == 0) == whole, \
            (B, most)
