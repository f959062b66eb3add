"""paged_tree_attention against its definition in 64 bits: trees, chunks, rows
that attend nothing, lengths around blocks and pages, shared key heads, page
sizes that end inside a block, both element types, bad entries, strides,
streams and graphs."""
import math

import pytest

torch = pytest.importorskip("torch")

import entropy_bounded_softmax_gb300 as cs
from paged_parity import cache, definition, tree_mask

pytestmark = pytest.mark.gpu


def run(args, mask=None, new=None, **kw):
    dev = [x.cuda() for x in args]
    return cs.paged_tree_attention(
        *dev, mask=None if mask is None else mask.cuda(),
        new_lengths=None if new is None else new.cuda(), **kw)


def compare(got, want):
    out, lse = (x.cpu() for x in got)
    ref, tol, wlse, tlse = want
    over = (out.double() - ref).abs() - tol
    assert (over <= 0).all(), float(over.max())
    empty = wlse == -math.inf
    assert torch.equal(lse == -math.inf, empty)
    assert ((lse.double() - wlse).abs()[~empty] <= tlse[~empty]).all()


def check(args, mask=None, new=None, scale=None, errors=frozenset()):
    got = run(args, mask, new, scale=scale, return_lse=True)
    assert got[0].dtype == args[0].dtype and got[0].shape == args[0].shape
    assert cs.get_error() == errors
    compare(got, definition(*args, mask, new, scale))
    return got


CASES = [
    # lengths, T, H, Hk, D, page
    ([1], 1, 1, 1, 8, 1),
    ([5, 3, 17], 3, 2, 1, 64, 16),
    ([77], 8, 8, 8, 64, 16),
    ([127, 128, 129], 5, 4, 2, 128, 16),          # around a block of 128
    ([63, 64, 65], 7, 2, 1, 256, 16),             # around a block of 64
    ([255, 9, 257], 9, 8, 1, 64, 5),              # pages end inside blocks
    ([300, 77], 13, 12, 4, 80, 48),
    ([1000, 33, 511], 33, 16, 2, 128, 1),         # 264 rows: a pair and more
    ([700], 64, 5, 1, 256, 64),                   # 320 rows of 256
    ([200, 90], 16, 40, 2, 96, 32),
    ([400, 130], 130, 4, 1, 16, 256),             # the draft longer than a block
    ([5000, 17], 4, 8, 2, 120, 100),
    ([333, 64], 11, 3, 3, 200, 7),
    ([2100, 300, 1500, 31], 31, 8, 2, 64, 16),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("case", CASES, ids=str)
def test_against_definition(case, dtype):
    args = cache(*case, dtype=dtype)
    B, T = args[0].shape[:2]
    check(args)
    check(args, tree_mask(B, T))


@pytest.mark.parametrize("case", CASES, ids=str)
def test_masks_that_leave_rows_empty(case):
    """Rows that attend none of the new tokens; where there is nothing before
    them they are zeros."""
    args = cache(*case, seed=1)
    B, T = args[0].shape[:2]
    check(args, tree_mask(B, T, empty=True))
    check(args, torch.zeros(B, T, T, dtype=torch.bool))
    check(args, torch.ones(T, T, dtype=torch.bool))
