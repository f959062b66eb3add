"""Units of paged_tree_attention that are cut and joined, by the joins of 32
columns that batches of middle size take: one for each place between two groups
of CTAs and, in the last case, one for each sequence."""
import pytest

torch = pytest.importorskip("torch")

import entropy_bounded_softmax_gb300 as cs
from paged_parity import cache, definition, tree_mask

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("B,T,H,Hk,D,longest", [
    (32, 16, 32, 8, 128, 1500), (32, 16, 32, 8, 72, 1500),
    (24, 9, 56, 8, 64, 1300), (20, 3, 64, 4, 200, 900)])
def test_joins_of_middle_batches(B, T, H, Hk, D, longest, dtype):
    gen = torch.Generator().manual_seed(B)
    lengths = torch.randint(T, longest, (B,), generator=gen).tolist()
    q, k, v, table, n = cache(lengths, T, H, Hk, D, 16, dtype, seed=B)
    table = torch.nn.functional.pad(table, (0, 64))   # rows for 1024 more
    mask = tree_mask(B, T, seed=B)
    dev = [x.cuda() for x in (q, k, v, table, n)]
    for m in (None, mask):
        out, lse = cs.paged_tree_attention(
            *dev, mask=None if m is None else m.cuda(), return_lse=True)
        assert cs.get_error() == set()
        ref, tol, wlse, tlse = definition(q, k, v, table, n, m)
        over = (out.cpu().double() - ref).abs() - tol
        assert (over <= 0).all(), float(over.max())
        assert ((lse.cpu().double() - wlse).abs() <= tlse).all()
