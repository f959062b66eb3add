"""A pool that runs out of pages in the middle of a sequence's new tokens: those
that have slots are attended as if there were no others."""
import math

import pytest

torch = pytest.importorskip("torch")

import entropy_bounded_softmax_gb300 as cs
from paged_parity import definition, extend, tree_mask

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("free", range(6))
def test_pool_runs_dry_in_a_sequence(free, masked):
    B, T, H, Hk, D, page = 4, 40, 8, 2, 64, 16
    gen = torch.Generator().manual_seed(free)
    lengths, new = [20, 5, 0, 31], [40, 17, 40, 3]
    order = torch.randperm(12, generator=gen).int()
    held = [2, 1, 0, 2]
    table = torch.full((B, 5), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = order[at:at + n]
        at += n
    pages = [torch.randn(12, page, Hk, D, generator=gen).bfloat16()
             for _ in range(2)]
    q, k, v = (torch.randn(B, T, h, D, generator=gen).bfloat16()
               for h in (H, Hk, Hk))
    some = order[at:at + free]
    mask = tree_mask(B, T, seed=free) if masked else None
    want = extend(table.tolist(), lengths, new, some.tolist(), page, T)

    dev = [x.cuda() for x in pages]
    count = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    on = table.cuda()
    slots, totals, have, _ = cs.paged_extend(
        on, count, torch.tensor(new, dtype=torch.int32, device="cuda"),
        some.cuda(), page, T)
    assert cs.get_error() == {"OUT_OF_PAGES"}
    assert slots.tolist() == want[1] and totals.tolist() == want[2]
    cs.paged_write(k.cuda(), v.cuda(), slots, *dev)
    there = totals - count
    out, lse = cs.paged_tree_attention(
        q.cuda(), *dev, on, totals, new_lengths=there,
        mask=None if mask is None else mask.cuda(), return_lse=True)
    assert cs.get_error() == set()
    for x, into in ((k, pages[0]), (v, pages[1])):
        for b in range(B):
            for i in range(int(there[b])):
                into.view(-1, Hk, D)[want[1][b][i]] = x[b, i]
    assert all(torch.equal(x.cpu(), y) for x, y in zip(dev, pages))
    ref, tol, wlse, tlse = definition(q, *pages, torch.tensor(want[0]),
                                      totals.cpu(), mask, there.cpu())
    assert ((out.cpu().double() - ref).abs() <= tol).all()
    empty = wlse == -math.inf
    assert torch.equal(lse.cpu() == -math.inf, empty)
    assert ((lse.cpu().double() - wlse).abs() <= tlse)[~empty].all()
