"""The operators around a paged cache at the ends of what they accept."""
import pytest

torch = pytest.importorskip("torch")

import entropy_bounded_softmax_gb300 as cs

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("n,new,given", [
    ((1 << 30), 1 << 30, True), ((1 << 30), 1 << 30, False),
    ((1 << 30) - 3, 1 << 30, False), (0, 1 << 30, False)])
def test_extend_past_the_largest_row(n, new, given):
    """Up to 2^31 tokens after a call, in pages of one: what the row holds is
    taken, nothing is written behind it, and it is reported."""
    most, page = 1 << 30, 1
    room = torch.full((most + 1024,), 5, dtype=torch.int32, device="cuda")
    table = room[:most].view(1, most)
    free = torch.arange(64, dtype=torch.int32, device="cuda")
    slots, totals, have, cursor = cs.paged_extend(
        table, i32([n]), i32([new]), free, page, most,
        held=i32([n]) if given else None)
    short = min(most - n, 64)
    # (From 0 the row holds all, of which the list has 64.)
    assert cs.get_error() == {"BAD_PAGE" if n else "OUT_OF_PAGES"}
    assert totals.tolist() == [n + short] and have.tolist() == [n + short]
    assert cursor.tolist() == [short]
    assert slots[0, :short].tolist() == list(range(short))
    assert bool((slots[0, short:] == -1).all())
    assert room[n:n + short].tolist() == list(range(short))
    room[n:n + short] = 5
    assert bool((room == 5).all())
