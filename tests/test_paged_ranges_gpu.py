"""The operators around a paged cache at the ends of what they accept."""
import pytest

torch = pytest.importorskip("torch")

import entropy_bounded_softmax_gb300 as cs
from paged_parity import cache, definition, tree_mask

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


# lengths, T, H, Hk, D, page, entries of the table beside those needed: one
# token; whole sequences; ones that are cut and joined; pairs of tiles; heads
# above 128.
SPREAD = [([1], 1, 4, 4, 64, 16, 0), ([300, 40], 5, 8, 2, 64, 16, 0),
          ([2000, 40, 700], 5, 8, 2, 128, 5, 64),
          ([1800, 900], 40, 16, 2, 128, 64, 64), ([1500], 7, 4, 1, 256, 16, 64)]


def within(got, want):
    out, lse = (x.cpu().double() for x in got)
    ref, tol, wlse, tlse = want
    assert out.isfinite().all()
    over = (out - ref).abs() - tol
    assert (over <= 0).all(), float(over.max())
    assert ((lse - wlse).abs() <= tlse).all()


def spread(case, kind):
    """A cache whose scores are all about the same (flat), or such that one
    late token has nearly all the weight (peak)."""
    *sizes, more = case
    q, k, v, table, lengths = cache(*sizes, seed=5)
    table = torch.nn.functional.pad(table, (0, more))
    scale = 0.01
    if kind == "peak":
        q, k, scale = torch.ones_like(q), k / 16, 40.0 / q.shape[-1]
        for b, n in enumerate(lengths.tolist()):
            j = n - n // 4 - q.shape[1]
            if j >= 0:
                k[int(table[b, j // k.shape[1]]), j % k.shape[1]] = 1.0
    return q, k, v, table, lengths, scale


@pytest.mark.parametrize("kind", ["flat", "peak"])
@pytest.mark.parametrize("case", SPREAD, ids=str)
def test_tree_values_as_large_as_bf16_has(case, kind):
    """The average of finite values is finite: all of one sign, up to the
    largest of the type."""
    q, k, v, table, lengths, scale = spread(case, kind)
    top = torch.finfo(torch.bfloat16).max
    v = ((0.5 + 0.5 * v.float().abs().clamp(max=1)) * top).bfloat16()
    assert v[~v.isnan()].isfinite().all() and v[~v.isnan()].max() == top
    mask = tree_mask(q.shape[0], q.shape[1])
    for m in (None, mask):
        got = cs.paged_tree_attention(
            *(x.cuda() for x in (q, k, v, table, lengths)), scale=scale,
            mask=None if m is None else m.cuda(), return_lse=True)
        within(got, definition(q, k, v, table, lengths, m, scale=scale))
        assert cs.get_error() == set()


@pytest.mark.parametrize("case", SPREAD, ids=str)
def test_tree_values_as_small_as_bf16_has(case):
    """Values near the least normal one of the type.  Weights are at least
    2^-6 / n times those of e^(s - m), n <= 2048: products with values of 2^-117
    are 2^-134, and fp32 has steps of 2^-149, of which 2^-15 is within half a
    step of bf16 and its 2048 sums, all of one sign."""
    q, k, v, table, lengths, scale = spread(case, "flat")
    v = ((1 + v.float().abs().clamp(max=1)) * 2.0 ** -117).bfloat16()
    out = cs.paged_tree_attention(
        *(x.cuda() for x in (q, k, v, table, lengths)), scale=scale)
    ref = definition(q, k, v, table, lengths, scale=scale)[0]
    # The result's rounding, the weights', and as much again for the rest.
    assert ((out.cpu().double() - ref).abs() <= 4 * 2.0 ** -8 * ref.abs()).all()
    assert cs.get_error() == set()


def one_token(q, k, v, table, lengths, scale):
    """paged_attention of each sequence's last query, beside the definition of
    a tree of one token."""
    q = q[:, -1].contiguous()
    out, lse = cs.paged_attention(
        *(x.cuda() for x in (q, k, v, table, lengths)), scale=scale,
        return_lse=True)
    want = definition(q[:, None], k, v, table, lengths, scale=scale)
    return (out[:, None], lse[:, None]), want


@pytest.mark.parametrize("kind", ["flat", "peak"])
@pytest.mark.parametrize("case", SPREAD, ids=str)
def test_paged_attention_values_as_large_as_bf16_has(case, kind):
    *args, scale = spread(case, kind)
    top = torch.finfo(torch.bfloat16).max
    args[2] = ((0.5 + 0.5 * args[2].float().abs().clamp(max=1))
               * top).bfloat16()
    within(*one_token(*args, scale))
    assert cs.get_error() == set()


@pytest.mark.parametrize("case", SPREAD, ids=str)
def test_paged_attention_values_as_small_as_bf16_has(case):
    """As for trees, n the 2^13 tokens of a table's row at most: an fp32 step is
    2^-13 of the smallest products."""
    *args, scale = spread(case, "flat")
    args[2] = ((1 + args[2].float().abs().clamp(max=1))
               * 2.0 ** -117).bfloat16()
    (out, _), want = one_token(*args, scale)
    assert ((out.cpu().double() - want[0]).abs()
            <= 4 * 2.0 ** -8 * want[0].abs()).all()
    assert cs.get_error() == set()
