"""The operators around a paged cache at the ends of what they accept."""
import math

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


@pytest.mark.parametrize("scale", [2.0 ** -119, 2.0 ** -104, 2.0 ** -95,
                                   2.0 ** -40, 1.0, 1.9, 4.0])
@pytest.mark.parametrize("case", [
    ([5], 3, 4, 4, 8, 16, 0), ([300, 9], 3, 4, 2, 8, 16, 0),
    ([2000, 40], 3, 4, 2, 72, 16, 64), ([2000], 40, 16, 4, 8, 5, 64),
    ([900], 3, 2, 1, 136, 16, 64)], ids=str)
@pytest.mark.parametrize("sign", [1, -1])
def test_tree_large_scores(case, scale, sign):
    """One score of 1.875 * 2^126 * scale, the row's others 0, or one of 0, the
    others that far below it: it takes the row; lse stays in fp32.  Other rows
    are as ever."""
    *sizes, more = case
    q, k, v, table, lengths = cache(*sizes, seed=6)
    table = torch.nn.functional.pad(table, (0, more))
    T, H, Hk = sizes[1:4]
    j, i = int(lengths[0]) // 2, T - 1
    q[:], k[:] = 0, 0
    q[0, i, 1, 0] = 1.5 * 2.0 ** 63
    at = int(table[0, j // k.shape[1]]), j % k.shape[1], Hk // H   # of head 1
    if sign < 0:
        k[..., 0] = -1.25 * 2.0 ** 63
        k[at][0] = 0
    else:
        k[at][0] = 1.25 * 2.0 ** 63
    out, lse = (x.cpu() for x in cs.paged_tree_attention(
        *(x.cuda() for x in (q, k, v, table, lengths)), scale=scale,
        return_lse=True))
    hit = torch.zeros(lse.shape, dtype=torch.bool)
    hit[0, i, 1] = True
    assert cs.get_error() == set()
    # One weight, which its sum takes away again, to fp32 (the others, 240 or
    # more below the maximum, are less than 2^-126).
    assert torch.equal(out[0, i, 1], v[at])
    score = min(1.875 * 2.0 ** 126 * scale, 2.0 ** 128 * math.log(2))
    score = score if sign > 0 else 0.0
    assert abs(float(lse[0, i, 1]) - score) <= 2.0 ** -21 * max(1, score)
    ref, tol, wlse, tlse = definition(q * 0, k * 0, v, table, lengths)
    assert ((out.double() - ref).abs() <= tol)[~hit].all()
    assert ((lse.double() - wlse).abs() <= tlse)[~hit].all()


@pytest.mark.parametrize("T,D,page", [(3, 64, 16), (40, 128, 5), (2, 200, 16)])
def test_tree_all_scores_far_below_zero(T, D, page):
    """Rows whose scores are all about -2^40, one of them the largest: the same
    as without what all have in common."""
    q, k, v, table, lengths = cache([1500, 90], T, 8, 2, D, page, seed=7)
    table = torch.nn.functional.pad(table, (0, 64))
    q[:], k[:] = 0, 0
    q[..., 0], k[..., 0] = 2.0 ** 20, -2.0 ** 20
    for b, n in enumerate(lengths.tolist()):
        for j in (0, n // 2):
            at = int(table[b, j // page]), j % page
            k[at][..., 0] = -2.0 ** 20 + 2.0 ** 12
    out, lse = cs.paged_tree_attention(
        *(x.cuda() for x in (q, k, v, table, lengths)), scale=1.0,
        return_lse=True)
    assert cs.get_error() == set()
    for b, n in enumerate(lengths.tolist()):
        rows = [v[int(table[b, j // page]), j % page] for j in (0, n // 2)]
        want = (rows[0].double() + rows[1].double()) / 2
        want = want.repeat_interleave(4, 0)
        # (Half a step of the result, and as much for fp32's.)
        assert ((out[b].cpu().double() - want).abs()
                <= 2.0 ** -8 * want.abs() + 2.0 ** -16).all()
    score = -2.0 ** 40 + 2.0 ** 32
    assert ((lse.cpu().double() - score).abs() <= 2.0 ** -21 * 2.0 ** 40).all()


@pytest.mark.parametrize("wide", [0, 64])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 5), (256, 64)])
def test_tree_infinite_scores(D, page, wide):
    """A score of +infinity makes its row NaN and is reported; a token with one
    of -infinity counts as removed, also where a row has no other."""
    T, j = 6, 700 - 6 + 4
    args = cache([700, 6], T, 4, 2, D, page, seed=8)
    q, k, v, table, lengths = args
    table = torch.nn.functional.pad(table, (0, wide))
    mask = tree_mask(2, T, seed=3)
    mask[0, :, 4] = False
    mask[0, 4, 4] = True                      # new token 4: row 4 alone
    mask[1] = torch.eye(T, dtype=torch.bool)  # each itself alone
    q[..., 5] = q[..., 5].abs() + 0.5
    for b, at in ((0, j), (1, 4)):
        k[int(table[b, at // page]), at % page, 1, 5] = math.inf
    hit = torch.zeros(2, T, 4, dtype=torch.bool)
    hit[:, 4, 2:] = True
    for sign in (1, -1):
        out, lse = cs.paged_tree_attention(
            *(x.cuda() for x in (sign * q, k, v, table, lengths)),
            mask=mask.cuda(), return_lse=True)
        out, lse = out.cpu(), lse.cpu()
        assert cs.get_error() == ({"NAN_INPUT"} if sign > 0 else set())
        # What the rows would be without the token, which in `k` is out of
        # reach of a product with 0.
        kk = k.clone()
        kk[kk.isinf()] = 0
        gone = mask.clone()
        gone[:, 4, 4] = False
        a = definition(sign * q, kk, v, table, lengths, mask)
        z = definition(sign * q, kk, v, table, lengths, gone)
        ref, tol, wlse, tlse = (torch.where(
            hit if x.dim() == 3 else hit[..., None], y, x)
            for x, y in zip(a, z))
        sound = ~hit if sign > 0 else torch.ones_like(hit)
        assert ((out.double() - ref).abs() <= tol)[sound].all()
        empty = wlse == -math.inf
        assert empty[1, 4, 2:].all() and empty.sum() == 2
        assert torch.equal(lse[sound] == -math.inf, empty[sound])
        some = sound & ~empty
        assert ((lse.double() - wlse).abs() <= tlse)[some].all()
        if sign > 0:
            assert out[hit].isnan().all() and lse[hit].isnan().all()
        else:
            assert (out[1, 4, 2:] == 0).all()
