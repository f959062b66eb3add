"""paged_extend against a loop that hands pages out one by one, and paged_write
against indexing: every result is exact."""
import random

import pytest

torch = pytest.importorskip("torch")

import entropy_bounded_softmax_gb300 as cs
from paged_parity import extend

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


def state(B, T, longest, page, seed=0, short=False, spare=0):
    """Sequences with some tokens and pages, and a free list; `spare`: pages
    held past the tokens'."""
    r = random.Random(seed)
    lengths = [r.randint(0, longest) for _ in range(B)]
    new = [r.randint(0, T) for _ in range(B)]
    held = [-(-n // page) + (r.randint(0, spare) if spare else 0)
            for n in lengths]
    width = max([-(-(longest + T) // page), *held]) + 2
    need = sum(max(0, -(-(n + w) // page) - h)
               for n, w, h in zip(lengths, new, held))
    cursor = r.randint(0, 5)
    have = need // 2 if short else need + r.randint(0, 3)
    pool = list(range(sum(held) + cursor + have))
    r.shuffle(pool)
    table, at = [], 0
    for h in held:
        table.append(pool[at:at + h] + [-5] * (width - h))
        at += h
    return table, lengths, new, held, pool[at:], cursor


def check_extend(s, page, T, errors=frozenset(), use_held=True):
    table, lengths, new, held, free, cursor = s
    dev = i32(table).reshape(len(lengths), -1).cuda()
    got = cs.paged_extend(
        dev, i32(lengths).cuda(), i32(new).cuda(), i32(free).cuda(), page, T,
        held=i32(held).cuda() if use_held else None,
        cursor=i32([cursor]).cuda())
    assert cs.get_error() == errors
    want = extend(table, lengths, new, free, page, T,
                  held if use_held else None, cursor)
    assert dev.tolist() == want[0]
    assert got[0].dtype == torch.int64 and got[0].shape == (len(lengths), T)
    for x, y in zip(got, (*want[1:4], [want[4]])):
        assert x.tolist() == y
    return got


@pytest.mark.parametrize("short", [False, True])
@pytest.mark.parametrize("B,T,longest,page", [
    (1, 1, 0, 1), (1, 1, 15, 16), (5, 3, 40, 16), (32, 1, 400, 16),
    (33, 61, 300, 64), (300, 7, 50, 5), (3, 2048, 30, 16), (2, 5000, 900, 48),
    (257, 9, 20, 1), (1000, 2, 64, 128), (4, 2049, 10, 4096), (6, 0, 30, 16),
])
def test_extend(B, T, longest, page, short):
    for seed in range(3):
        s = state(B, T, longest, page, seed, short, spare=2 * (seed == 2))
        need = sum(max(0, -(-(n + w) // page) - h)
                   for n, w, h in zip(*s[1:4]))
        lacks = need > len(s[4]) - s[5]
        check_extend(s, page, T, {"OUT_OF_PAGES"} if lacks else set(),
                     use_held=seed == 2)


def cache(pages, page, Hk, D, dtype, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(pages, page, Hk, D, device="cuda",
                        generator=gen).to(dtype) for _ in range(2)]


def inputs(B, T, Hk, D, pages, page, dtype, seed=0, gone=0.3):
    gen = torch.Generator().manual_seed(seed)
    k, v = (torch.randn(B, T, Hk, D, generator=gen).to(dtype).cuda()
            for _ in range(2))
    slots = torch.randperm(pages * page, generator=gen)[:B * T].view(B, T)
    slots = slots.masked_fill(torch.rand(B, T, generator=gen) < gone, -1)
    return k, v, slots.cuda()


def written(into, x, slots):
    """What indexing makes of a copy of `into`."""
    out = into.clone()
    flat = out.reshape(-1, *into.shape[2:])
    kept = (slots >= 0) & (slots < flat.shape[0])
    flat[slots[kept]] = x[kept]
    return flat.view(into.shape)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("B,T,Hk,D,pages,page", [
    (1, 1, 1, 8, 1, 1), (1, 8, 8, 64, 9, 16), (3, 5, 2, 128, 40, 1),
    (7, 33, 12, 80, 20, 48), (2, 700, 1, 256, 30, 64), (65, 1, 3, 24, 70, 2),
    (4, 129, 8, 128, 600, 5),
])
def test_write(B, T, Hk, D, pages, page, dtype):
    kp, vp = cache(pages, page, Hk, D, dtype)
    k, v, slots = inputs(B, T, Hk, D, pages, page, dtype)
    want = written(kp, k, slots), written(vp, v, slots)
    assert cs.paged_write(k, v, slots, kp, vp) is None
    assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])
    assert cs.get_error() == set()


def test_extend_reports_what_is_out_of_range():
    """Sequences with bad lengths get nothing, the others what they would get
    without them."""
    table = [[3, 4, 0, 0], [5, 0, 0, 0], [6, 7, 0, 0], [8, 0, 0, 0]]
    lengths, new, held = [5, 2, 8, 1], [4, 3, 2, 6], [2, 1, 2, 1]
    free, page = [9, 10, 11, 12, 13, 14], 4
    for change in (dict(lengths=-1), dict(new=-1), dict(new=7),
                   dict(held=-1), dict(held=5), dict(lengths=9)):
        l2, n2, h2 = list(lengths), list(new), list(held)
        for name, x in (("lengths", l2), ("new", n2), ("held", h2)):
            if name in change:
                x[2] = change[name]
        dev = i32(table).cuda()
        slots, totals, have, cursor = cs.paged_extend(
            dev, i32(l2).cuda(), i32(n2).cuda(), i32(free).cuda(), page, 6,
            held=i32(h2).cuda())
        assert cs.get_error() == {"BAD_PAGE"}
        want = extend(table, lengths, [4, 3, 0, 6], free, page, 6, held, 0)
        got = dev.tolist()
        assert got[:2] + got[3:] == want[0][:2] + want[0][3:]
        assert got[2] == table[2]
        assert (slots[2] == -1).all()
        for y, x in ((slots, want[1]), (totals, want[2]), (have, want[3])):
            y = y.tolist()
            assert y[:2] + y[3:] == x[:2] + x[3:]
        assert totals[2] == l2[2] and have[2] == h2[2]
        assert cursor.tolist() == [want[4]]
    # A row of the table that is too short, a cursor past the list's ends, a
    # page number below 0 among the held ones.
    dev = i32([[3, 4]]).cuda()
    slots, totals, have, cursor = cs.paged_extend(
        dev, i32([5]).cuda(), i32([6]).cuda(), i32(free).cuda(), page, 6)
    assert cs.get_error() == {"BAD_PAGE"}
    assert slots.tolist() == [[17, 18, 19, -1, -1, -1]]
    assert (totals.tolist(), have.tolist(), cursor.tolist()) == ([8], [2], [0])
    for at, end in ((-3, 1), (99, 6)):
        dev = i32([[3, 4, 0]]).cuda()
        slots, totals, have, cursor = cs.paged_extend(
            dev, i32([8]).cuda(), i32([1]).cuda(), i32(free).cuda(), page, 1,
            cursor=i32([at]).cuda())
        assert cs.get_error() == ({"BAD_PAGE"} if at < 0 else
                                  {"BAD_PAGE", "OUT_OF_PAGES"})
        assert cursor.tolist() == [end]
        assert slots.tolist() == [[36 if at < 0 else -1]]
        assert totals.tolist() == [9 if at < 0 else 8]
    slots, *_ = cs.paged_extend(
        i32([[3, -1, 0]]).cuda(), i32([5]).cuda(), i32([4]).cuda(),
        i32(free).cuda(), page, 4)
    assert slots.tolist() == [[-1, -1, -1, 36]]
    assert cs.get_error() == {"BAD_PAGE"}


def test_extend_nothing():
    free = i32([1, 2, 3]).cuda()
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    slots, totals, have, cursor = cs.paged_extend(
        none.view(0, 4), none, none, free, 16, 5, cursor=i32([2]).cuda())
    assert slots.shape == (0, 5) and totals.shape == have.shape == (0,)
    assert cursor.tolist() == [2]
    table = i32([[7], [8]]).cuda()
    got = cs.paged_extend(table, i32([3, 0]).cuda(), i32([0, 0]).cuda(), none,
                          16, 0)
    assert [x.tolist() for x in got] == [[[], []], [3, 0], [1, 0], [0]]
    assert table.tolist() == [[7], [8]] and cs.get_error() == set()


def test_extend_leaves_the_rest_of_a_table():
    """A slice of a larger table; nothing beside the new entries changes."""
    table, lengths, new, held, free, cursor = state(40, 30, 200, 16, 5)
    big = torch.full((42, len(table[0]) + 7), -99, dtype=torch.int32,
                     device="cuda")
    inner = big[1:41, 3:3 + len(table[0])]
    inner.copy_(i32(table))
    before = big.clone()
    cs.paged_extend(inner, i32(lengths).cuda(), i32(new).cuda(),
                    i32(free).cuda(), 16, 30, cursor=i32([cursor]).cuda())
    want = extend(table, lengths, new, free, 16, 30, None, cursor)
    assert inner.tolist() == want[0]
    before[1:41, 3:3 + len(table[0])] = i32(want[0]).cuda()
    assert torch.equal(big, before) and cs.get_error() == set()


def test_extend_largest():
    """65535 sequences of one token, and lengths near the table's 2^30."""
    B = 65535
    lengths = torch.arange(B, dtype=torch.int32, device="cuda") % 50
    table = torch.zeros(B, 4, dtype=torch.int32, device="cuda")
    free = torch.arange(2 * B, dtype=torch.int32, device="cuda").flip(0)
    slots, totals, have, cursor = cs.paged_extend(
        table, lengths, torch.ones_like(lengths), free.contiguous(), 16, 1)
    need = (lengths % 16 == 0).int()
    first = torch.cumsum(need, 0) - need
    fresh = free[first.long()].long() * 16
    want = torch.where(need.bool(), fresh, (lengths % 16).long())
    assert torch.equal(slots[:, 0], want)
    assert cursor.tolist() == [int(need.sum())]
    assert torch.equal(totals, lengths + 1) and cs.get_error() == set()
    page = 1 << 20
    table = torch.arange(1024, dtype=torch.int32, device="cuda")[None].clone()
    slots, totals, have, _ = cs.paged_extend(
        table, i32([(1 << 30) - 3]).cuda(), i32([3]).cuda(), free, page, 5)
    assert slots.tolist() == [[(1 << 30) - 3, (1 << 30) - 2, (1 << 30) - 1,
                               -1, -1]]
    assert totals.tolist() == [1 << 30] and have.tolist() == [1024]
    table[0, -1] = 2 ** 31 - 1
    slots, *_ = cs.paged_extend(
        table, i32([(1 << 30) - 1]).cuda(), i32([1]).cuda(), free, page, 1)
    assert slots.tolist() == [[(2 ** 31 - 1) * page + page - 1]]
    assert cs.get_error() == set()


def test_write_strided():
    """Slices of a packed projection, keys and values side by side in one
    buffer, heads before slots; what lies beside stays."""
    for page in (16, 7):
        k, v, slots = inputs(3, 20, 2, 80, 9, page, torch.bfloat16, 1)
        kp, vp = cache(9, page, 2, 80, torch.bfloat16, 2)
        want = written(kp, k, slots), written(vp, v, slots)
        both = torch.full((9, 2, page, 2, 96), 7.0, dtype=kp.dtype,
                          device="cuda")
        both[:, 0, ..., 8:88], both[:, 1, ..., 8:88] = kp, vp
        packed = torch.randn(3, 20, 10, 80, device="cuda").bfloat16()
        packed[:, :, 6:8], packed[:, :, 8:] = k, v
        cs.paged_write(packed[:, :, 6:8], packed[:, :, 8:], slots,
                       both[:, 0, ..., 8:88], both[:, 1, ..., 8:88])
        assert torch.equal(both[:, 0, ..., 8:88], want[0])
        assert torch.equal(both[:, 1, ..., 8:88], want[1])
        both[..., 8:88] = 7.0
        assert (both == 7.0).all()
        hk, hv = (x.transpose(1, 2).contiguous().transpose(1, 2)
                  for x in (kp, vp))
        wide = torch.full((3, 31), -1, dtype=torch.int64, device="cuda")
        wide[:, 5:25] = slots
        ht = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in (k, v)]
        cs.paged_write(*ht, wide[:, 5:25], hk, hv)
        assert torch.equal(hk, want[0]) and torch.equal(hv, want[1])
        one = k[:1, :1].expand(3, 20, 2, 80)
        cs.paged_write(one, v, slots, kp, vp)
        assert torch.equal(vp, want[1])
        assert torch.equal(kp, written(kp, one, slots))
        assert cs.get_error() == set()


def test_write_slots_out_of_range():
    kp, vp = cache(4, 16, 2, 64, torch.float16)
    k, v, slots = inputs(2, 9, 2, 64, 4, 16, torch.float16, 3, gone=0)
    bad = slots.clone()
    bad[0, 1], bad[1, 2], bad[1, 3] = 64, 1 << 40, (1 << 63) - 1
    bad[0, 5] = -(1 << 63)
    want = written(kp, k, bad), written(vp, v, bad)
    cs.paged_write(k, v, bad, kp, vp)
    assert cs.get_error() == {"BAD_PAGE"}
    assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])
    cs.paged_write(k, v, torch.full_like(slots, -1), kp, vp)
    cs.paged_write(k[:, :0], v[:, :0], slots[:, :0], kp, vp)
    cs.paged_write(k[:0], v[:0], slots[:0], kp, vp)
    assert torch.equal(kp, want[0]) and cs.get_error() == set()
    cs.paged_write(k, v, slots, kp[:0], vp[:0])
    assert cs.get_error() == {"BAD_PAGE"}


def test_write_past_32_bits():
    """Pages more than 2^32 elements apart, and slots past 2^32."""
    k, v, slots = inputs(2, 30, 2, 64, 6, 16, torch.bfloat16, 4)
    kp, vp = cache(6, 16, 2, 64, torch.bfloat16)
    step = (1 << 32) // 5 + 8 & ~7
    big = torch.empty(5 * step + kp[0].numel(), dtype=kp.dtype, device="cuda")
    far = big.as_strided(kp.shape, (step, 128, 64, 1))
    far.copy_(kp)
    cs.paged_write(k, v, slots, far, vp)
    assert torch.equal(far, written(kp, k, slots))
    assert cs.get_error() == set()
    del big, far
    torch.cuda.empty_cache()


def test_write_slots_past_32_bits():
    """A cache of more than 2^32 slots: 138 GB, of which a few are written."""
    if torch.cuda.mem_get_info()[0] < 150 << 30:
        pytest.skip("not enough free memory")
    x = torch.randn(1, 3, 1, 8, device="cuda").bfloat16()
    kp, vp = (torch.empty((1 << 12) + 1, 1 << 20, 1, 8, dtype=x.dtype,
                          device="cuda") for _ in range(2))
    last = kp.shape[0] << 20
    slots = torch.tensor([[5, last - 1, last]], device="cuda")
    for pages in (kp, vp):
        pages[0, 5] = 0
        pages[-1, -1] = 0
    cs.paged_write(x, -x, slots, kp, vp)
    assert cs.get_error() == {"BAD_PAGE"}
    for pages, want in ((kp, x), (vp, -x)):
        assert torch.equal(pages[0, 5], want[0, 0])
        assert torch.equal(pages[-1, -1], want[0, 1])
    del kp, vp, pages
    torch.cuda.empty_cache()


def test_write_wide_tokens():
    """Tokens of more units than a CTA takes, and of a single one."""
    for Hk, D in ((5000, 256), (1, 8)):
        k, v, slots = inputs(2, 3, Hk, D, 3, 4, torch.bfloat16, 6)
        kp, vp = cache(3, 4, Hk, D, torch.bfloat16)
        want = written(kp, k, slots), written(vp, v, slots)
        cs.paged_write(k, v, slots, kp, vp)
        assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])
    k, v, slots = inputs(50, 999, 8, 128, 4000, 16, torch.bfloat16, 7)
    kp, vp = cache(4000, 16, 8, 128, torch.bfloat16)
    want = written(kp, k, slots), written(vp, v, slots)
    cs.paged_write(k, v, slots, kp, vp)
    assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])
    assert cs.get_error() == set()


def test_refusals():
    table = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    n = i32([3, 5]).cuda()
    free = i32([1, 2, 3]).cuda()
    good = dict(page_table=table, lengths=n, new_lengths=n, free_pages=free,
                page_size=16, max_new=5)
    for bad in (dict(page_table=table.cpu()), dict(page_table=table.long()),
                dict(page_table=table[0]), dict(page_table=table.T),
                dict(page_table=table[:1].expand(2, 4)),
                dict(lengths=n.long()), dict(lengths=n[:1]),
                dict(lengths=n.cpu()), dict(lengths=None),
                dict(new_lengths=n[:, None]), dict(new_lengths=None),
                dict(free_pages=free[None]), dict(free_pages=free.cpu()),
                dict(free_pages=i32([1, 0, 2, 0]).cuda()[::2]),
                dict(free_pages=None), dict(page_size=0), dict(max_new=-1),
                dict(page_size=1 << 40), dict(held=n.long()),
                dict(held=n[:1]), dict(cursor=n)):
        with pytest.raises(ValueError):
            cs.paged_extend(**{**good, **bad})
    for bad in (dict(lengths=table.view(-1)[:2]),
                dict(free_pages=table.view(-1)), dict(page_size=1 << 29)):
        with pytest.raises(cs.CsError):
            cs.paged_extend(**{**good, **bad})
    k, v, slots = inputs(2, 5, 2, 64, 4, 16, torch.bfloat16)
    kp, vp = cache(4, 16, 2, 64, torch.bfloat16)
    keep = kp.clone(), vp.clone()
    good = dict(keys=k, values=v, slots=slots, key_pages=kp, value_pages=vp)
    for error, bad in (
            (ValueError, dict(keys=k.cpu())), (ValueError, dict(keys=k[0])),
            (TypeError, dict(keys=k.float())), (TypeError, dict(values=v.half())),
            (ValueError, dict(values=v[:, :4])),
            (ValueError, dict(keys=k[..., :60], values=v[..., :60])),
            (ValueError, dict(keys=k[:, :, :1], values=v[:, :, :1])),
            (TypeError, dict(key_pages=kp.half())),
            (ValueError, dict(value_pages=vp[:3])),
            (ValueError, dict(slots=slots.int())),
            (ValueError, dict(slots=slots[:1])),
            (ValueError, dict(slots=slots.cpu())),
            (ValueError, dict(slots=slots.T.contiguous().T)),
            (ValueError, dict(slots=slots[:1].expand(2, 5))),
            (cs.CsError, dict(value_pages=kp)),
            (cs.CsError, dict(key_pages=kp[:1].expand(4, 16, 2, 64))),
            (cs.CsError, dict(keys=kp[:2, :5]))):
        with pytest.raises(error):
            cs.paged_write(**{**good, **bad})
    assert torch.equal(kp, keep[0]) and torch.equal(vp, keep[1])
    assert cs.get_error() == set()


def test_captured_step():
    """Slots and the write in one graph, replayed on new lengths."""
    B, T, page = 5, 6, 16
    lengths, new = i32([0] * B).cuda(), i32([0] * B).cuda()
    own = torch.randperm(200).int().cuda()
    table, free = own[:100].view(B, 20).clone(), own[100:]
    k, v, _ = inputs(B, T, 2, 64, 100, page, torch.bfloat16)
    kp, vp = cache(200, page, 2, 64, torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cs.paged_extend(table, lengths, new, free, page, T)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        slots, totals, have, cursor = cs.paged_extend(table, lengths, new,
                                                      free, page, T)
        cs.paged_write(k, v, slots, kp, vp)
    for seed in range(4):
        r = random.Random(seed)
        more = [r.randint(0, T) for _ in range(B)]
        was = [r.randint(0, 200) for _ in range(B)]
        new.copy_(i32(more))
        lengths.copy_(i32(was))
        table.copy_(own[:100].view(B, 20))
        before = kp.clone(), table.tolist()
        graph.replay()
        want = extend(before[1], was, more, free.tolist(), page, T)
        assert table.tolist() == want[0] and slots.tolist() == want[1]
        assert torch.equal(kp, written(before[0], k, slots))
    assert cs.get_error() == set()
