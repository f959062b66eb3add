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
