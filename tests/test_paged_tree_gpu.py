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


@pytest.mark.parametrize("case,new", [
    (([300, 77, 0, 40, 513], 13, 12, 4, 80, 48), [13, 0, 0, 5, 1]),
    (([1000, 600], 33, 16, 2, 128, 16), [33, 2]),
    (([700, 90], 20, 5, 1, 256, 64), [1, 20]),
    (([3000, 1200, 0], 70, 4, 1, 64, 32), [3, 70, 0]),
], ids=str)
def test_fewer_new_tokens(case, new):
    """Rows behind a sequence's new tokens are zeros, whatever query and mask
    hold there; all of `out` is written."""
    args = cache(*case, seed=2)
    B, T = args[0].shape[:2]
    new = torch.tensor(new, dtype=torch.int32)
    mask = tree_mask(B, T, seed=2)
    for b in range(B):
        args[0][b, int(new[b]):] = math.nan
        mask[b, int(new[b]):] = True
        mask[b, :, int(new[b]):] = True
    want = definition(*args, mask, new)
    out = torch.full_like(args[0], 7.0).cuda()
    got = run(args, mask, new, out=out, return_lse=True)
    assert got[0] is out and cs.get_error() == set()
    compare(got, want)
    for b in range(B):
        assert (got[0][b, int(new[b]):] == 0).all()
    check(args, None, new)


def test_one_token_is_paged_attention():
    """A single new token attends what paged_attention gives it; several in a
    row, each what it would get alone."""
    args = cache([400, 33, 1290], 6, 8, 2, 128, 16, seed=3)
    q, k, v, table, lengths = (x.cuda() for x in args)
    last = cs.paged_tree_attention(q[:, -1:], k, v, table, lengths)
    one = cs.paged_attention(q[:, -1].contiguous(), k, v, table, lengths)
    # The weights of one are rounded to bf16, the other's are not: half a step
    # of each weight and of both results.
    scale = definition(*args)[0][:, -1].abs().amax()
    assert (last[:, 0].float() - one.float()).abs().max() < 3 * 2.0 ** -8 * scale * 4
    out, lse = cs.paged_tree_attention(q, k, v, table, lengths,
                                       return_lse=True)
    for i in range(6):
        single = cs.paged_attention(q[:, i].contiguous(), k, v, table,
                                    lengths - (5 - i), return_lse=True)
        compare((single[0].cpu()[:, None], single[1].cpu()[:, None]),
                [x[:, i:i + 1] for x in definition(*args)])
        assert (lse[:, i] - single[1]).abs().max() < 2.0 ** -12
    chain = torch.ones(6, 6, dtype=torch.bool, device="cuda").tril()
    masked = cs.paged_tree_attention(q, k, v, table, lengths, mask=chain)
    assert torch.equal(masked, out)


def test_masks_in_other_layouts():
    """One mask for all sequences, slices of a larger one, odd bases."""
    args = cache([300, 77], 13, 12, 4, 80, 48, seed=4)
    shared = tree_mask(1, 13)[0]
    want = run(args, shared.expand(2, 13, 13).contiguous())
    assert torch.equal(run(args, shared), want)
    dev = [x.cuda() for x in args]
    big = torch.ones(2, 20, 31, dtype=torch.bool, device="cuda")
    big[:, 3:16, 5:18] = shared.cuda()
    assert torch.equal(
        cs.paged_tree_attention(*dev, mask=big[:, 3:16, 5:18]), want)
    one = shared.cuda()[None].expand(2, 13, 13)
    assert torch.equal(cs.paged_tree_attention(*dev, mask=one), want)


def test_strided_caches_queries_and_outputs():
    """Keys and values in one buffer, heads before slots, a query that is a
    slice of a packed projection, an output that is a slice; what lies beside it
    stays.  An expanded cache, which tensor copies do not take."""
    for page in (16, 5):
        args = cache([333, 40, 0], 7, 6, 2, 80, page, seed=5)
        mask = tree_mask(3, 7)
        new = torch.tensor([7, 7, 0], dtype=torch.int32)
        dev = [x.cuda() for x in args]
        kw = dict(mask=mask.cuda(), new_lengths=new.cuda())
        want = cs.paged_tree_attention(*dev, **kw)
        both = torch.stack([dev[1], dev[2]], 1)
        assert torch.equal(want, cs.paged_tree_attention(
            dev[0], both[:, 0], both[:, 1], *dev[3:], **kw))
        hk, hv = (x.transpose(1, 2).contiguous().transpose(1, 2)
                  for x in dev[1:3])
        assert torch.equal(want, cs.paged_tree_attention(
            dev[0], hk, hv, *dev[3:], **kw))
        packed = torch.zeros(3, 7, 10, 96, dtype=want.dtype, device="cuda")
        packed[:, :, 1:7, 8:88] = dev[0]
        big = torch.full((4, 9, 8, 96), 7.0, dtype=want.dtype, device="cuda")
        got = cs.paged_tree_attention(packed[:, :, 1:7, 8:88], *dev[1:],
                                      out=big[:3, 1:8, 2:, 8:88], **kw)
        assert torch.equal(got, want)
        big[:3, 1:8, 2:, 8:88] = 7.0
        assert (big == 7.0).all()
        heads_first = dev[0].transpose(1, 2).contiguous().transpose(1, 2)
        assert torch.equal(want, cs.paged_tree_attention(heads_first,
                                                         *dev[1:], **kw))
    k = torch.randn(1, 1, 2, 64, device="cuda").bfloat16()
    many = k.expand(30, 16, 2, 64)
    q = torch.randn(2, 3, 4, 64, device="cuda").bfloat16()
    table = torch.zeros(2, 30, dtype=torch.int32, device="cuda")
    lengths = torch.tensor([480, 100], dtype=torch.int32, device="cuda")
    out = cs.paged_tree_attention(q, many, many, table, lengths)
    # Every token has the same value.
    value = k[0, 0].repeat_interleave(2, 0).double()
    assert ((out.double() - value).abs() <= 2.0 ** -7 * value.abs()).all()
    assert cs.get_error() == set()


@pytest.mark.parametrize("H,Hk", [(8, 2), (6, 2), (128, 1), (4, 4)])
def test_queries_in_other_layouts(H, Hk):
    """Queries that tensor copies take (key heads of a power of two of query
    heads) and others; expanded, token-major, one token or one head of more."""
    q, k, v, table, lengths = cache([300, 77, 150], 5, H, Hk, 64, 16, seed=11)
    args = (k, v, table, lengths)
    want = check((q, *args))
    q = q.cuda()     # (a copy to the device would straighten the strides)
    for other in (
            q.transpose(0, 1).contiguous().transpose(0, 1),
            q.transpose(1, 2).contiguous().transpose(1, 2),
            torch.nn.functional.pad(q, (8, 16, 1, 2, 3, 0))[:, 3:, 1:-2, 8:-16]):
        assert not other.is_contiguous()
        got = run((other, *args), return_lse=True)
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    one = q[:1].expand(3, 5, H, 64)
    got = run((one, *args), return_lse=True)
    check((one.cpu().contiguous(), *args))
    want = run((one.contiguous(), *args), return_lse=True)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    want = run((q[:, 4:].contiguous(), *args), return_lse=True)
    got = run((q[:, 4:], *args), return_lse=True)
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_offsets_past_32_bits():
    """Pages more than 2^32 elements apart, in both kinds of copies."""
    for page in (16, 3):
        args = cache([50, 3 * page], 5, 4, 2, 64, page, seed=6, extra=1)
        k, v = args[1], args[2]
        n = k.shape[0]
        step = (1 << 32) // n + 1 << 3
        big = torch.empty(((n - 1) * step + k[0].numel()) * 1, device="cuda",
                          dtype=torch.bfloat16)
        far = big.as_strided(k.shape, (step, 2 * 64, 64, 1))
        for x in (k, v):
            assert step * (n - 1) > 1 << 32
        far.copy_(k)
        q, vv, table, lengths = (x.cuda() for x in (args[0], v, *args[3:]))
        want = cs.paged_tree_attention(q, k.cuda(), vv, table, lengths)
        assert torch.equal(
            cs.paged_tree_attention(q, far, vv, table, lengths), want)
        far.copy_(v)
        assert torch.equal(
            cs.paged_tree_attention(q, k.cuda(), far, table, lengths), want)
        del big, far


@pytest.mark.parametrize("page", [16, 7, 128])
def test_bad_pages_and_lengths(page):
    """A page number outside the cache leaves its tokens out; lengths out of
    range are the nearest in it; all are reported."""
    args = cache([200, 900], 9, 4, 2, 64, page, seed=7)
    q, k, v, table, lengths = args
    mask = torch.ones(9, 9, dtype=torch.bool)
    for bad in (-1, k.shape[0], 2 ** 31 - 1, -2 ** 31):
        broken = table.clone()
        broken[0, 0] = bad
        got = run((q, k, v, broken, lengths), mask, return_lse=True)
        assert cs.get_error() == {"BAD_PAGE"}
        t2, n2 = table.clone(), lengths.clone()
        t2[0, :-1] = table[0, 1:]
        n2[0] -= page
        compare(got, definition(q, k, v, t2, n2, mask))
    new = torch.tensor([10, -4], dtype=torch.int32)
    got = run(args, mask, new, return_lse=True)
    assert cs.get_error() == {"BAD_PAGE"}
    compare(got, definition(*args, mask, torch.tensor([9, 0])))
    few = torch.tensor([4, -7], dtype=torch.int32)     # fewer than new tokens
    got = run((q, k, v, table, few), mask, return_lse=True)
    assert cs.get_error() == {"BAD_PAGE"}
    compare(got, definition(q, k, v, table, torch.tensor([4, 0]), mask,
                            torch.tensor([4, 0])))
    many = table.shape[1] * page + 50
    full = torch.arange(table.shape[1], dtype=torch.int32).expand(
        2, -1).contiguous() % k.shape[0]
    kk, vv = (torch.randn(k.shape).bfloat16() for _ in range(2))
    got = run((q, kk, vv, full, torch.tensor([many, 60], dtype=torch.int32)),
              mask, return_lse=True)
    assert cs.get_error() == {"BAD_PAGE"}
    compare(got, definition(q, kk, vv, full,
                            torch.tensor([many - 50, 60]), mask))


def test_every_page_bad():
    q, k, v, table, lengths = cache([100, 1400], 5, 4, 2, 128, 16)
    table = torch.full_like(table, -1)
    out, lse = run((q, k, v, table, lengths), return_lse=True)
    assert (out == 0).all() and (lse == -math.inf).all()
    assert cs.get_error() == {"BAD_PAGE"}
    nothing = torch.empty(0, 16, 2, 128, dtype=q.dtype)
    out = run((q, nothing, nothing, table, lengths))
    assert (out == 0).all() and cs.get_error() == {"BAD_PAGE"}


def test_nothing_to_do():
    q, k, v, table, lengths = cache([40, 300], 5, 4, 2, 64, 16)
    none = run((q, k, v, table, torch.zeros_like(lengths)), new=torch.zeros(
        2, dtype=torch.int32))
    assert (none == 0).all() and cs.get_error() == set()
    empty = run((q[:, :0], k, v, table, lengths))
    assert empty.shape == (2, 0, 4, 64)
    empty = run((q[:0], k, v, table[:0], lengths[:0]))
    assert empty.shape == (0, 5, 4, 64)
    out, lse = run((q, k, v, table[:, :0], torch.zeros_like(lengths)),
                   new=torch.zeros(2, dtype=torch.int32), return_lse=True)
    assert (out == 0).all() and (lse == -math.inf).all()


@pytest.mark.parametrize("D,page", [(64, 16), (128, 5), (256, 64)])
def test_what_a_nan_reaches(D, page):
    """A NaN query its row; a NaN key the rows that attend it; a NaN value the
    rows of its sequence and head.  Infinite keys of removed tokens nothing."""
    args = cache([700, 300], 6, 4, 2, D, page, seed=8)
    mask = tree_mask(2, 6, seed=3)
    mask[0, :, 4] = False
    mask[0, 4, 4] = True                      # new token 4: row 4 alone
    want, _ = run(args, mask, return_lse=True)
    cs.get_error()
    j = 700 - 6 + 4
    at = (int(args[3][0, j // page]), j % page)
    for which, x in (("query", math.nan), ("key", math.nan),
                     ("key", math.inf), ("value", math.nan)):
        q, k, v, table, lengths = (x.clone() for x in args)
        hit = torch.zeros(2, 6, 4, dtype=torch.bool)
        if which == "query":
            q[0, 2, 1, 3] = x
            hit[0, 2, 1] = True
        elif which == "key":
            k[at[0], at[1], 1, 5] = x
            hit[0, 4, 2:] = True
        else:
            v[at[0], at[1], 1, 5] = x
            hit[0, :, 2:] = True
        got, lse = run((q, k, v, table, lengths), mask, return_lse=True)
        errors = cs.get_error()
        assert torch.equal(got.cpu()[~hit], want.cpu()[~hit])
        if which != "value":
            assert errors == {"NAN_INPUT"} or math.isinf(x)
        if which == "key" and math.isnan(x) or which == "query":
            assert got.cpu()[hit].isnan().all() and lse.cpu()[hit].isnan().all()
        if which == "value":
            assert got.cpu()[0, 4, 2:, 5].isnan().all() and errors == set()


@pytest.mark.parametrize("batch", [1, 75, 257, 700, 3000])
def test_many_sequences(batch):
    """Around and past the sequences whose lengths one warp adds up, some empty
    and some without new tokens: shares and a join against whole sequences in a
    table of few pages."""
    gen = torch.Generator(device="cuda").manual_seed(batch)
    lengths = torch.randint(4, 17, (batch,), dtype=torch.int32, device="cuda",
                            generator=gen)
    k, v = (torch.randn(batch, 16, 2, 64, device="cuda",
                        generator=gen).bfloat16() for _ in range(2))
    table = torch.zeros(batch, 80, dtype=torch.int32, device="cuda")
    table[:, 0] = torch.randperm(batch, device="cuda", generator=gen)
    longer = torch.arange(batch, device="cuda") % 5 == 0
    table[longer, 1:32] = torch.randint(
        0, batch, (int(longer.sum()), 31), dtype=torch.int32, device="cuda",
        generator=gen)
    lengths[longer] += 496
    new = torch.full_like(lengths, 4)
    new[1::7] = 0
    lengths[1::14] = 0
    q = torch.randn(batch, 4, 8, 64, device="cuda", generator=gen).bfloat16()
    args = (q, k, v, table, lengths)
    mask = torch.ones(4, 4, dtype=torch.bool, device="cuda").tril()
    wide = cs.paged_tree_attention(*args, mask=mask, new_lengths=new,
                                   return_lse=True)
    few = cs.paged_tree_attention(q, k, v, table[:, :32].contiguous(), lengths,
                                  new_lengths=new, return_lse=True)
    assert cs.get_error() == set()
    a, b = wide[0].float(), few[0].float()
    # Weights of other maxima round otherwise: a step of the result's type, and
    # half a step of each weight of values of about 1 (up to 4.5).
    assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 2 * 2.0 ** -8 * 4.5).all()
    empty = few[1] == -math.inf
    assert torch.equal(wide[1] == -math.inf, empty)
    assert torch.equal(empty[:, 0, 0], new == 0)
    assert ((wide[1] - few[1]).abs()[~empty]
            <= 2.0 ** -16 * (1 + few[1].abs()[~empty])).all()
    some = [0, batch // 2, batch - 1]
    compare([x[some].cpu() for x in wide],
            definition(q[some].cpu(), k.cpu(), v.cpu(), table[some].cpu(),
                       lengths[some].cpu(), mask.cpu(), new[some].cpu()))


@pytest.mark.parametrize("B,T,H,Hk,D,longest", [
    (10, 256, 8, 8, 128, 1300),   # a join for each sequence, many rows,
    (3, 40, 16, 4, 64, 2600),     # some,
    (1, 5, 8, 4, 80, 5900),       # and few, of many parts;
    (20, 256, 8, 8, 128, 1100),   # one for each place between two groups
    (40, 9, 8, 2, 96, 1500),
    (170, 1, 1, 1, 64, 900),
])
def test_joins(B, T, H, Hk, D, longest):
    """Units that are cut, joined in each of the ways there are."""
    gen = torch.Generator().manual_seed(B)
    lengths = torch.randint(T, longest, (B,), generator=gen).tolist()
    args = cache(lengths, T, H, Hk, D, 16, seed=B)
    table = torch.nn.functional.pad(args[3], (0, 64))   # rows for 1024 more
    check((*args[:3], table, args[4]), tree_mask(1, T, seed=B)[0])


def test_repeated_calls_give_the_same_bits():
    for case in CASES:
        args = [x.cuda() for x in cache(*case, seed=9)]
        mask = tree_mask(*args[0].shape[:2]).cuda()
        first = cs.paged_tree_attention(*args, mask=mask, return_lse=True)
        for _ in range(5):
            again = cs.paged_tree_attention(*args, mask=mask, return_lse=True)
            assert all(torch.equal(x, y) for x, y in zip(first, again))


def test_streams_and_threads():
    """Calls at once from several threads, each on its own stream."""
    import threading
    jobs = []
    for n, case in enumerate(CASES[3:] * 2):
        args = [x.cuda() for x in cache(*case, seed=20 + n)]
        mask = tree_mask(*args[0].shape[:2], seed=n).cuda()
        jobs.append((args, mask, cs.paged_tree_attention(*args, mask=mask)))
    torch.cuda.synchronize()
    wrong = []

    def work(part):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(5):
                for args, mask, want in part:
                    got = cs.paged_tree_attention(*args, mask=mask)
                    stream.synchronize()
                    if not torch.equal(got, want):
                        wrong.append(tuple(args[0].shape))

    threads = [threading.Thread(target=work, args=(jobs[i::4],))
               for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and cs.get_error() == set()


def test_captured_calls():
    """Two graphs captured one after the other, replayed in turn on new inputs
    and lengths."""
    shapes = [([2500, 300], 9, 8, 2, 128, 16), ([700, 40, 90], 40, 8, 2, 64, 5)]
    graphs = []
    for n, case in enumerate(shapes):
        args = [x.cuda() for x in cache(*case, seed=n)]
        mask = tree_mask(*args[0].shape[:2]).cuda()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            cs.paged_tree_attention(*args, mask=mask)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = cs.paged_tree_attention(*args, mask=mask, return_lse=True)
        graphs.append((graph, args, mask, out, case))
    for seed in (30, 31, 32):
        for graph, args, mask, out, case in graphs:
            shorter = [max(n - 7 * (seed - 30), case[1]) for n in case[0]]
            fresh = cache(case[0], *case[1:], seed=seed)
            for dst, src in zip(args, fresh):
                dst.copy_(src)
            args[4].copy_(torch.tensor(shorter))
            mask.copy_(tree_mask(*mask.shape[:2], seed=seed))
        for graph, *_ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for graph, args, mask, out, case in graphs:
            want = cs.paged_tree_attention(*args, mask=mask, return_lse=True)
            assert all(torch.equal(x, y) for x, y in zip(out, want))
    assert cs.get_error() == set()


def test_random_cases():
    """Seeded draws over the documented ranges."""
    import random
    r = random.Random(11)
    for n in range(60):
        Hk = r.choice([1, 2, 3])
        H = Hk * r.choice([1, 2, 4, 5, 8, 20])
        D = 8 * r.randint(1, 32)
        T = r.choice([1, 2, 7, 30, 64, 100])
        page = r.choice([1, 8, 16, 24, 64, 96, 128, 256, r.randint(1, 300)])
        lengths = [max(T, r.choice([T, r.randint(1, 300), r.randint(1, 3000)]))
                   for _ in range(r.randint(1, 4))]
        args = cache(lengths, T, H, Hk, D, page, seed=n,
                     dtype=r.choice([torch.bfloat16, torch.float16]))
        mask = r.choice([None, tree_mask(len(lengths), T, n),
                         tree_mask(len(lengths), T, n, empty=True)])
        new = r.choice([None, torch.tensor(
            [r.randint(0, T) for _ in lengths], dtype=torch.int32)])
        check(args, mask, new, r.choice([None, 0.3, 1.5]))


def test_largest_sizes():
    """2^16 key heads of one new token, the most rows of a key head that fit a
    test, and a row of the table with room for 2^30 tokens."""
    gen = torch.Generator(device="cuda").manual_seed(2)

    def rand(*shape):
        return torch.randn(*shape, device="cuda", generator=gen).bfloat16()

    H = 1 << 16
    k, v = rand(1, 8, H, 8), rand(1, 8, H, 8)
    q = rand(1, 2, H, 8)
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    lengths = torch.tensor([5], dtype=torch.int32, device="cuda")
    out, lse = cs.paged_tree_attention(q, k, v, table, lengths,
                                       return_lse=True)
    pick = [0, 1, H // 2, H - 1]
    compare([x[:, :, pick].cpu() for x in (out, lse)],
            definition(q[:, :, pick].cpu(), k[:, :, pick].cpu(),
                       v[:, :, pick].cpu(), table.cpu(), lengths.cpu()))
    T = 1 << 15
    k, v = rand(T // 128, 128, 1, 64), rand(T // 128, 128, 1, 64)
    q = rand(1, T, 2, 64)
    table = torch.arange(T // 128, dtype=torch.int32, device="cuda")[None]
    lengths = torch.tensor([T], dtype=torch.int32, device="cuda")
    out, lse = cs.paged_tree_attention(q, k, v, table.contiguous(), lengths,
                                       return_lse=True)
    fused = cs.fused_attention(
        q.transpose(1, 2), k.view(1, 1, T, 64), v.view(1, 1, T, 64),
        causal=True, return_lse=True)
    assert ((lse.transpose(1, 2) - fused[1]).abs().max()) < 2.0 ** -10
    a, b = out.transpose(1, 2).float(), fused[0].float()
    assert float((a - b).norm() / b.norm()) < 2 * 2.0 ** -8
    k, v = rand(1, 1, 1, 8), rand(1, 1, 1, 8)
    many = (x.expand(1, 1 << 30, 1, 8) for x in (k, v))
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    lengths = torch.tensor([1 << 30], dtype=torch.int32, device="cuda")
    q = rand(1, 2, 2, 8)
    out, lse = cs.paged_tree_attention(q, *many, table, lengths,
                                       return_lse=True)
    value = v[0, 0, 0].double()
    # Half a step of bf16 (2^-8), and an accumulator that truncates: by at most
    # 2^-23 at each of its 2^30 / (152 CTAs, 2 accumulators, 16 tokens) =
    # 2^17.75 steps.
    assert ((out.double() - value).abs()
            <= (2.0 ** -8 + 2.0 ** -5.25) * value.abs()).all()
    s = (q.double() @ k[0, 0, 0].double()) * 8 ** -0.5
    n = torch.tensor([2.0 ** 30 - 1, 2.0 ** 30], device="cuda").double()
    assert float((lse.double() - s - n.log()[None, :, None]).abs().max()) \
        < 2.0 ** -16
    assert cs.get_error() == set()


def test_refusals():
    q, k, v, table, lengths = (x.cuda() for x in cache([40, 300], 5, 4, 2, 64,
                                                       16))
    mask = torch.ones(5, 5, dtype=torch.bool, device="cuda")
    good = dict(query=q, key_pages=k, value_pages=v, page_table=table,
                lengths=lengths, mask=mask)
    want = cs.paged_tree_attention(**good)
    wide = torch.zeros(2, 5, 4, 65, dtype=q.dtype, device="cuda")
    for error, bad in (
            (ValueError, dict(query=q.cpu())), (ValueError, dict(query=q[0])),
            (TypeError, dict(query=q.float())), (TypeError, dict(query=q.half())),
            (ValueError, dict(query=q[..., :60])),
            (ValueError, dict(query=q[:, :, :3])),
            (ValueError, dict(query=wide[..., :64])),
            (ValueError, dict(key_pages=k[..., :32])),
            (ValueError, dict(value_pages=v[:-1])),
            (TypeError, dict(value_pages=v.half())),
            (ValueError, dict(page_table=table.long())),
            (ValueError, dict(page_table=table[:1])),
            (ValueError, dict(page_table=table.cpu())),
            (ValueError, dict(lengths=lengths.long())),
            (ValueError, dict(lengths=lengths[:1])),
            (ValueError, dict(new_lengths=lengths.long())),
            (ValueError, dict(new_lengths=lengths[:1])),
            (ValueError, dict(mask=mask.int())),
            (ValueError, dict(mask=mask[:4])),
            (ValueError, dict(mask=mask.cpu())),
            (ValueError, dict(mask=mask.expand(3, 5, 5))),
            (ValueError, dict(mask=mask.T[:, :1].expand(5, 5))),
            (ValueError, dict(mask=mask[:1].expand(5, 5))),
            (ValueError, dict(scale=0.0)), (ValueError, dict(scale=-1.0)),
            (ValueError, dict(scale=math.inf)),
            (ValueError, dict(scale=math.nan)),
            (ValueError, dict(out=torch.empty_like(q)[:, :4])),
            (TypeError, dict(out=torch.empty_like(q).half())),
            (cs.CsError, dict(out=q)),
            (cs.CsError, dict(out=torch.empty(
                1, 5, 4, 64, dtype=q.dtype, device="cuda").expand(q.shape)))):
        with pytest.raises(error):
            cs.paged_tree_attention(**{**good, **bad})
    assert torch.equal(cs.paged_tree_attention(**good), want)
    assert cs.get_error() == set()
