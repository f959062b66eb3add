"""The operators around a paged cache as a server runs them: prompts in chunks,
then trees of drafted tokens of which some are accepted, then single tokens; one
attention layer, against attention over the tokens that count, in 64 bits."""
import math
import random

import pytest

torch = pytest.importorskip("torch")

import entropy_bounded_softmax_gb300 as cs
from paged_parity import tree_mask

pytestmark = pytest.mark.gpu

H, HK = 8, 2


class Server:
    """Sequences in a paged cache.  `kept` holds, on the CPU, the keys and
    values of the tokens that count, in their order."""

    def __init__(self, B, D, page, pages, dtype, seed):
        gen = torch.Generator().manual_seed(seed)
        self.page, self.D, self.dtype, self.gen = page, D, dtype, gen
        self.pages = [torch.full((pages, page, HK, D), math.nan, dtype=dtype,
                                 device="cuda") for _ in range(2)]
        self.table = torch.full((B, 64), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(pages, generator=gen).int().cuda()
        self.cursor = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.lengths = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.held = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.kept = [[torch.empty(0, HK, D, dtype=dtype)] * 2
                     for _ in range(B)]

    def step(self, new, T, mask=None):
        """Queries, keys and values of up to T new tokens through the cache;
        the attention's output, and what it has to be with its allowance."""
        B, D = len(new), self.D
        q, k, v = (torch.randn(B, T, h, D, generator=self.gen).to(self.dtype)
                   for h in (H, HK, HK))
        count = torch.tensor(new, dtype=torch.int32, device="cuda")
        slots, totals, self.held, self.cursor = cs.paged_extend(
            self.table, self.lengths, count, self.free, self.page, T,
            held=self.held, cursor=self.cursor)
        cs.paged_write(k.cuda(), v.cuda(), slots, *self.pages)
        out = cs.paged_tree_attention(
            q.cuda(), *self.pages, self.table, totals,
            mask=None if mask is None else mask.cuda(), new_lengths=count)
        if T == 1:
            one = cs.paged_attention(q[:, 0].cuda(), *self.pages, self.table,
                                     totals)
            half = torch.finfo(self.dtype).eps / 2
            assert (one[count > 0].float() - out[count > 0, 0].float()
                    ).abs().max() < 4 * half * 4.5
        assert cs.get_error() == set()
        self.check(out.cpu().double(), q, k, v, new, mask)
        return k, v, totals

    def check(self, out, q, k, v, new, mask):
        half = torch.finfo(self.dtype).eps / 2
        for b, n in enumerate(new):
            assert (out[b, n:] == 0).all()
            if n == 0:
                continue
            old = self.kept[b][0].shape[0]
            keys = torch.cat([self.kept[b][0], k[b, :n]]).double()
            values = torch.cat([self.kept[b][1], v[b, :n]]).double()
            sees = torch.ones(n, old + n, dtype=torch.bool)
            sees[:, old:] = (torch.ones(n, n, dtype=torch.bool).tril()
                             if mask is None else mask[b, :n, :n])
            for h in range(H):
                s = q[b, :n, h].double() @ keys[:, h * HK // H].T
                s = (s * self.D ** -0.5).masked_fill(~sees, -math.inf)
                p = torch.softmax(s, 1)
                x = values[:, h * HK // H]
                # Half a step of the result and of each weight; the scores' and
                # sums' fp32 below a sixteenth of that.
                tol = (half * (p @ x).abs() + 1.0625 * half * (p @ x.abs())
                       + 2.0 ** -24)
                assert ((out[b, :n, h] - p @ x).abs() <= tol).all()

    def accept(self, k, v, path):
        """Keeps the new tokens of each sequence's path: their keys and values
        move to the first slots behind its tokens."""
        B, T = k.shape[:2]
        longest = max(1, max(len(x) for x in path))
        slots = torch.full((B, longest), -1, dtype=torch.int64, device="cuda")
        moved = [torch.zeros(B, longest, HK, self.D, dtype=self.dtype,
                             device="cuda") for _ in range(2)]
        table = self.table.cpu()
        for b, nodes in enumerate(path):
            old = self.kept[b][0].shape[0]
            for i, node in enumerate(nodes):
                at = old + i
                slots[b, i] = (int(table[b, at // self.page]) * self.page
                               + at % self.page)
                moved[0][b, i], moved[1][b, i] = k[b, node], v[b, node]
            self.kept[b] = [torch.cat([x, y[b, nodes]]) for x, y in
                            zip(self.kept[b], (k, v))]
        cs.paged_write(*moved, slots, *self.pages)
        self.lengths = torch.tensor([x[0].shape[0] for x in self.kept],
                                    dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("D,page", [(64, 16), (128, 5), (80, 64), (256, 8)])
def test_prompts_trees_and_tokens(D, page, dtype):
    r = random.Random(D + page)
    s = Server(5, D, page, 5 * 64, dtype, seed=D)
    prompts = [300, 1, 77, 150, 0]
    done = [0] * 5
    if 64 * page < 400:
        prompts = [64 * page * n // 400 for n in prompts]
    while any(d < n for d, n in zip(done, prompts)):     # in chunks of 64
        new = [min(64, n - d) for d, n in zip(done, prompts)]
        k, v, totals = s.step(new, 64)
        assert totals.tolist() == [d + n for d, n in zip(done, new)]
        s.accept(k, v, [list(range(n)) for n in new])
        done = [d + n for d, n in zip(done, new)]
    for seed in range(4):
        T = 13
        mask = tree_mask(5, T, seed=seed)
        new = [r.randint(0, T) for _ in range(5)]
        k, v, _ = s.step(new, T, mask)
        paths = []
        for b, n in enumerate(new):            # one node and its ancestors
            leaf = r.randint(-1, n - 1)
            paths.append([] if leaf < 0 else
                         mask[b, leaf].nonzero().flatten().tolist())
        s.accept(k, v, paths)
        k, v, _ = s.step([1, 1, 0, 1, 1], 1)
        s.accept(k, v, [[0], [0], [], [0], [0]])
    # No page was taken twice or lost.
    held, table = s.held.tolist(), s.table.tolist()
    taken = [x for row, n in zip(table, held) for x in row[:n]]
    assert sorted(taken) == sorted(s.free[:int(s.cursor)].tolist())
    for n, length in zip(held, s.lengths.tolist()):
        assert n * page >= length


def test_pool_runs_dry():
    """Tokens without a page are in no result; what is there stays right."""
    s = Server(3, 64, 16, 6, torch.bfloat16, seed=1)
    q, k, v = (torch.randn(3, 40, h, 64).bfloat16().cuda()
               for h in (H, HK, HK))
    new = torch.tensor([40, 40, 40], dtype=torch.int32, device="cuda")
    slots, totals, held, cursor = cs.paged_extend(
        s.table, s.lengths, new, s.free, 16, 40)
    assert cs.get_error() == {"OUT_OF_PAGES"}
    assert totals.tolist() == [40, 40, 0] and held.tolist() == [3, 3, 0]
    assert cursor.tolist() == [6] and (slots[2] == -1).all()
    cs.paged_write(k, v, slots, *s.pages)
    out = cs.paged_tree_attention(q, *s.pages, s.table, totals,
                                  new_lengths=totals)
    want = cs.fused_attention(q.transpose(1, 2), k.transpose(1, 2),
                              v.transpose(1, 2), causal=True).transpose(1, 2)
    assert (out[2] == 0).all() and cs.get_error() == set()
    # Two roundings of results and weights.
    assert (out[:2].float() - want[:2].float()).abs().max() < 4 * 2.0 ** -8 * 4.5


@pytest.mark.parametrize("B,most", [(3, 4096), (40, 512), (300, 16)])
def test_lengths_of_the_call_before(B, most):
    """paged_tree_attention with the lengths that paged_extend just wrote: what
    its kernels look up ahead may not be of the lengths before.  One captured
    run, replayed with lengths that grow and shrink."""
    T, D, page, dtype = 4, 64, 16, torch.bfloat16
    gen = torch.Generator().manual_seed(B)
    longest = 3000 if B < 10 else 600
    entries = (longest + most) // page + 1
    pages = [torch.randn(2048, page, HK, D, generator=gen).to(dtype).cuda()
             for _ in range(2)]
    table = torch.randint(0, 2048, (B, entries), generator=gen).int().cuda()
    free = torch.arange(2048, dtype=torch.int32, device="cuda")
    q = torch.randn(B, T, H, D, generator=gen).to(dtype).cuda()
    count = torch.randint(0, T + 1, (B,), generator=gen).int().cuda()
    lengths = torch.zeros(B, dtype=torch.int32, device="cuda")

    def run():
        totals = cs.paged_extend(table, lengths, count, free, page, most)[1]
        return cs.paged_tree_attention(q, *pages, table, totals,
                                       new_lengths=count)

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for i in range(12):
        top = longest if i % 2 else 1 + longest // 50
        now = torch.randint(0, top, (B,), generator=gen).int().cuda()
        lengths.copy_(now)
        torch.cuda.synchronize()
        graph.replay()
        got = out.clone()
        want = cs.paged_tree_attention(q, *pages, table, now + count,
                                       new_lengths=count)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        assert cs.get_error() <= {"OUT_OF_PAGES"}


@pytest.mark.parametrize("B,T,page", [(3, 5, 16), (24, 4, 64), (2, 64, 5)])
def test_captured_step(B, T, page):
    """A step of drafts as one captured graph, its state updated in place, over
    steps that take new pages; each as the same calls made one by one."""
    D, dtype, steps = 128, torch.bfloat16, 12
    gen = torch.Generator().manual_seed(B)
    entries = (600 + steps * T) // page + 2
    num = B * entries
    start = torch.randint(0, 600, (B,), generator=gen).int()
    pages = torch.randn(2, num, page, HK, D, generator=gen).to(dtype).cuda()
    free = torch.randperm(num, generator=gen).int().cuda()
    table = torch.full((B, entries), -1, dtype=torch.int32, device="cuda")
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    _, lengths, held, cursor = cs.paged_extend(table, zero, start.cuda(), free,
                                               page, 600)
    count = torch.zeros(B, dtype=torch.int32, device="cuda")
    q = torch.zeros(B, T, H, D, dtype=dtype, device="cuda")
    k, v = (torch.zeros(B, T, HK, D, dtype=dtype, device="cuda")
            for _ in range(2))
    mask = torch.zeros(B, T, T, dtype=torch.bool, device="cuda")

    def step(table, lengths, held, cursor, pages, wait=False):
        def settle():
            if wait:
                torch.cuda.synchronize()
        slots, totals, have, after = cs.paged_extend(
            table, lengths, count, free, page, T, held=held, cursor=cursor)
        settle()
        cs.paged_write(k, v, slots, *pages)
        settle()
        out, lse = cs.paged_tree_attention(q, *pages, table, totals, mask,
                                           count, return_lse=True)
        settle()
        return out, lse, totals, have, after

    copies = [x.clone() for x in (table, lengths, held, cursor, pages)]
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step(*[x.clone() for x in copies])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse, totals, have, after = step(table, lengths, held, cursor,
                                             pages)
        lengths.copy_(totals)
        held.copy_(have)
        cursor.copy_(after)
    for i in range(steps):
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=gen))
        mask.copy_(tree_mask(B, T, seed=i))
        count.copy_(torch.randint(0, T + 1, (B,), generator=gen))
        graph.replay()
        want = step(*copies, wait=True)
        for x, y in zip(copies[1:4], want[2:]):
            x.copy_(y)
        torch.cuda.synchronize()
        for x, y in zip((out, lse, totals, have, after), want):
            assert torch.equal(x, y)
        assert torch.equal(table, copies[0]) and torch.equal(pages, copies[4])
        assert cs.get_error() == set()
