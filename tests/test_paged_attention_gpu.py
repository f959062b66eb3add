"""paged_attention against its definition in 64 bits: lengths around tiles,
pages and chunks, shared key heads, page sizes that end inside a tile, both
element types, and caches with bad entries.

Allowance per element: half a step of the result's type; the weights enter
as two halves, 2^-16 of each in bf16 (2^-21 in fp16); a score's dot product
errs by (D + 8) 2^-23 of the sum of its terms' magnitudes, 2^x by 2^-21; the
sums of n <= 6000 terms by 2^-17 of the sum of magnitudes (each step rounds
by 2^-24, mostly cancelling)."""
import math

import pytest

torch = pytest.importorskip("torch")

import entropy_bounded_softmax_gb300 as cs

pytestmark = pytest.mark.gpu

F32 = 2.0 ** -23


def cache(lengths, H, Hk, D, page, dtype=torch.bfloat16, seed=0, extra=3):
    """A cache whose pages lie in no order, with spare pages and spare table
    entries (both hold what a reader must not use)."""
    gen = torch.Generator().manual_seed(seed)
    per = [-(-n // page) for n in lengths]
    total = sum(per) + extra

    def pages():
        return torch.randn(total, page, Hk, D, generator=gen).to(dtype)

    k, v = pages(), pages()
    order = torch.randperm(total, generator=gen).to(torch.int32)
    table = torch.full((len(lengths), max(max(per), 1) + 1), -7,
                       dtype=torch.int32)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        at += n
        if lengths[b] % page:   # the slots past the length
            for x in (k, v):
                x[order[at - 1], lengths[b] % page:] = math.nan
    for x in (k, v):
        x[order[at:].long()] = math.nan
    q = torch.randn(len(lengths), H, D, generator=gen).to(dtype)
    return q, k, v, table, torch.tensor(lengths, dtype=torch.int32)


def definition(q, k, v, table, lengths, scale):
    B, H, D = q.shape
    page, Hk = k.shape[1:3]
    half = torch.finfo(q.dtype).eps / 2
    split = 2.0 ** -16 if q.dtype == torch.bfloat16 else 2.0 ** -21
    out = torch.zeros(B, H, D, dtype=torch.float64)
    tol = torch.full_like(out, 1e-37)
    lse = torch.full((B, H), -math.inf, dtype=torch.float64)
    tol_lse = torch.zeros(B, H, dtype=torch.float64)
    for b, n in enumerate(lengths.tolist()):
        if n == 0:
            continue
        j = torch.arange(n)
        rows = table[b, j // page].long()
        for h in range(H):
            kk = k[rows, j % page, h * Hk // H].double()
            vv = v[rows, j % page, h * Hk // H].double()
            qq = q[b, h].double()
            s = kk @ qq * scale
            lse[b, h] = torch.logsumexp(s, 0)
            p = torch.exp(s - lse[b, h])
            out[b, h] = p @ vv
            es = (2 * (D + 8) * F32 * scale * float((kk.abs() @ qq.abs()).max())
                  + 4 * F32 * float(s.abs().max()) + 2.0 ** -21 + 2.0 ** -17)
            tol[b, h] += (half * out[b, h].abs()
                          + (2 * es + split) * (p @ vv.abs()))
            tol_lse[b, h] = es + 4 * F32 * lse[b, h].abs()
    return out, tol, lse, tol_lse


def check(args, scale=None, errors=frozenset()):
    q, k, v, table, lengths = args
    dev = [x.cuda() for x in args]
    out, lse = cs.paged_attention(*dev, scale=scale, return_lse=True)
    assert out.dtype == q.dtype and out.shape == q.shape
    assert cs.get_error() == errors
    want, tol, wlse, tlse = definition(
        *args, 1 / math.sqrt(q.shape[2]) if scale is None else scale)
    assert ((out.cpu().double() - want).abs() <= tol).all()
    empty = wlse == -math.inf
    assert torch.equal(lse.cpu() == -math.inf, empty)
    assert ((lse.cpu().double() - wlse).abs()[~empty] <= tlse[~empty]).all()
    return out, lse


CASES = [
    # lengths, H, Hk, D, page
    ([1], 1, 1, 8, 1),
    ([0, 1, 15, 16, 17], 4, 2, 64, 16),
    ([63, 64, 65, 127, 128, 129], 8, 8, 128, 16),    # around a chunk of 128
    ([255, 1, 257], 8, 1, 64, 5),                    # pages end inside tiles
    ([300, 77], 12, 4, 80, 48),
    ([1000, 3, 0, 511], 16, 2, 128, 1),
    ([700], 5, 1, 256, 64),
    ([200, 90], 40, 2, 96, 32),                      # 20 heads: two tiles
    ([130, 20], 64, 1, 16, 256),
    ([5000, 17], 8, 2, 120, 100),
    ([333, 64], 3, 3, 200, 7),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("case", CASES, ids=str)
def test_against_definition(case, dtype):
    check(cache(*case, dtype=dtype))


def test_rows_are_split_and_joined():
    """More CTAs than rows: the rows' steps are dealt out, and the parts
    join; a batch of short sequences needs no workspace."""
    args = cache([4111, 300, 0, 128], 8, 2, 64, 16)
    shape = cs.cs_paged_shape(4, 8, 2, 64, 16, args[1].shape[0],
                              args[3].shape[1], 0, 1.0)
    assert cs.cs_paged_attention_workspace(shape) > 0
    check(args)
    shape.max_pages = 16
    assert cs.cs_paged_attention_workspace(shape) == 0


def test_many_sequences():
    """More sequences than a CTA has threads, some without tokens: the walk
    over the lengths takes several rounds."""
    lengths = [(37 * b) % 400 for b in range(300)]
    check(cache(lengths, 2, 1, 64, 16))


def test_bad_pages_and_lengths():
    """A page number outside the cache leaves its tokens out; a length past
    the table is the table's, a negative one nothing; all are reported."""
    q, k, v, table, lengths = cache([200, 90, 300], 4, 2, 64, 16)
    table, lengths = table.clone(), lengths.clone()
    for bad in (-1, k.shape[0], 2 ** 31 - 1, -2 ** 31):
        broken = table.clone()
        broken[0, 3] = bad
        dev = [x.cuda() for x in (q, k, v, broken, lengths)]
        out, lse = cs.paged_attention(*dev, return_lse=True)
        assert cs.get_error() == {"BAD_PAGE"}
        # The same as a sequence without that page.
        keep = [i for i in range(table.shape[1]) if i != 3]
        t2, n2 = table.clone(), lengths.clone()
        t2[0, :len(keep)] = table[0, keep]
        n2[0] -= 16
        want, tol, wlse, tlse = definition(q, k, v, t2, n2, 1 / 8)
        assert ((out.cpu().double() - want).abs() <= tol).all()
        assert ((lse.cpu().double() - wlse).abs() <= tlse).all()
    full = torch.arange(19, dtype=torch.int32)[None].contiguous()
    qq = q[:1].cuda()
    kk, vv = (torch.randn(19, 16, 2, 64).bfloat16() for _ in range(2))
    args = (kk.cuda(), vv.cuda(), full.cuda())
    long = cs.paged_attention(
        qq, *args, torch.tensor([5000], dtype=torch.int32).cuda())
    assert cs.get_error() == {"BAD_PAGE"}
    want = cs.paged_attention(
        qq, *args, torch.tensor([304], dtype=torch.int32).cuda())
    assert torch.equal(long, want) and cs.get_error() == set()
    none = cs.paged_attention(
        qq, *args, torch.tensor([-3], dtype=torch.int32).cuda())
    assert (none == 0).all() and cs.get_error() == {"BAD_PAGE"}


def test_every_page_bad():
    q, k, v, table, lengths = cache([100, 400], 4, 2, 128, 16)
    table = torch.full_like(table, -1)
    out, lse = cs.paged_attention(*(x.cuda() for x in (q, k, v, table,
                                                       lengths)),
                                  return_lse=True)
    assert (out == 0).all() and (lse == -math.inf).all()
    assert cs.get_error() == {"BAD_PAGE"}
    nothing = torch.empty(0, 16, 2, 128, dtype=q.dtype, device="cuda")
    out = cs.paged_attention(q.cuda(), nothing, nothing, table.cuda(),
                             lengths.cuda())
    assert (out == 0).all() and cs.get_error() == {"BAD_PAGE"}


def test_strided_caches_and_outputs():
    """Keys and values side by side in one buffer, heads before slots, a query
    and an output that are slices; what lies beside the output stays."""
    q, k, v, table, lengths = cache([333, 40, 0], 6, 2, 80, 16)
    dev = [x.cuda() for x in (q, k, v, table, lengths)]
    want = cs.paged_attention(*dev)
    both = torch.stack([k, v], 1).cuda()              # [pages, 2, page, Hk, D]
    got = cs.paged_attention(dev[0], both[:, 0], both[:, 1], *dev[3:])
    assert torch.equal(got, want)
    hk, hv = (x.cuda().transpose(1, 2).contiguous().transpose(1, 2)
              for x in (k, v))
    assert torch.equal(cs.paged_attention(dev[0], hk, hv, *dev[3:]), want)
    wide = torch.zeros(3, 9, 96, dtype=q.dtype, device="cuda")
    wide[:, 2:8, 8:88] = dev[0]
    big = torch.full((4, 9, 96), 7.0, dtype=q.dtype, device="cuda")
    got = cs.paged_attention(wide[:, 2:8, 8:88], *dev[1:],
                             out=big[:3, 2:8, 8:88])
    assert torch.equal(got, want)
    big[:3, 2:8, 8:88] = 7.0
    assert (big == 7.0).all()


def test_caches_past_32_bits():
    """Pages more than 2^31 elements into the cache."""
    page, Hk, D = 16, 8, 128
    pages = (1 << 31) // (page * Hk * D) + 50
    k = torch.empty(pages, page, Hk, D, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    q, k0, v0, table, lengths = cache([500], 8, 8, D, page)
    shift = pages - k0.shape[0]
    k[shift:], v[shift:] = k0.cuda(), v0.cuda()
    want = cs.paged_attention(*(x.cuda() for x in (q, k0, v0, table, lengths)))
    got = cs.paged_attention(q.cuda(), k, v, (table + shift).cuda(),
                             lengths.cuda())
    assert torch.equal(got, want)
    del k, v


def test_empty_batches_and_tables():
    q, k, v, table, lengths = (x.cuda() for x in cache([20, 5], 4, 2, 64, 16))
    out, lse = cs.paged_attention(q[:0], k, v, table[:0], lengths[:0],
                                  return_lse=True)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    out, lse = cs.paged_attention(q, k, v, table[:, :0].contiguous(),
                                  torch.zeros_like(lengths), return_lse=True)
    assert (out == 0).all() and (lse == -math.inf).all()
    assert cs.get_error() == set()


def test_nan_scores_are_reported():
    q, k, v, table, lengths = cache([300, 20], 4, 2, 64, 16)
    q[0, 1, 3] = math.nan
    out = cs.paged_attention(*(x.cuda() for x in (q, k, v, table, lengths)))
    assert out[0, 1].isnan().all()
    assert out[0, [0, 2, 3]].isfinite().all() and out[1].isfinite().all()
    assert cs.get_error() == {"NAN_INPUT"}


def test_sharp_scores():
    for dtype in (torch.bfloat16, torch.float16):
        q, k, v, table, lengths = cache([3000, 70], 4, 2, 64, 16, dtype=dtype)
        # Scores to about 200, growing with the position, so that the largest
        # weight is at the end and the first are far below its last bit.
        for b, n in enumerate(lengths.tolist()):
            j = torch.arange(n)
            rows = table[b, j // 16].long()
            ramp = (j / n * 4)[:, None, None]
            k[rows, j % 16] = (k[rows, j % 16].abs() * ramp).to(dtype)
        check((q.abs(), k, v, table, lengths), scale=1.0)


def test_refusals():
    q, k, v, table, lengths = (x.cuda() for x in cache([20, 5], 4, 2, 64, 16))

    def bad(error, *args, **kw):
        with pytest.raises(error):
            cs.paged_attention(*args, **kw)

    bad(TypeError, q.float(), k.float(), v.float(), table, lengths)
    bad(TypeError, q, k.half(), v.half(), table, lengths)
    bad(ValueError, q[0], k, v, table, lengths)
    bad(ValueError, q, k[0], v[0], table, lengths)
    bad(ValueError, q, k, v[:, :8], table, lengths)
    bad(ValueError, q[:, :3], k, v, table, lengths)
    bad(ValueError, q[..., :56], k, v, table, lengths)
    bad(ValueError, q, k, v, table.long(), lengths)
    bad(ValueError, q, k, v, table, lengths.long())
    bad(ValueError, q, k, v, table[:1], lengths)
    bad(ValueError, q, k, v, table, lengths[:1])
    bad(ValueError, q, k, v, table.cpu(), lengths)
    bad(ValueError, q, k, v, table[:1].expand(2, -1), lengths)
    bad(ValueError, q, k, v, table, lengths, scale=0.0)
    bad(ValueError, q, k, v, table, lengths, out=q[:1])
    bad(cs.CsError, q, k, v, table, lengths, out=q)


def test_streams_and_graphs():
    """Captured once, replayed while the lengths grow; two graphs at once."""
    q, k, v, table, lengths = cache([400, 90, 700], 8, 2, 128, 16)
    dev = [x.cuda() for x in (q, k, v, table, lengths)]
    want = {}
    for cut in (0, 1, 17, 89):
        n = lengths - cut
        want[cut] = cs.paged_attention(*dev[:4], n.cuda(), return_lse=True)
    graphs, results = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            results.append(cs.paged_attention(*dev, return_lse=True))
        graphs.append(graph)
    side = torch.cuda.Stream()
    for cut in (89, 17, 1, 0):
        dev[4].copy_(lengths - cut)
        side.wait_stream(torch.cuda.current_stream())
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
        torch.cuda.synchronize()
        for out, lse in results:
            assert torch.equal(out, want[cut][0])
            assert torch.equal(lse, want[cut][1])
    with torch.cuda.stream(side):
        out = cs.paged_attention(*dev)
    side.synchronize()
    assert torch.equal(out, want[0][0])


def test_repeated_calls_agree():
    args = [x.cuda() for x in cache([2000, 90, 700, 0, 1300], 16, 4, 128, 16)]
    first = cs.paged_attention(*args, return_lse=True)
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(200):
        for a, b in zip(cs.paged_attention(*args, return_lse=True), first):
            differ += (a.view(torch.int16) != b.view(torch.int16)).sum()
    assert int(differ) == 0 and cs.get_error() == set()


@pytest.mark.parametrize("D", [64, 128])
def test_prompt_then_tokens(D):
    """As a server uses them together: the prompt through fused_attention,
    its keys and values into pages, then token after token through
    paged_attention, each equal to fused_attention over all so far."""
    gen = torch.Generator().manual_seed(5)
    B, H, Hk, page, steps = 2, 8, 2, 16, 5
    prompts = [37, 130]
    most = max(prompts) + steps

    def heads(h):
        return torch.randn(B, h, most, D, generator=gen).bfloat16().cuda()

    q, k, v = heads(H), heads(Hk), heads(Hk)
    pages = -(-most // page)
    order = torch.randperm(B * pages, generator=gen).to(torch.int32).cuda()
    table = order.view(B, pages)
    cache_k = torch.zeros(B * pages, page, Hk, D, dtype=torch.bfloat16,
                          device="cuda")
    cache_v = torch.zeros_like(cache_k)

    def write(b, start, stop):
        j = torch.arange(start, stop, device="cuda")
        rows = table[b, j // page].long()
        cache_k[rows, j % page] = k[b, :, start:stop].transpose(0, 1)
        cache_v[rows, j % page] = v[b, :, start:stop].transpose(0, 1)

    n = max(prompts)
    mask = (torch.arange(n, device="cuda")[None]
            < torch.tensor(prompts, device="cuda")[:, None])
    cs.fused_attention(q[:, :, :n], k[:, :, :n], v[:, :, :n], mask, True)
    for b in range(B):
        write(b, 0, prompts[b])
    lengths = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    for step in range(steps):
        for b in range(B):
            write(b, prompts[b] + step, prompts[b] + step + 1)
        lengths += 1
        now = [p + step for p in prompts]
        token = torch.stack([q[b, :, now[b]] for b in range(B)])
        out = cs.paged_attention(token, cache_k, cache_v, table, lengths)
        for b in range(B):
            m = now[b] + 1
            whole = cs.fused_attention(q[b:b + 1, :, :m], k[b:b + 1, :, :m],
                                       v[b:b + 1, :, :m], causal=True)
            last = whole[0, :, -1].float()
            # One rounding of each result, and the fused weights' of bf16,
            # 2^-8 of each, over values of a few units.
            p = torch.softmax(
                (token[b].float().view(Hk, H // Hk, D)
                 @ k[b, :, :m].float().mT) / D ** 0.5, -1)
            c = torch.sqrt((p ** 2) @ (v[b, :, :m].float() ** 2)).view(H, D)
            tol = 2.0 ** -7 * last.abs() + 7 * 2.0 ** -8 * c + 1e-4
            assert ((out[b].float() - last).abs() <= tol).all()
    assert cs.get_error() == set()


def test_many_longer_sequences():
    """As test_many_sequences, past the length up to which large batches are
    not cut: the dealing walks over the lengths in several rounds."""
    lengths = [(53 * b) % 700 for b in range(300)]
    check(cache(lengths, 2, 1, 64, 16))


@pytest.mark.parametrize("D,page", [(64, 1), (128, 7), (80, 100), (256, 64)])
def test_page_sizes_off_the_step(D, page):
    """Pages that divide no step of 64 tokens, one token a page, pages longer
    than a step: entry and slot are walked without a division."""
    check(cache([700, 1, 64, 65, 333], 4, 2, D, page))
    check(cache([150, 0, 99], 4, 4, D, page))
