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
