"""Paged caches and, in 64 bits, what the operators around them have to give:
the page-by-page hand-out of paged_extend, and the attention of several new
tokens.  Shared by the GPU tests and pinned on the CPU.

Allowances of the attention, per element: half a step of the result's type;
half a step of the cache's for each weight; a score's dot product errs by
(D + 8) 2^-23 of the sum of its terms' magnitudes, 2^x by 2^-21; the sums of
n <= 6000 terms by 2^-17 of the sum of magnitudes (each step rounds by 2^-23,
mostly cancelling).  In fp16, whose steps are never below 2^-24: results err by
up to 2^-25, and weights, which carry a factor 2^8 or more and have a sum of at
least as much, by up to 2^-33 of that sum each."""
import math

import torch

F32 = 2.0 ** -23


def cache(lengths, T, H, Hk, D, page, dtype=torch.bfloat16, seed=0, extra=3):
    """Query, pages, table and lengths: pages in no order, with spare pages and
    spare table entries (both hold what a reader must not use)."""
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
    q = torch.randn(len(lengths), T, H, D, generator=gen).to(dtype)
    return q, k, v, table, torch.tensor(lengths, dtype=torch.int32)


def tree_mask(B, T, seed=0, empty=False):
    """Random trees: each node hangs on any node before it, or is a root; with
    `empty`, some rows lose even themselves."""
    gen = torch.Generator().manual_seed(1000 + seed)
    reach = torch.zeros(B, T, T, dtype=torch.bool)
    for b in range(B):
        for i in range(T):
            reach[b, i, i] = True
            parent = int(torch.randint(-1, max(i, 1), (1,), generator=gen))
            if 0 <= parent < i:
                reach[b, i] |= reach[b, parent]
        if empty:
            reach[b, torch.rand(T, generator=gen) < 0.3] = False
    return reach


def kept(n, new, T, mask):
    """Which of n tokens the T new tokens' rows attend; mask [T, T] or None."""
    j = torch.arange(n)[None, :] - (n - new)     # of the new tokens, or negative
    i = torch.arange(T)[:, None]
    if mask is None:
        sees = j <= i
    else:
        sees = (j < 0) | mask[:, (j[0]).clamp(0, max(T - 1, 0))]
    return sees & (i < new)


def definition(q, k, v, table, lengths, mask=None, new_lengths=None,
               scale=None):
    """out, its allowance, lse and its allowance."""
    B, T, H, D = q.shape
    page, Hk = k.shape[1:3]
    scale = D ** -0.5 if scale is None else scale
    half = torch.finfo(q.dtype).eps / 2
    out = torch.zeros(B, T, H, D, dtype=torch.float64)
    tol = torch.full_like(out, 1e-37)
    lse = torch.full((B, T, H), -math.inf, dtype=torch.float64)
    tol_lse = torch.zeros(B, T, H, dtype=torch.float64)
    for b, n in enumerate(lengths.tolist()):
        new = T if new_lengths is None else int(new_lengths[b])
        if n == 0 or new == 0:
            continue
        m = mask if mask is None or mask.dim() == 2 else mask[b]
        sees = kept(n, new, T, m)
        j = torch.arange(n)
        rows = table[b, j // page].long()
        for h in range(H):
            kk = k[rows, j % page, h * Hk // H].double()
            vv = v[rows, j % page, h * Hk // H].double()
            qq = q[b, :, h].double()
            s = (qq @ kk.T * scale).masked_fill(~sees, -math.inf)
            some = sees.any(1)
            lse[b, some, h] = torch.logsumexp(s[some], 1)
            p = torch.exp(s[some] - lse[b, some, h][:, None])
            out[b, some, h] = p @ vv
            es = (2 * (D + 8) * F32 * scale
                  * (qq[some].abs() @ kk.abs().T).amax(1)
                  + 4 * F32 * s[some].masked_fill(~sees[some], 0).abs().amax(1)
                  + 2.0 ** -21 + 2.0 ** -17)[:, None]
            tol[b, some, h] += (half * out[b, some, h].abs()
                                + (2 * es + half) * (p @ vv.abs()))
            if q.dtype == torch.float16:
                tol[b, some, h] += (2.0 ** -25 + 2.0 ** -33 *
                                    (sees[some].double() @ vv.abs()))
            tol_lse[b, some, h] = es[:, 0] + 4 * F32 * lse[b, some, h].abs()
    return out, tol, lse, tol_lse


def extend(table, lengths, new_lengths, free, page, max_new, held=None,
           cursor=0):
    """paged_extend by a loop over sequences and pages; lists of lists."""
    slots, totals, have = [], [], []
    table = [list(r) for r in table]
    for b, (n, more) in enumerate(zip(lengths, new_lengths)):
        h = -(-n // page) if held is None else held[b]
        while h * page < n + more and cursor < len(free):
            table[b][h] = free[cursor]
            h, cursor = h + 1, cursor + 1
        total = max(n, min(n + more, h * page))
        slots.append([table[b][x // page] * page + x % page
                      for x in range(n, total)]
                     + [-1] * (max_new - (total - n)))
        totals.append(total)
        have.append(h)
    return table, slots, totals, have, cursor
