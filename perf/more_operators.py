"""The operators around a paged key-value cache that serve several new tokens a
sequence, as measured: pages and slots for new tokens, the write of their keys
and values, and the attention of a tree of drafted tokens over the cache.

``run`` is one pass of an operator; where ``own`` is false it is computed with
elementary torch operations, in fp32, rounded once at the end.
"""
import math
import random

import torch

own = False

BF16, FP16 = "bfloat16", "float16"


def listed():
    return [
        # A decode step of a serving batch: one token each, a page now and then.
        _extend("extend_step_32", 32, 1, 4096, 16),
        # A step of speculative decoding: trees of up to 61 drafted tokens, and
        # a pool that runs out of pages for the last sequences.
        _extend("extend_drafts_256", 256, 61, 4096, 64, ragged=True,
                short=True),
        # A large batch of prompts is admitted: every slot of the step.
        _extend("extend_prompts_512x4096", 512, 4096, 4096, 16, ragged=True),
        # One user's drafted tokens: the latency of a call.
        _write("write_short", 1, 8, 8, 77, 64, 16),
        # Prompts of a batch, padded on the right, the keys and values slices
        # of one packed projection.
        _write("write_prompts_32x4096", 32, 4096, 8, 4096, 128, 16,
               ragged=True, packed=True),
        # fp16, every head its own keys, odd head size, page size and lengths.
        _write("write_odd_fp16", 7, 333, 12, 1531, 80, 48, dtype=FP16,
               ragged=True),
        # One user, a short history, a small tree: the latency of a step.
        _tree("tree_short", 1, 8, 8, 77, 64, 16),
        # A serving batch with histories of every length, trees of 16.
        _tree("tree_batch_32x4096", 32, 16, 32, 4096, 128, 16, Hk=8,
              ragged=True),
        # One user with a very long history and a tree of 32.
        _tree("tree_long_131072", 1, 32, 32, 131072, 128, 64, Hk=8),
        # Wide trees: 64 drafted tokens of 4 heads to a key head.
        _tree("tree_wide_8x8192", 8, 64, 32, 8192, 128, 64, Hk=8),
        # A prompt's next chunk over what is cached: no tree, each token sees
        # the ones before it.
        _tree("chunk_2x512_of_8192", 2, 512, 32, 8192, 128, 64, Hk=8,
              tree=False),
        # fp16, every head its own keys, odd head size, page size and lengths,
        # trees of up to 13.
        _tree("tree_odd_fp16", 7, 13, 12, 1531, 80, 48, dtype=FP16,
              ragged=True),
    ]


def _extend(name, B, T, longest, page, ragged=False, short=False):
    return {"name": name, "op": "extend", "B": B, "T": T, "longest": longest,
            "page": page, "ragged": ragged, "short": short}


def _write(name, B, T, Hk, longest, D, page, dtype=BF16, ragged=False,
           packed=False):
    return {"name": name, "op": "write", "B": B, "T": T, "Hk": Hk,
            "longest": longest, "D": D, "page": page, "dtype": dtype,
            "ragged": ragged, "packed": packed}


def _tree(name, B, T, H, longest, D, page, Hk=None, dtype=BF16, ragged=False,
          tree=True):
    return {"name": name, "op": "tree", "B": B, "T": T, "H": H,
            "Hk": Hk or H, "longest": longest, "D": D, "page": page,
            "dtype": dtype, "ragged": ragged, "tree": tree}


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["extend", "write", "tree", "tree"])
    page = rng.choice([1, 16, 64, 128, rng.randint(2, 256)])
    dtype = rng.choice([BF16, FP16])
    ragged = rng.random() < 0.7
    Hk = rng.choice([1, 2, 3, 4, 8])
    D = rng.choice([64, 128, 128, 8 * rng.randint(2, 32)])
    if op == "extend":
        B = _log_uniform(rng, 1, 1024)
        T = _log_uniform(rng, 1, min(4096, 512 * 4096 // B))
        c = _extend("", B, T, max(T, _log_uniform(rng, 1, 4096)), page,
                    ragged, rng.random() < 0.3)
    elif op == "write":
        B = _log_uniform(rng, 1, 64)
        # At most the tokens of the largest listed write.
        T = _log_uniform(rng, 1, min(4096, 32 * 4096 * 8 * 128
                                     // (B * Hk * max(D, 128))))
        c = _write("", B, T, Hk, max(T, _log_uniform(rng, 1, 4096)), D, page,
                   dtype, ragged, rng.random() < 0.5)
    else:
        H = Hk * rng.choice([1, 2, 4, 5, 8, 16])
        tree = rng.random() < 0.7
        B = _log_uniform(rng, 1, 64)
        # At most the scores of the largest listed pass, and its tokens.
        most = 2 * 32 * 512 * 8192
        T = _log_uniform(rng, 1, min(128 if tree else 512,
                                     math.isqrt(most // (B * H))))
        top = min(131072, most // (B * H * T),
                  131072 * 8 * 128 // (B * Hk * max(D, 128)))
        c = _tree("", B, T, H, max(T, _log_uniform(rng, 1, max(1, top))), D,
                  page, Hk, dtype, ragged, tree)
    del c["name"]
    return c


def _counts(case):
    """New tokens and tokens after the step of every sequence: the longest
    first, the others spread over their logarithm."""
    top, T = case["longest"], case["T"]
    if not case["ragged"]:
        return [T] * case["B"], [top] * case["B"]
    r = random.Random(1000 * case["B"] + top + T)
    new = [T] + [_log_uniform(r, max(1, T // 16), T)
                 for _ in range(case["B"] - 1)]
    after = [top] + [_log_uniform(r, max(1, top // 16), top)
                     for _ in range(case["B"] - 1)]
    return new, [max(a, n) for a, n in zip(after, new)]


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _tensor(gen, shape, dtype):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    return x.to(dtype)


def _table(gen, after, page, spare=0):
    """A page table of sequences of these lengths, whose pages are handed out
    in no order, as by a server's free list, with `spare` pages besides; the
    pages in all; the spare ones."""
    per = [-(-n // page) for n in after]
    total = sum(per) + spare
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    width = max(max(per), 1)
    kept = (torch.arange(width, device="cuda")[None, :]
            < _int32(per)[:, None])
    table = torch.zeros((len(per), width), dtype=torch.int32, device="cuda")
    table[kept] = order[:sum(per)]
    return table, total, order[sum(per):]


def _tree_mask(gen, B, T):
    """Drafted token i attends itself and its ancestors: trees whose nodes
    hang on any node before them."""
    reach = torch.eye(T, dtype=torch.bool, device="cuda").repeat(B, 1, 1)
    at = torch.rand((B, T), generator=gen, device="cuda")
    every = torch.arange(B, device="cuda")
    for i in range(1, T):
        parent = (at[:, i] * (i + 1)).long() - 1      # -1: a root
        up = reach[every, parent.clamp(min=0)]
        reach[:, i] |= up & (parent >= 0)[:, None]
    return reach


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, B, T, page = case["op"], case["B"], case["T"], case["page"]
    new, after = _counts(case)
    state = {"op": op, "page": page, "T": T}
    if op == "extend":
        used = 3   # pages that earlier steps took from the list's front
        full, _, spent = _table(gen, after, page, spare=used)
        before = [a - n for a, n in zip(after, new)]
        have = _int32([-(-n // page) for n in before])[:, None]
        want = _int32([-(-n // page) for n in after])[:, None]
        j = torch.arange(full.shape[1], device="cuda")[None, :]
        fresh = full[(j >= have) & (j < want)]
        fresh = fresh[torch.randperm(len(fresh), generator=gen, device="cuda")]
        if case["short"]:
            fresh = fresh[:len(fresh) * 3 // 4]
        state.update(page_table=full.masked_fill(j >= have, 0),
                     held=have[:, 0].contiguous(), lengths=_int32(before),
                     new_lengths=_int32(new),
                     free_pages=torch.cat([spent, fresh]),
                     cursor=_int32([used]))
        return state
    dtype = getattr(torch, case["dtype"])
    Hk, D = case["Hk"], case["D"]
    table, total, _ = _table(gen, after, page, spare=2)
    shape = (total, page, Hk, D)
    state.update(key_pages=_tensor(gen, shape, dtype),
                 value_pages=_tensor(gen, shape, dtype))
    lengths, count = _int32(after), _int32(new)
    if op == "write":
        i = torch.arange(T, device="cuda")[None, :]
        at = (lengths - count).long()[:, None] + i
        slots = table.long().gather(
            1, (at // page).clamp(max=table.shape[1] - 1)) * page + at % page
        state["slots"] = torch.where(i < count[:, None], slots, -1)
        if case["packed"]:
            both = _tensor(gen, (B, T, 2 * Hk, D), dtype)
            state.update(keys=both[:, :, :Hk], values=both[:, :, Hk:])
        else:
            state.update(keys=_tensor(gen, (B, T, Hk, D), dtype),
                         values=_tensor(gen, (B, T, Hk, D), dtype))
        return state
    state.update(query=_tensor(gen, (B, T, case["H"], D), dtype),
                 page_table=table, lengths=lengths,
                 new_lengths=count if case["ragged"] else None,
                 mask=_tree_mask(gen, B, T) if case["tree"] else None,
                 scale=1.0 / math.sqrt(D))
    return state


def _extend_plain(state):
    page, free = state["page"], state["free_pages"]
    table, held = state["page_table"], state["held"].long()
    before, new = state["lengths"].long(), state["new_lengths"].long()
    cursor = state["cursor"].long()
    left = free.shape[0] - cursor
    need = ((before + new + page - 1) // page - held).clamp(min=0)
    first = torch.cumsum(need, 0) - need
    got = torch.minimum(need, (left - first).clamp(min=0))
    have = held + got
    totals = torch.minimum(before + new, have * page)
    j = torch.arange(table.shape[1], device="cuda")[None, :]
    entry = (cursor + first - held)[:, None] + j
    taken = free[entry.clamp(0, free.shape[0] - 1)]
    table.copy_(torch.where((j >= held[:, None]) & (j < have[:, None]), taken,
                            table))
    i = torch.arange(state["T"], device="cuda")[None, :]
    at = before[:, None] + i
    number = table.long().gather(1, (at // page).clamp(max=table.shape[1] - 1))
    slots = torch.where(i < (totals - before)[:, None],
                        number * page + at % page, -1)
    after = cursor + torch.minimum(left, need.sum())
    return (table, slots, totals.to(torch.int32), have.to(torch.int32),
            after.to(torch.int32))


def _write_plain(state):
    keys, values = state["keys"], state["values"]
    pages, page, Hk, D = state["key_pages"].shape
    slots = state["slots"].reshape(-1)
    # A token without a slot writes what the first one writes.
    source = torch.arange(slots.shape[0], device="cuda")
    source = torch.where(slots >= 0, source, 0)
    slots = slots[source]
    for x, into in ((keys, "key_pages"), (values, "value_pages")):
        state[into].view(pages * page, Hk, D)[slots] = (
            x.reshape(-1, Hk, D)[source])
    return state["key_pages"], state["value_pages"]


def _tree_plain(state):
    q, table = state["query"], state["page_table"].long()
    B, T, H, D = q.shape
    page, Hk = state["key_pages"].shape[1:3]
    G, n = H // Hk, table.shape[1] * page
    k, v = (state[name][table].reshape(B, n, Hk, D).transpose(1, 2).float()
            for name in ("key_pages", "value_pages"))
    rows = q.float().reshape(B, T, Hk, G, D).transpose(1, 2).reshape(
        B, Hk, T * G, D)
    s = (torch.matmul(rows, k.transpose(-1, -2)) * state["scale"]).view(
        B, Hk, T, G, n)
    after = state["lengths"].long()
    new = state["new_lengths"]
    new = torch.full_like(after, T) if new is None else new.long()
    i = torch.arange(T, device="cuda")
    # Position j is drafted token j - (length - new) where that is not negative.
    draft = torch.arange(n, device="cuda")[None, :] - (after - new)[:, None]
    if state["mask"] is None:
        sees = draft[:, None, :] <= i[None, :, None]
    else:
        sees = (draft < 0)[:, None, :] | state["mask"].gather(
            2, draft.clamp(0, T - 1)[:, None, :].expand(B, T, n))
    sees = sees & (draft < new[:, None])[:, None, :]
    sees = sees & (i[None, :] < new[:, None])[:, :, None]
    s = s.masked_fill(~sees[:, None, :, None, :], -math.inf)
    m = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    total = e.sum(-1, keepdim=True)
    out = torch.matmul(e.view(B, Hk, T * G, n), v).view(B, Hk, T, G, D)
    out = out / torch.where(total == 0, 1.0, total)
    lse = (m + torch.log(total)).squeeze(-1)
    return (out.transpose(1, 2).reshape(B, T, H, D).to(q.dtype),
            lse.transpose(1, 2).reshape(B, T, H))


def run(state):
    if own:
        import entropy_bounded_softmax_gb300 as cs
        if state["op"] == "extend":
            return (state["page_table"], *cs.paged_extend(
                state["page_table"], state["lengths"], state["new_lengths"],
                state["free_pages"], state["page"], state["T"],
                held=state["held"], cursor=state["cursor"]))
        if state["op"] == "write":
            cs.paged_write(state["keys"], state["values"], state["slots"],
                           state["key_pages"], state["value_pages"])
            return state["key_pages"], state["value_pages"]
        return cs.paged_tree_attention(
            state["query"], state["key_pages"], state["value_pages"],
            state["page_table"], state["lengths"], mask=state["mask"],
            new_lengths=state["new_lengths"], scale=state["scale"],
            return_lse=True)
    if state["op"] == "extend":
        return _extend_plain(state)
    return _write_plain(state) if state["op"] == "write" else _tree_plain(state)


def work(case):
    B, T, page = case["B"], case["T"], case["page"]
    new, after = _counts(case)
    if case["op"] == "extend":
        # Counts read and written, pages taken, one slot for every place.
        taken = sum(-(-a // page) + ((n - a) // page)
                    for n, a in zip(new, after))
        return {"bytes": 20 * B + 8 * taken + 8 * B * T, "flops": 0}
    Hk, D = case["Hk"], case["D"]
    if case["op"] == "write":
        return {"bytes": 8 * sum(new) * Hk * D + 8 * B * T, "flops": 0}
    H = case["H"]
    # Every cached key and value once, the queries, out and its sums.
    tokens, rows = sum(after), B * T * H
    pairs = sum(n * (a - n) + (n * (n + 1) // 2) for n, a in zip(new, after))
    return {"bytes": 4 * tokens * Hk * D + 4 * rows * D + 4 * rows
            + 4 * (tokens // page) + (B * T * T if case["tree"] else 0),
            "flops": 4 * D * H * pairs}


def exact(case, seed):
    """The definition in 64 bits, one sequence at a time."""
    state = prepare(case, seed)
    return {"extend": _exact_extend, "write": _exact_write,
            "tree": _exact_tree}[case["op"]](case, state)


def _exact_extend(case, state):
    """Page after page, as a server's loop on the host hands them out."""
    page, table = case["page"], state["page_table"].tolist()
    free, at = state["free_pages"].tolist(), state["cursor"].item()
    slots, totals, held = [], [], []
    for row, n, more, h in zip(table, state["lengths"].tolist(),
                               state["new_lengths"].tolist(),
                               state["held"].tolist()):
        while h * page < n + more and at < len(free):
            row[h] = free[at]
            h, at = h + 1, at + 1
        total = min(n + more, h * page)
        slots.append([row[x // page] * page + x % page
                      for x in range(n, total)]
                     + [-1] * (case["T"] - (total - n)))
        totals.append(total)
        held.append(h)
    return (_int32(table), torch.tensor(slots, device="cuda"), _int32(totals),
            _int32(held), _int32([at]))


def _exact_write(case, state):
    out = []
    for name in ("key", "value"):
        pages = state[name + "_pages"]
        flat = pages.view(-1, *pages.shape[2:])
        for b in range(case["B"]):
            n = int((state["slots"][b] >= 0).sum())
            flat.index_copy_(0, state["slots"][b, :n],
                             state[name + "s"][b, :n].contiguous())
        out.append(pages)
    return tuple(out)


def _exact_tree(case, state):
    B, T, H, Hk, D = (case[x] for x in ("B", "T", "H", "Hk", "D"))
    G, page = H // Hk, case["page"]
    out = torch.zeros(B, T, H, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, T, H), -math.inf, dtype=torch.float64, device="cuda")
    for b, (new, n) in enumerate(zip(*_counts(case))):
        j = torch.arange(n, device="cuda")
        row = state["page_table"][b, j // page].long()
        drafted = torch.ones(new, new, dtype=torch.bool, device="cuda").tril()
        if state["mask"] is not None:
            drafted = state["mask"][b, :new, :new]
        removed = torch.zeros(new, n, dtype=torch.bool, device="cuda")
        removed[:, n - new:] = ~drafted
        for g in range(Hk):
            k = state["key_pages"][row, j % page, g].double()
            v = state["value_pages"][row, j % page, g].double()
            for h in range(g * G, (g + 1) * G):
                z = state["query"][b, :new, h].double() @ k.T * state["scale"]
                z[removed] = -math.inf
                lse[b, :new, h] = torch.logsumexp(z, 1)
                out[b, :new, h] = torch.softmax(z, 1) @ v
    return out, lse
