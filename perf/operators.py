"""The attention operators of language models, as measured: fused attention, its
backward pass, and attention of one new token over a paged key-value cache.

``run`` is one pass of an operator; where ``own`` is false it is computed with
elementary torch operations in fp32, rounded once at the end.
"""
import math
import random

import torch

own = False

BF16, FP16 = "bfloat16", "float16"


def listed():
    return [
        # One short prompt of a small model: launch and latency.
        _attn("forward_short", "forward", 1, 8, 2, 77, 77, 64, causal=True),
        # The framework's own attention shape: 32 sequences, 8 heads, 512 keys,
        # an encoder's batch padded on the right.
        _attn("forward_32x8x512_padded", "forward", 32, 8, 8, 512, 512, 64,
              mask="right"),
        # Training of a causal model at the framework's long sequence.
        _attn("forward_2x8x4096_causal", "forward", 2, 8, 8, 4096, 4096, 128,
              causal=True, layout="bshd"),
        # Ragged prompts continued over a cached prefix: odd lengths, more keys
        # than queries, left padding, a head size between the usual ones.
        _attn("forward_ragged", "forward", 3, 12, 4, 1000, 1531, 80,
              causal=True, mask="left", layout="bshd"),
        # The same four for the gradients.
        _attn("backward_short", "backward", 1, 8, 2, 77, 77, 64, causal=True),
        _attn("backward_32x8x512_padded", "backward", 32, 8, 8, 512, 512, 64,
              mask="right"),
        _attn("backward_2x8x4096_causal", "backward", 2, 8, 8, 4096, 4096, 128,
              causal=True, layout="bshd"),
        _attn("backward_ragged", "backward", 3, 12, 4, 1000, 1531, 80,
              causal=True, mask="left", layout="bshd"),
        # One user, a short history: the latency of a decode step.
        _paged("paged_short", 1, 8, 8, 77, 64, 16),
        # A serving batch of users with histories of every length.
        _paged("paged_batch_32x4096", 32, 32, 8, 4096, 128, 16, ragged=True),
        # One user with a very long history: the cache's length is split.
        _paged("paged_long_131072", 1, 32, 8, 131072, 128, 64),
        # fp16, every head its own keys, odd head size, page size and lengths.
        _paged("paged_odd_fp16", 7, 12, 12, 1531, 80, 48, dtype=FP16,
               ragged=True),
    ]


def _attn(name, op, B, H, Hk, Sq, Sk, D, causal=False, mask="none",
          layout="bhsd"):
    return {"name": name, "op": op, "B": B, "H": H, "Hk": Hk, "Sq": Sq,
            "Sk": Sk, "D": D, "causal": causal, "mask": mask,
            "layout": layout}


def _paged(name, B, H, Hk, longest, D, page, dtype=BF16, ragged=False):
    return {"name": name, "op": "paged", "B": B, "H": H, "Hk": Hk,
            "longest": longest, "D": D, "page": page, "dtype": dtype,
            "ragged": ragged}


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["forward", "backward", "paged"])
    Hk = rng.choice([1, 2, 3, 4, 8])
    if op == "paged":
        H = Hk * rng.choice([1, 2, 4, 5, 8, 16])
        D = rng.choice([64, 128, 128, 8 * rng.randint(2, 32)])
        B = _log_uniform(rng, 1, 64)
        # At most the tokens of the longest listed history.
        longest = _log_uniform(rng, 1, min(131072, 131072 * 8 * 128
                                           // (B * Hk * max(D, 128))))
        c = _paged("", B, H, Hk, longest, D, rng.choice([1, 16, 64, 128,
                                                         rng.randint(2, 256)]),
                   rng.choice([BF16, FP16]), rng.random() < 0.7)
    else:
        H = Hk * rng.choice([1, 1, 2, 3, 4, 8])
        D = rng.choice([64, 128, 8 * rng.randint(2, 16)])
        B = _log_uniform(rng, 1, 32)
        # At most the pairs of the largest listed case, on a full square.
        top = min(4096, math.isqrt(2 * 8 * 4096 * 4096 // 2 // (B * H)))
        # A query that keeps a single key has no gradient but rounding, so
        # the gradients' range starts at a few keys.
        Sk = _log_uniform(rng, 16 if op == "backward" else 1, top)
        Sq = Sk if rng.random() < 0.5 else _log_uniform(rng, 1, top)
        c = _attn("", op, B, H, Hk, Sq, Sk, D, rng.random() < 0.6,
                  rng.choice(["none", "none", "right", "left", "holes"]),
                  rng.choice(["bhsd", "bshd"]))
    del c["name"]
    return c


def _kept_lengths(case):
    """Kept keys of each sequence of a padded batch: from all of them down to
    a quarter, evenly."""
    B, Sk = case["B"], case["Sk"]
    return [max(1, Sk - (3 * Sk * b) // (4 * max(1, B - 1)))
            for b in range(B)]


def _cache_lengths(case):
    """Cache lengths of a serving batch: the longest first, the others spread
    over their logarithm."""
    top = case["longest"]
    if not case["ragged"]:
        return [top] * case["B"]
    r = random.Random(1000 * case["B"] + top)
    return [top] + [_log_uniform(r, max(1, top // 16), top)
                    for _ in range(case["B"] - 1)]


def _tensor(gen, shape, dtype):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    return x.to(dtype)


def _heads(gen, case, heads, length):
    """A [B, heads, length, D] tensor, stored in the case's order."""
    if case["layout"] == "bshd":
        return _tensor(gen, (case["B"], length, heads, case["D"]),
                       torch.bfloat16).transpose(1, 2)
    return _tensor(gen, (case["B"], heads, length, case["D"]), torch.bfloat16)


def _key_mask(gen, case):
    if case["mask"] == "none":
        return None
    B, Sk = case["B"], case["Sk"]
    if case["mask"] == "holes":
        return torch.rand((B, Sk), generator=gen, device="cuda") < 0.8
    kept = torch.tensor(_kept_lengths(case), device="cuda")[:, None]
    j = torch.arange(Sk, device="cuda")[None, :]
    return j < kept if case["mask"] == "right" else j >= Sk - kept


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    state = {"op": case["op"], "scale": 1.0 / math.sqrt(case["D"])}
    if case["op"] == "paged":
        dtype = getattr(torch, case["dtype"])
        lengths = _cache_lengths(case)
        per = [-(-n // case["page"]) for n in lengths]
        total = sum(per)
        shape = (total, case["page"], case["Hk"], case["D"])
        # Pages are handed out in no order, as by a server's free list.
        order = torch.randperm(total, generator=gen, device="cuda")
        table = torch.zeros((case["B"], max(per)), dtype=torch.int32,
                            device="cuda")
        at = 0
        for b, n in enumerate(per):
            table[b, :n] = order[at:at + n].to(torch.int32)
            at += n
        state.update(
            query=_tensor(gen, (case["B"], case["H"], case["D"]), dtype),
            key_pages=_tensor(gen, shape, dtype),
            value_pages=_tensor(gen, shape, dtype), page_table=table,
            lengths=torch.tensor(lengths, dtype=torch.int32, device="cuda"))
        return state
    state.update(query=_heads(gen, case, case["H"], case["Sq"]),
                 keys=_heads(gen, case, case["Hk"], case["Sk"]),
                 values=_heads(gen, case, case["Hk"], case["Sk"]),
                 mask=_key_mask(gen, case), causal=case["causal"])
    if case["op"] == "backward":
        # What the forward pass left, and the gradient that comes in.
        state["out"], state["lse"] = _forward(state)
        state["grad"] = _heads(gen, case, case["H"], case["Sq"])
    return state


def _kept(state, Sq, Sk):
    """Kept (query, key) pairs, [B or 1, 1, 1, Sq, Sk], or None for all."""
    kept = None
    if state["causal"]:
        i = torch.arange(Sq, device="cuda")[:, None]
        j = torch.arange(Sk, device="cuda")[None, :]
        kept = (j <= i + (Sk - Sq))[None, None, None]
    if state["mask"] is not None:
        m = state["mask"][:, None, None, None, :]
        kept = m if kept is None else kept & m
    return kept


def _split(x, Hk):
    """[B, H, S, D] as fp32 [B, Hk, H / Hk, S, D]."""
    B, H, S, D = x.shape
    return x.float().reshape(B, Hk, H // Hk, S, D)


def _scores(state, q, k):
    s = torch.matmul(q, k.transpose(-1, -2)) * state["scale"]
    kept = _kept(state, q.shape[-2], k.shape[-2])
    return s if kept is None else s.masked_fill(~kept, -math.inf)


def _forward(state):
    Hk = state["keys"].shape[1]
    q, k, v = (_split(state[n], Hk) for n in ("query", "keys", "values"))
    s = _scores(state, q, k)
    m = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    total = e.sum(-1, keepdim=True)
    out = torch.matmul(e, v) / torch.where(total == 0, 1.0, total)
    lse = (m + torch.log(total)).squeeze(-1)
    B, H, Sq, D = state["query"].shape
    out = out.reshape(B, H, Sq, D).to(torch.bfloat16)
    if state["query"].stride(1) < state["query"].stride(2):
        # out is stored in the query's order
        out = out.transpose(1, 2).contiguous().transpose(1, 2)
    return out, lse.reshape(B, H, Sq)


def _backward(state):
    Hk = state["keys"].shape[1]
    q, k, v, o, g = (_split(state[n], Hk)
                     for n in ("query", "keys", "values", "out", "grad"))
    B, H, Sq, D = state["query"].shape
    lse = state["lse"].reshape(B, Hk, H // Hk, Sq, 1)
    p = torch.exp(_scores(state, q, k)
                  - torch.where(lse == -math.inf, math.inf, lse))
    dv = torch.matmul(p.transpose(-1, -2), g).sum(2)
    ds = p * (torch.matmul(g, v.transpose(-1, -2))
              - (g * o).sum(-1, keepdim=True))
    dq = torch.matmul(ds, k).reshape(B, H, Sq, D) * state["scale"]
    dk = torch.matmul(ds.transpose(-1, -2), q).sum(2) * state["scale"]
    return tuple(x.to(torch.bfloat16) for x in (dq, dk, dv))


def _paged_attention(state):
    q, table = state["query"], state["page_table"].long()
    B, H, D = q.shape
    page, Hk = state["key_pages"].shape[1:3]
    n = table.shape[1] * page
    k, v = (state[name][table].reshape(B, n, Hk, D).transpose(1, 2).float()
            for name in ("key_pages", "value_pages"))
    s = torch.matmul(q.float().reshape(B, Hk, H // Hk, D),
                     k.transpose(-1, -2)) * state["scale"]
    past = (torch.arange(n, device="cuda")[None, :]
            >= state["lengths"].long()[:, None])[:, None, None, :]
    s = s.masked_fill(past, -math.inf)
    m = s.amax(-1, keepdim=True)
    e = torch.exp(s - m)
    total = e.sum(-1, keepdim=True)
    out = torch.matmul(e, v) / total
    return (out.reshape(B, H, D).to(q.dtype),
            (m + torch.log(total)).reshape(B, H))


def run(state):
    if own:
        import entropy_bounded_softmax_gb300 as cs
        if state["op"] == "paged":
            return cs.paged_attention(
                state["query"], state["key_pages"], state["value_pages"],
                state["page_table"], state["lengths"], scale=state["scale"],
                return_lse=True)
        if state["op"] == "backward":
            return cs.fused_attention_backward(
                state["query"], state["keys"], state["values"], state["out"],
                state["lse"], state["grad"], mask=state["mask"],
                causal=state["causal"], scale=state["scale"])
        return cs.fused_attention(
            state["query"], state["keys"], state["values"],
            mask=state["mask"], causal=state["causal"], scale=state["scale"],
            return_lse=True)
    if state["op"] == "paged":
        return _paged_attention(state)
    return _backward(state) if state["op"] == "backward" else _forward(state)


def _pairs(case):
    """Kept (query, key) pairs of one head, over the batch; holes count as
    kept."""
    B, Sq, Sk = case["B"], case["Sq"], case["Sk"]
    kept = _kept_lengths(case) if case["mask"] in ("right", "left") else [Sk] * B
    total = 0
    for n in kept:
        lo, hi = (Sk - n, Sk) if case["mask"] == "left" else (0, n)
        if case["causal"]:
            total += sum(max(0, min(hi, i + Sk - Sq + 1) - lo)
                         for i in range(Sq))
        else:
            total += Sq * n
    return total


def work(case):
    B, H, Hk, D = case["B"], case["H"], case["Hk"], case["D"]
    if case["op"] == "paged":
        tokens = sum(_cache_lengths(case))
        return {"bytes": 4 * tokens * Hk * D + 4 * B * H * D + 4 * B * H
                + 4 * (tokens // case["page"]),
                "flops": 4 * D * H * tokens}
    q, k = B * H * case["Sq"], B * Hk * case["Sk"]
    pairs = H * _pairs(case)
    if case["op"] == "forward":
        return {"bytes": 4 * q * D + 4 * k * D + 4 * q, "flops": 4 * D * pairs}
    # q, out and grad_output read, dq written; k, v read, dk, dv written.
    return {"bytes": 8 * q * D + 8 * k * D + 4 * q, "flops": 10 * D * pairs}


def exact(case, seed):
    """The definition in 64 bits, one sequence and one head at a time."""
    state = prepare(case, seed)
    if case["op"] == "paged":
        return _exact_paged(case, state)
    B, H, Hk = case["B"], case["H"], case["Hk"]
    Sq, Sk, D = case["Sq"], case["Sk"], case["D"]
    if B * H * Sq * Sk > 2 ** 30:
        return None
    new = dict(dtype=torch.float64, device="cuda")
    out, lse = torch.zeros(B, H, Sq, D, **new), torch.zeros(B, H, Sq, **new)
    dq = torch.zeros(B, H, Sq, D, **new)
    dk, dv = torch.zeros(B, Hk, Sk, D, **new), torch.zeros(B, Hk, Sk, D, **new)
    for b in range(B):
        removed = torch.zeros(Sq, Sk, dtype=torch.bool, device="cuda")
        if case["causal"]:
            removed |= torch.ones_like(removed).triu(1 + Sk - Sq)
        if state["mask"] is not None:
            removed |= ~state["mask"][b]
        for h in range(H):
            g = h * Hk // H
            q = state["query"][b, h].double()
            k = state["keys"][b, g].double()
            v = state["values"][b, g].double()
            z = torch.einsum("id,jd->ij", q, k) * state["scale"]
            z = torch.where(removed, -math.inf, z)
            lse[b, h] = torch.logsumexp(z, 1)
            p = torch.nan_to_num(torch.softmax(z, 1), nan=0.0)
            out[b, h] = p @ v
            if case["op"] == "backward":
                do = state["grad"][b, h].double()
                dp = torch.einsum("id,jd->ij", do, v)
                dz = p * (dp - (p * dp).sum(1, keepdim=True))
                dq[b, h] = dz @ k * state["scale"]
                dk[b, g] += torch.einsum("ij,id->jd", dz, q) * state["scale"]
                dv[b, g] += torch.einsum("ij,id->jd", p, do)
    return (dq, dk, dv) if case["op"] == "backward" else (out, lse)


def _exact_paged(case, state):
    B, H, Hk, D = case["B"], case["H"], case["Hk"], case["D"]
    out = torch.zeros(B, H, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(B, H, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_cache_lengths(case)):
        j = torch.arange(n, device="cuda")
        row = state["page_table"][b, j // case["page"]].long()
        for g in range(Hk):
            k = state["key_pages"][row, j % case["page"], g].double()
            v = state["value_pages"][row, j % case["page"], g].double()
            heads = slice(g * (H // Hk), (g + 1) * (H // Hk))
            z = state["query"][b, heads].double() @ k.T * state["scale"]
            lse[b, heads] = torch.logsumexp(z, 1)
            out[b, heads] = torch.softmax(z, 1) @ v
    return out, lse
