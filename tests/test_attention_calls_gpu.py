"""Calls of the attention operators that their documentation allows and that
the tests against their definitions do not make."""
import math
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

import entropy_bounded_softmax_gb300 as cs
from fused_attention_parity import Forward, excess, gradients
from test_fused_attention_gpu import inputs

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _best_us(call, repeats=5):
    call()
    torch.cuda.synchronize()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    best = math.inf
    for _ in range(repeats):
        start.record()
        call()
        end.record()
        end.synchronize()
        best = min(best, 1e3 * start.elapsed_time(end))
    return best


def _short_sequences(batch, heads=8, D=64):
    """Sequences of one page in a table with room for 64 pages each, which
    makes the call deal shares and join them."""
    gen = torch.Generator(device="cuda").manual_seed(batch)
    lengths = torch.randint(1, 17, (batch,), dtype=torch.int32, device="cuda",
                            generator=gen)
    k, v = (torch.randn(batch, 16, 1, D, device="cuda",
                        generator=gen).bfloat16() for _ in range(2))
    table = torch.zeros(batch, 64, dtype=torch.int32, device="cuda")
    table[:, 0] = torch.randperm(batch, device="cuda", generator=gen)
    q = torch.randn(batch, heads, D, device="cuda", generator=gen).bfloat16()
    return q, k, v, table, lengths


def test_paged_cost_follows_the_batch():
    """Eight times the sequences take about eight times the time (a join that
    walks all lengths for each of them takes 40 times)."""
    small, large = _short_sequences(4096), _short_sequences(32768)
    assert (_best_us(lambda: cs.paged_attention(*large))
            < 16 * _best_us(lambda: cs.paged_attention(*small)))


@pytest.mark.parametrize("batch", [75, 303, 304, 305, 700, 5000])
def test_paged_large_batches(batch):
    """Around and far past the number of groups, whole rows against shares and
    a join: the same sequences in a table of few pages are not cut."""
    q, k, v, table, lengths = _short_sequences(batch, heads=16, D=128)
    k, v = (x.repeat(1, 1, 4, 1) for x in (k, v))
    longer = torch.arange(batch, device="cuda") % 5 == 2
    table[longer, 1:16] = torch.randint(
        0, batch, (int(longer.sum()), 15), dtype=torch.int32, device="cuda")
    lengths[longer] += 200
    wide = cs.paged_attention(q, k, v, table, lengths, return_lse=True)
    whole = cs.paged_attention(q, k, v, table[:, :16].contiguous(), lengths,
                               return_lse=True)
    # Sums in another order: a rounding of the result to bf16 apart at most.
    a, b = wide[0].float(), whole[0].float()
    assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 1e-5).all()
    assert ((wide[1] - whole[1]).abs() <= 2.0 ** -16 * (1 + whole[1].abs())).all()
    assert cs.get_error() == set()


def test_smoke_warns_of_nothing():
    """In a process of its own: torch gives such a warning once."""
    run = subprocess.run(
        [sys.executable, "-W", "error::UserWarning", "-c",
         "import __graft_entry__ as g; g.smoke()"], cwd=ROOT,
        capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr[-2000:]


def test_gradients_are_not_dropped():
    """fused_attention on tensors that require gradients: those of
    FusedAttentionFunction, for each of the three alone too."""
    q, k, v, g, mask, causal = inputs((2, 4, 2, 90, 150, 64, True, "holes"), 9)
    want, lse = cs.fused_attention(q, k, v, mask, causal, 0.2, return_lse=True)
    grads = cs.fused_attention_backward(q, k, v, want, lse, g, mask, causal,
                                        0.2)
    for needed in ((0, 1, 2), (0,), (1,), (2,)):
        args = [x.clone().requires_grad_(n in needed)
                for n, x in enumerate((q, k, v))]
        out, sums = cs.fused_attention(*args, mask, causal, 0.2,
                                       return_lse=True)
        assert torch.equal(out, want) and torch.equal(sums, lse)
        assert out.requires_grad and not sums.requires_grad
        out.backward(g)
        for n, x in enumerate(args):
            assert (torch.equal(x.grad, grads[n]) if n in needed
                    else x.grad is None)
    leaf = q.clone().requires_grad_()
    cs.fused_attention(leaf, k, v, mask, causal, 0.2).backward(g)
    assert torch.equal(leaf.grad, grads[0])
    with torch.no_grad():
        assert not cs.fused_attention(leaf, k, v).requires_grad
        into = torch.empty_like(q)
        assert cs.fused_attention(leaf, k, v, mask, causal, 0.2,
                                  out=into) is into
    assert torch.equal(into, want)
    assert not cs.fused_attention(q, k, v).requires_grad


def test_what_autograd_refuses():
    q, k, v, g, _, _ = inputs((1, 2, 1, 40, 50, 64, False, None))
    leaf = q.clone().requires_grad_()
    with pytest.raises(ValueError):
        cs.fused_attention(leaf, k, v, out=torch.empty_like(q))
    with pytest.raises(ValueError):            # as without a gradient
        cs.fused_attention(leaf, k.expand(1, 2, 50, 64), v.expand(1, 2, 50, 64))
    with pytest.raises(TypeError):
        cs.fused_attention(leaf, k.half(), v.half())
    out = cs.fused_attention(leaf, k, v)
    first, = torch.autograd.grad(out, leaf, g, create_graph=True)
    with pytest.raises(RuntimeError):          # no second derivative
        first.sum().backward()
    import torch.autograd.forward_ad as fwd
    with fwd.dual_level(), pytest.raises((RuntimeError, NotImplementedError)):
        cs.FusedAttentionFunction.apply(fwd.make_dual(q, g), k, v)


def test_autograd_takes_an_expanded_mask():
    """One sequence's mask for all of them, and a transposed one."""
    q, k, v, g, _, _ = inputs((2, 4, 2, 60, 130, 64, False, None))
    one = torch.arange(130, device="cuda")[None] % 3 != 1
    tall = torch.empty(130, 2, dtype=torch.bool, device="cuda")
    tall.copy_(one.T)
    want, lse = cs.fused_attention(q, k, v, one.repeat(2, 1), return_lse=True)
    dq, _, _ = cs.fused_attention_backward(q, k, v, want, lse, g,
                                           one.repeat(2, 1))
    for mask in (one.expand(2, 130), tall.T):
        leaf = q.clone().requires_grad_()
        out = cs.FusedAttentionFunction.apply(leaf, k, v, mask)
        out.backward(g)
        assert torch.equal(out, want) and torch.equal(leaf.grad, dq)


def _attention64(q, k, v, g, scale):
    """One head in 64 bits on the GPU: out, lse, dq, dk, dv of all keys."""
    q, k, v, g = (x.double() for x in (q, k, v, g))
    s = q @ k.T * scale
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse[:, None])
    out = p @ v
    ds = p * (g @ v.T - (g * out).sum(-1, keepdim=True))
    return out, lse, ds @ k * scale, ds.T @ q * scale, p.T @ g


@pytest.mark.parametrize("B,H,Hk,Sq,Sk", [
    (65535, 1, 1, 1, 3),           # the most sequences
    (1, 1 << 20, 1 << 18, 1, 5),   # the most heads
    (1, 1, 1, 8388480, 9),         # the most queries
    (1, 1, 1, 3, 8388480),         # the most keys
])
def test_largest_sizes(B, H, Hk, Sq, Sk):
    """The far ends of the ranges, with heads of 8.  Few keys and queries: a
    few heads by elements.  Long sums: by norms, where P and dS, delta's out
    and the result are rounded by at most 2^-8 each (less on average), and an
    accumulator that truncates loses at most 2^-24 of the sum on average at
    each of its 2^16 steps: 2^-8."""
    gen = torch.Generator(device="cuda").manual_seed(2)

    def heads(h, n):
        return torch.randn(B, h, n, 8, device="cuda", generator=gen).bfloat16()

    q, g, k, v = heads(H, Sq), heads(H, Sq), heads(Hk, Sk), heads(Hk, Sk)
    out, lse = cs.fused_attention(q, k, v, return_lse=True)
    dq, dk, dv = cs.fused_attention_backward(q, k, v, out, lse, g)
    assert cs.get_error() == set()
    group = H // Hk
    if Sq * Sk < 100:
        for b, hk in ((0, 0), (B // 2, Hk // 2), (B - 1, Hk - 1)):
            b, h = slice(b, b + 1), slice(hk * group, (hk + 1) * group)
            hk = slice(hk, hk + 1)
            ref = Forward(q[b, h], k[b, hk], v[b, hk], None, False, 8 ** -0.5)
            assert excess(out[b, h], ref.out, ref.out_tol()) <= 1
            assert excess(lse[b, h], ref.lse, ref.lse_tol()) <= 1
            want, tol = gradients(ref, out[b, h], g[b, h])
            for x, y, t in zip((dq[b, h], dk[b, hk], dv[b, hk]), want, tol):
                assert excess(x, y, t) <= 1
        return
    ref = _attention64(q[0, 0], k[0, 0], v[0, 0], g[0, 0], 8 ** -0.5)
    assert float((lse[0, 0].double() - ref[1]).abs().max()) < 2.0 ** -12
    for x, y in zip((out, dq, dk, dv), (ref[0], *ref[2:])):
        assert float((x[0, 0].double() - y).norm() / y.norm()) < 4 * 2.0 ** -8


def test_pages_used_twice():
    """A page that two sequences share, and one that a sequence has twice."""
    gen = torch.Generator(device="cuda").manual_seed(6)
    k, v = (torch.randn(4, 16, 2, 64, device="cuda", generator=gen).bfloat16()
            for _ in range(2))
    q = torch.randn(2, 4, 64, device="cuda", generator=gen).bfloat16()
    table = torch.tensor([[2, 0, 2, 3], [2, 2, 1, 0]], dtype=torch.int32,
                         device="cuda")
    lengths = torch.tensor([64, 41], dtype=torch.int32, device="cuda")
    got = cs.paged_attention(q, k, v, table, lengths)
    rows = table.flatten().long()
    apart = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
    want = cs.paged_attention(q, k[rows].contiguous(), v[rows].contiguous(),
                              apart, lengths)
    assert torch.equal(got, want) and cs.get_error() == set()


def test_longest_cache():
    """A row of the table with room for 2^30 tokens, in one page and in pages
    of 2^20 slots, the tokens at the far end of it."""
    gen = torch.Generator(device="cuda").manual_seed(7)
    q = torch.randn(1, 2, 8, device="cuda", generator=gen).bfloat16()
    # All slots the same token: out is its value, lse the score plus ln 2^30.
    k, v = (torch.randn(1, 1, 1, 8, device="cuda", generator=gen).bfloat16()
            for _ in range(2))
    many = (x.expand(1, 1 << 30, 1, 8) for x in (k, v))
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    lengths = torch.tensor([1 << 30], dtype=torch.int32, device="cuda")
    out, lse = cs.paged_attention(q, *many, table, lengths, return_lse=True)
    s = (q.double() @ k[0, 0, 0].double()) * 8 ** -0.5
    # Half a step of bf16, and at most 2^-24 on average at each of the 2^16
    # steps of an accumulator that truncates.
    value = v[0, 0].double()
    assert ((out.double() - value).abs() <= 2.0 ** -7 * value.abs()).all()
    # (The sums are of whole multiples of one weight, fewer than 2^24.)
    assert float((lse.double() - s - 30 * math.log(2)).abs().max()) < 2.0 ** -16
    page = 1 << 20
    k, v = (torch.randn(2, page, 1, 8, device="cuda", generator=gen).bfloat16()
            for _ in range(2))
    table = torch.zeros(3, 1024, dtype=torch.int32, device="cuda")
    table[1, 1] = 1
    lengths = torch.tensor([5, page + 3, 0], dtype=torch.int32, device="cuda")
    q = torch.randn(3, 2, 8, device="cuda", generator=gen).bfloat16()
    out = cs.paged_attention(q, k, v, table, lengths)
    for b, keys, values in ((0, k[0, :5], v[0, :5]),
                            (1, torch.cat([k[0], k[1, :3]]),
                             torch.cat([v[0], v[1, :3]]))):
        want = _attention64(q[b], keys[:, 0], values[:, 0], q[b], 8 ** -0.5)[0]
        # Half a step of bf16; the sums' fp32, cancelling, far below it.
        assert float((out[b].double() - want).norm() / want.norm()) < 2.0 ** -8
    assert (out[2] == 0).all() and cs.get_error() == set()


def test_captured_training_step():
    """Forward and backward through autograd, captured after a warm-up on a
    side stream, and replayed on new inputs."""
    first = inputs((2, 4, 2, 90, 150, 64, True, "right"), 20)
    second = inputs((2, 4, 2, 90, 150, 64, True, "right"), 21)
    leaves = [x.clone().requires_grad_() for x in first[:3]]
    g, mask = first[3].clone(), first[4]

    def step():
        out = cs.fused_attention(*leaves, mask, True)
        return (out.detach(), *torch.autograd.grad(out, leaves, g))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        results = step()
    for q, k, v, up, _, _ in (second, first):
        with torch.no_grad():
            for dst, src in zip((*leaves, g), (q, k, v, up)):
                dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        out, lse = cs.fused_attention(q, k, v, mask, True, return_lse=True)
        want = (out, *cs.fused_attention_backward(q, k, v, out, lse, up, mask,
                                                  True))
        for a, b in zip(results, want):
            assert torch.equal(a, b)
