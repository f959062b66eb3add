"""Calls of the attention operators that their documentation allows and that
the tests against their definitions do not make."""
import math
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

import entropy_bounded_softmax_gb300 as cs
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


@pytest.mark.parametrize("batch", [75, 76, 77, 700, 5000])
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
