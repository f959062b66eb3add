"""What a NaN in one row reaches: the rows that do not attend it keep the bits
that they have without it, with one CTA a tile and where a cluster of CTAs
shares a tile's keys and joins their parts."""
import math

import pytest

torch = pytest.importorskip("torch")

import entropy_bounded_softmax_gb300 as cs
from test_fused_attention_gpu import inputs

pytestmark = pytest.mark.gpu

# Key lengths that one CTA walks, and that a cluster shares.
LENGTHS = [300, 4096]


def step(q, k, v, g, causal):
    out, lse = cs.fused_attention(q, k, v, causal=causal, return_lse=True)
    return out, lse, *cs.fused_attention_backward(q, k, v, out, lse, g,
                                                  causal=causal)


@pytest.mark.parametrize("Sk", LENGTHS)
@pytest.mark.parametrize("D", [64, 128])
def test_nan_in_one_query(D, Sk):
    """Its row of the output, of lse and of its gradient alone is NaN (the
    gradients of the keys and values, which it has a part in, all are)."""
    q, k, v, g, _, _ = inputs((1, 2, 1, 170, Sk, D, False, None))
    clean = step(q, k, v, g, False)
    assert cs.get_error() == set()
    at = 37
    q[0, 1, at, 3] = math.nan
    got = step(q, k, v, g, False)
    assert cs.get_error() == {"NAN_INPUT"}
    hit = torch.zeros(1, 2, 170, dtype=torch.bool, device="cuda")
    hit[0, 1, at] = True
    for a, b in zip(got[:3], clean):
        assert a[hit].isnan().all()
        assert torch.equal(a[~hit], b[~hit])


@pytest.mark.parametrize("Sk", LENGTHS)
@pytest.mark.parametrize("D", [64, 128])
def test_nan_in_a_key_that_later_queries_keep(D, Sk):
    """Under the causal mask the queries before it keep their bits, those of
    its own tile and block among them."""
    Sq = 200
    q, k, v, _, _, _ = inputs((1, 2, 1, Sq, Sk, D, True, None))
    clean = cs.fused_attention(q, k, v, causal=True, return_lse=True)
    first = 70                       # the first query that keeps the key
    k[0, 0, Sk - Sq + first, 3] = math.nan
    got = cs.fused_attention(q, k, v, causal=True, return_lse=True)
    assert cs.get_error() == {"NAN_INPUT"}
    for a, b in zip(got, clean):
        assert a[:, :, first:].isnan().all()
        assert torch.equal(a[:, :, :first], b[:, :, :first])


@pytest.mark.parametrize("H", [2, 80])
@pytest.mark.parametrize("D", [64, 128])
def test_nan_in_a_value_of_a_later_block(D, H):
    """A causal sequence of whole blocks (2 heads: by clusters): the queries
    whose tile ends before the value's block keep their bits, those that
    attend it are NaN."""
    q, k, v, _, _, _ = inputs((1, H, H, 1024, 1024, D, True, None))
    clean = cs.fused_attention(q, k, v, causal=True)
    v[:, :, 900, 5] = math.nan
    got = cs.fused_attention(q, k, v, causal=True)
    assert torch.equal(got[:, :, :896], clean[:, :, :896])
    assert got[:, :, 900:, 5].isnan().all()
    others = [d for d in range(D) if d != 5]
    assert torch.equal(got[..., others], clean[..., others])
    assert cs.get_error() == set()


def test_nan_in_one_cached_key():
    """paged_attention: only the sequence and the heads that read it."""
    gen = torch.Generator().manual_seed(1)
    k = torch.randn(300, 16, 2, 64, generator=gen).bfloat16().cuda()
    v = torch.randn(300, 16, 2, 64, generator=gen).bfloat16().cuda()
    q = torch.randn(3, 8, 64, generator=gen).bfloat16().cuda()
    table = torch.arange(300, dtype=torch.int32, device="cuda").view(3, 100)
    lengths = torch.tensor([1600, 900, 40], dtype=torch.int32, device="cuda")
    clean = cs.paged_attention(q, k, v, table, lengths, return_lse=True)
    k[110, 3, 1, 7] = math.nan       # sequence 1, token 163, key head 1
    got = cs.paged_attention(q, k, v, table, lengths, return_lse=True)
    assert cs.get_error() == {"NAN_INPUT"}
    for a, b in zip(got, clean):
        assert a[1, 4:].isnan().all()
        assert torch.equal(a[1, :4], b[1, :4])
        assert torch.equal(a[[0, 2]], b[[0, 2]])
