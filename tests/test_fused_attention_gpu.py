"""fused_attention and fused_attention_backward against their definitions in
64 bits, at the sizes and masks where tiled kernels go wrong."""
import math

import pytest

torch = pytest.importorskip("torch")

import entropy_bounded_softmax_gb300 as cs
from fused_attention_parity import Forward, excess, gradients

pytestmark = pytest.mark.gpu

# B, H, Hk, Sq, Sk, D, causal, mask
CASES = [
    (1, 1, 1, 1, 1, 8, False, None),
    (1, 2, 1, 1, 200, 64, True, None),          # one new token
    (1, 2, 2, 128, 128, 64, False, None),       # exactly one tile
    (1, 2, 2, 128, 128, 128, False, None),
    (2, 4, 2, 77, 77, 64, True, None),
    (1, 2, 2, 256, 256, 128, True, None),
    (1, 1, 1, 257, 129, 16, False, None),       # one past a tile, both sides
    (2, 3, 1, 129, 257, 80, True, None),        # longer keys, odd head size
    (1, 2, 1, 300, 100, 40, True, None),        # queries without keys
    (1, 8, 1, 65, 190, 128, True, None),        # eight heads share a key head
    (2, 2, 2, 100, 300, 96, False, "right"),
    (2, 2, 1, 200, 200, 128, True, "left"),     # rows left empty
    (2, 4, 4, 130, 515, 64, False, "holes"),
    (3, 2, 1, 300, 700, 120, True, "holes"),
    (2, 1, 1, 70, 260, 128, False, "all"),      # one sequence without keys
    (1, 2, 2, 640, 1000, 128, True, None),
    (2, 2, 2, 512, 512, 64, False, "right"),
]


def inputs(case, seed=0, layout="bhsd", scale=1.0):
    B, H, Hk, Sq, Sk, D, causal, kind = case
    gen = torch.Generator().manual_seed(seed)

    def heads(h, s):
        if layout == "bshd":
            x = torch.randn(B, s, h, D, generator=gen) * scale
            return x.bfloat16().cuda().transpose(1, 2)
        return (torch.randn(B, h, s, D, generator=gen) * scale).bfloat16().cuda()

    q, k, v, g = heads(H, Sq), heads(Hk, Sk), heads(Hk, Sk), heads(H, Sq)
    mask = None
    if kind is not None:
        j = torch.arange(Sk)[None, :]
        n = torch.tensor([Sk - (b * Sk) // (2 * B) - 3 for b in range(B)])[:, None]
        mask = {"right": j < n, "left": j >= Sk - n,
                "holes": torch.rand(B, Sk, generator=gen) < 0.7,
                "all": (j < n) & (torch.arange(B)[:, None] > 0)}[kind].cuda()
    return q, k, v, g, mask, causal


def run_both(q, k, v, g, mask, causal, scale=None):
    out, lse = cs.fused_attention(q, k, v, mask, causal, scale,
                                  return_lse=True)
    grads = cs.fused_attention_backward(q, k, v, out, lse, g, mask, causal,
                                        scale)
    torch.cuda.synchronize()
    assert cs.get_error() == set()
    return out, lse, grads


def check(q, k, v, g, mask, causal, scale=None):
    out, lse, grads = run_both(q, k, v, g, mask, causal, scale)
    ref = Forward(q, k, v, mask, causal,
                  1 / math.sqrt(q.shape[3]) if scale is None else scale)
    empty = ref.lse == -math.inf
    assert torch.equal(lse.cpu() == -math.inf, empty)
    assert (out.cpu()[empty] == 0).all() and (grads[0].cpu()[empty] == 0).all()
    assert excess(lse.cpu()[~empty], ref.lse[~empty],
                  ref.lse_tol()[~empty]) <= 1
    assert excess(out, ref.out, ref.out_tol()) <= 1
    want, tol = gradients(ref, out, g)
    for name, x, w, t in zip(("dq", "dk", "dv"), grads, want, tol):
        assert x.dtype == torch.bfloat16
        assert excess(x, w, t) <= 1, name
    if mask is not None:
        gone = ~mask.cpu()
        for x in grads[1:]:
            assert (x.cpu().transpose(1, 2)[gone] == 0).all()
    return out, lse, grads


@pytest.mark.parametrize("case", CASES, ids=str)
def test_against_definition(case):
    check(*inputs(case))


@pytest.mark.parametrize("case", CASES[4:12:3], ids=str)
def test_sequence_major_storage(case):
    q, k, v, g, mask, causal = inputs(case, 1, "bshd")
    out, _, grads = check(q, k, v, g, mask, causal)
    assert out.stride() == q.stride()
    assert [x.stride() for x in grads] == [x.stride() for x in (q, k, v)]
    same = run_both(*(x.contiguous() for x in (q, k, v, g)), mask, causal)
    assert torch.equal(out, same[0])
    for a, b in zip(grads, same[2]):
        assert torch.equal(a, b)


@pytest.mark.parametrize("case", [
    (1, 4, 2, 300, 700, 64, True, "holes"),
    (1, 4, 2, 300, 700, 128, True, "holes"),
    (3, 8, 4, 700, 700, 64, True, None),
    (3, 8, 4, 700, 700, 128, True, None),
], ids=str)
def test_repeated_calls_agree(case):
    """Hundreds of launches beside another stream's work: the same bits, and
    no wait that gives up (the warps' order differs from launch to launch)."""
    q, k, v, g, mask, causal = inputs(case, 5)
    out, lse, grads = check(q, k, v, g, mask, causal)
    noise = torch.randn(2048, 2048, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(150):
        if i % 3 == 0:
            with torch.cuda.stream(side):
                noise = noise @ noise * 1e-3
        o, l = cs.fused_attention(q, k, v, mask, causal, return_lse=True)
        d = cs.fused_attention_backward(q, k, v, o, l, g, mask, causal)
        for a, b in zip((o, l, *d), (out, lse, *grads)):
            differ += (a.view(torch.int16) != b.view(torch.int16)).sum()
    torch.cuda.synchronize()
    assert int(differ) == 0
    assert cs.get_error() == set()
