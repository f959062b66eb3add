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


def test_removed_keys_may_hold_anything():
    """NaN and infinities in the keys and values that the mask removes, and a
    mask whose rows are a slice of a wider, unaligned one."""
    for case in [(2, 2, 1, 200, 300, 64, True, "right"),
                 (2, 2, 2, 150, 260, 128, False, "left"),
                 (2, 4, 2, 140, 400, 96, True, "holes")]:
        q, k, v, g, mask, causal = inputs(case, 2)
        want = run_both(q, k, v, g, mask, causal)
        gone = ~mask[:, None, :, None]
        k2 = k.masked_fill(gone, math.nan)
        v2 = v.masked_fill(gone, math.inf)
        v2[..., ::2] = v2[..., ::2].masked_fill(gone, math.nan)
        wide = torch.ones(mask.shape[0], mask.shape[1] + 13, dtype=torch.bool,
                          device="cuda")
        wide[:, 5:5 + mask.shape[1]] = mask
        sliced = wide[:, 5:5 + mask.shape[1]]
        got = run_both(q, k2, v2, g, sliced, causal)
        for a, b in zip((*got[:2], *got[2]), (*want[:2], *want[2])):
            assert torch.equal(a, b)


@pytest.mark.parametrize("D", [64, 128])
def test_sharp_and_growing_scores(D):
    """Scores in the hundreds, whose maximum grows block after block (every
    block rescales the output) or stands at the first key."""
    for order in (1, -1):
        q, k, v, g, mask, causal = inputs((1, 2, 2, 130, 600, D, False, None),
                                          3, scale=4.0)
        q, g, v = q / 4, g / 4, v / 4
        ramp = torch.linspace(0.2, 3.0, 600, device="cuda")[None, None, :, None]
        q = q.abs()
        k = (k.abs() * (ramp if order > 0 else ramp.flip(2))).bfloat16()
        check(q, k, v, g, mask, causal, scale=0.2)


def test_scale_and_uniform_scores():
    q, k, v, g, mask, causal = inputs((1, 2, 1, 140, 200, 64, True, None), 4)
    check(q, k, v, g, mask, causal, scale=2.0 ** -20)
    zero = torch.zeros_like(k)
    out, _ = cs.fused_attention(q, zero, v, causal=True, return_lse=True)
    ref = Forward(q, zero, v, None, True, 0.125)
    assert excess(out, ref.out, ref.out_tol()) <= 1


def test_slices_of_a_packed_projection():
    """Query, keys and values as views of one [B, S, H + 2 Hk, D] projection;
    the output into a slice of a larger buffer, whose rest stays."""
    B, S, H, Hk, D = 2, 150, 4, 2, 64
    gen = torch.Generator().manual_seed(7)
    packed = torch.randn(B, S, H + 2 * Hk, D, generator=gen).bfloat16().cuda()
    q, k, v = (x.transpose(1, 2) for x in packed.split([H, Hk, Hk], 2))
    g = torch.randn(B, S, H, D, generator=gen).bfloat16().cuda().transpose(1, 2)
    check(q, k, v, g, None, True)
    for fill, width in ((3.0, D), (5.0, D + 8)):
        big = torch.full((B + 1, H + 1, S + 40, width), fill,
                         dtype=torch.bfloat16, device="cuda")
        into = big[:B, :H, 8:8 + S, :D]
        out = cs.fused_attention(q, k, v, causal=True, out=into)
        assert out.data_ptr() == into.data_ptr()
        assert torch.equal(into, cs.fused_attention(q, k, v, causal=True))
        rest = big.clone()
        rest[:B, :H, 8:8 + S, :D] = fill
        assert (rest == fill).all()


def test_strides_past_32_bits():
    """Batches more than 2^31 elements apart."""
    far = (1 << 31) + 64
    store = torch.empty(far + 200 * 64, dtype=torch.bfloat16, device="cuda")
    case = (2, 1, 1, 130, 190, 64, True, None)
    q, k, v, g, _, _ = inputs(case, 8)
    want = run_both(q, k, v, g, None, True)

    def spread(x):
        y = store.as_strided(x.shape, (far, x.shape[2] * 64, 64, 1))
        y.copy_(x)
        return y

    for i in range(4):
        args = [q, k, v, g]
        args[i] = spread(args[i])
        got = run_both(*args, None, True)
        for a, b in zip((*got[:2], *got[2]), (*want[:2], *want[2])):
            assert torch.equal(a, b)
    del store


def test_empty_sizes():
    def t(*n):
        return torch.randn(*n, device="cuda").bfloat16()

    out, lse = cs.fused_attention(t(0, 2, 5, 16), t(0, 2, 7, 16),
                                  t(0, 2, 7, 16), return_lse=True)
    assert out.shape == (0, 2, 5, 16) and lse.shape == (0, 2, 5)
    out = cs.fused_attention(t(2, 2, 0, 16), t(2, 2, 7, 16), t(2, 2, 7, 16))
    assert out.shape == (2, 2, 0, 16)
    for D in (16, 128):
        q, k, g = t(2, 2, 5, D), t(2, 2, 0, D), t(2, 2, 5, D)
        out, lse = cs.fused_attention(q, k, k, return_lse=True)
        assert (out == 0).all() and (lse == -math.inf).all()
        dq, dk, dv = cs.fused_attention_backward(q, k, k, out, lse, g)
        assert (dq == 0).all() and dk.shape == k.shape
        q, k, lse = t(2, 4, 0, D), t(2, 2, 5, D), torch.empty(2, 4, 0,
                                                             device="cuda")
        dq, dk, dv = cs.fused_attention_backward(q, k, k, q, lse, q)
        assert dq.shape == q.shape and (dk == 0).all() and (dv == 0).all()
    torch.cuda.synchronize()
    assert cs.get_error() == set()


def test_nan_scores_are_reported():
    q, k, v, _, _, _ = inputs((1, 1, 1, 40, 50, 64, False, None))
    q[0, 0, 3, 5] = math.nan
    out = cs.fused_attention(q, k, v)
    assert out[0, 0, 3].isnan().all()
    rows = [i for i in range(40) if i != 3]
    assert out[0, 0, rows].isfinite().all()
    assert cs.get_error() == {"NAN_INPUT"}


def test_refusals():
    q, k, v, g, mask, _ = inputs((2, 4, 2, 20, 30, 64, False, "right"))
    out, lse = cs.fused_attention(q, k, v, return_lse=True)

    def bad(error, *args, **kw):
        with pytest.raises(error):
            cs.fused_attention(*args, **kw)

    bad(TypeError, q.float(), k, v)
    bad(TypeError, q, k.half(), v.half())
    bad(ValueError, q[0], k, v)
    bad(ValueError, q, k, v[:, :1])
    bad(ValueError, q, k[:1], v[:1])
    bad(ValueError, q[:, :3], k, v)
    bad(ValueError, q, k[..., :56], v[..., :56])
    bad(ValueError, q[..., :60].contiguous(), k[..., :60].contiguous(),
        v[..., :60].contiguous())
    bad(ValueError, q.expand(2, 4, 20, 64)[..., ::2], k[..., ::2],
        v[..., ::2])
    bad(ValueError, q, k[:, :1].expand(2, 2, 30, 64), v)
    bad(ValueError, q, k, v, scale=0.0)
    bad(ValueError, q, k, v, scale=-1.0)
    bad(ValueError, q, k, v, scale=math.inf)
    bad(ValueError, q, k, v, mask=mask.float())
    bad(ValueError, q, k, v, mask=mask[:, :-1])
    bad(ValueError, q, k, v, mask=mask.cpu())
    bad(ValueError, q, k, v, mask=mask[:1].expand(2, 30))
    bad(ValueError, q, k, v, out=out[:, :2])
    bad(TypeError, q, k, v, out=out.float())
    bad(cs.CsError, q, k, v, out=q)
    odd = torch.empty(2 * 4 * 20 * 64 + 1, dtype=torch.bfloat16,
                      device="cuda")[1:].view(2, 4, 20, 64)
    bad(ValueError, odd, k, v)
    for args in ((q, k, v, out[:, :2], lse, g), (q, k, v, out, lse[:1], g),
                 (q, k, v, out, lse.half(), g), (q, k, v, out, lse, g[:1])):
        with pytest.raises(ValueError):
            cs.fused_attention_backward(*args)
    with pytest.raises(TypeError):
        cs.fused_attention_backward(q, k, v, out, lse, g.float())


def test_autograd():
    """The function's gradients are those of the calls, an expanded key and
    value (copied) and an expanded upstream gradient among the inputs."""
    q, k, v, g, mask, _ = inputs((2, 4, 2, 100, 150, 64, True, "holes"), 9)
    leaves = [x.clone().requires_grad_() for x in (q, k, v)]
    y = cs.FusedAttentionFunction.apply(*leaves, mask, True, 0.2)
    y.backward(g)
    out, lse = cs.fused_attention(q, k, v, mask, True, 0.2, return_lse=True)
    assert torch.equal(y, out)
    want = cs.fused_attention_backward(q, k, v, out, lse, g, mask, True, 0.2)
    for x, w in zip(leaves, want):
        assert torch.equal(x.grad, w)
    one = k[:, :1].clone().requires_grad_()
    y = cs.FusedAttentionFunction.apply(q, one.expand_as(k), v)
    y.sum().backward()
    out, lse = cs.fused_attention(q, k[:, :1].expand_as(k).contiguous(), v,
                                  return_lse=True)
    ones = torch.ones_like(out)
    _, dk, _ = cs.fused_attention_backward(
        q, k[:, :1].expand_as(k).contiguous(), v, out, lse, ones)
    assert torch.equal(one.grad, dk.sum(1, keepdim=True))


def test_streams_and_graphs():
    """A side stream; a captured step replayed on new inputs, twice, beside
    another graph of the same kernels."""
    case = (2, 4, 2, 150, 200, 128, True, "right")
    first = inputs(case, 10)
    second = inputs(case, 11)
    want = [run_both(*x) for x in (first, second)]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        got = run_both(*first)
    stream.synchronize()
    assert torch.equal(got[0], want[0][0])
    q, k, v, g, mask, causal = first
    fixed = [x.clone() for x in (q, k, v, g, mask)]
    graphs, results = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out, lse = cs.fused_attention(*fixed[:3], fixed[4], causal,
                                          return_lse=True)
            grads = cs.fused_attention_backward(*fixed[:3], out, lse,
                                                fixed[3], fixed[4], causal)
        graphs.append(graph)
        results.append((out, lse, *grads))
    for data, w in ((second, want[1]), (first, want[0]), (second, want[1])):
        for dst, src in zip(fixed, data[:5]):
            dst.copy_(src)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
        torch.cuda.synchronize()
        for r in results:
            for a, b in zip(r, (w[0], w[1], *w[2])):
                assert torch.equal(a, b)


def test_training_step():
    """Attention inside a projection, as it is trained: the gradients of the
    weights against differences of the same loss in 64 bits."""
    torch.manual_seed(3)
    B, S, H, Hk, D, E = 2, 70, 4, 2, 16, 32
    x = torch.randn(B, S, E).bfloat16()
    mask = torch.ones(B, S, dtype=torch.bool)
    mask[1, 50:] = False
    weight = (torch.randn(E, (H + 2 * Hk) * D) / E ** 0.5).bfloat16()
    target = torch.randn(B, H, S, D).bfloat16()

    def heads(y):
        y = y.view(B, S, H + 2 * Hk, D).transpose(1, 2)
        return y[:, :H], y[:, H:H + Hk], y[:, H + Hk:]

    w = weight.cuda().requires_grad_()
    out = cs.FusedAttentionFunction.apply(*heads(x.cuda() @ w), mask.cuda(),
                                          True)
    (out.float() * target.cuda().float()).sum().backward()
    w64 = weight.double().requires_grad_()
    q, k, v = heads(x.double() @ w64)
    s = q @ k.repeat_interleave(2, 1).mT / D ** 0.5
    keep = mask[:, None, None] & torch.ones(S, S, dtype=torch.bool).tril()
    p = s.masked_fill(~keep, -math.inf).softmax(-1)
    ((p @ v.repeat_interleave(2, 1)) * target.double()).sum().backward()
    # Each of the projection, its weights' rounding, P, dS and the gradients
    # that reach the weights is rounded to 2^-8 of its value at most, seven
    # roundings in a chain and independent between the terms of the sums.
    off = (w.grad.cpu().double() - w64.grad).norm() / w64.grad.norm()
    assert float(off) < 7 * 2.0 ** -8


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


@pytest.mark.parametrize("D", [64, 128])
def test_queries_without_keys_stay_zero_beside_nan(D):
    """Queries 0..39 keep no key; the keys and values that others of their
    block keep hold NaN, which 0 weights would carry over to them."""
    q, k, v, g, _, _ = inputs((1, 2, 1, 100, 60, D, True, None))
    v[0, 0, 5] = math.nan
    k[0, 0, 5] = math.nan
    out, lse = cs.fused_attention(q, k, v, causal=True, return_lse=True)
    assert (out[:, :, :40] == 0).all() and (lse[:, :, :40] == -math.inf).all()
    dq, _, _ = cs.fused_attention_backward(q, k, v, out, lse, g, causal=True)
    assert (dq[:, :, :40] == 0).all()
    assert out[:, :, 45:].isnan().all()
    assert cs.get_error() == {"NAN_INPUT"}


def test_autograd_takes_an_odd_base():
    """A contiguous input whose base is not 16-byte aligned is copied."""
    q, k, v, g, _, _ = inputs((1, 2, 2, 40, 50, 64, False, None))
    store = torch.empty(q.numel() + 1, dtype=torch.bfloat16, device="cuda")
    odd = store[1:].view(q.shape).copy_(q).requires_grad_()
    assert odd.data_ptr() % 16 != 0
    out = cs.FusedAttentionFunction.apply(odd, k, v)
    out.backward(g)
    want, lse = cs.fused_attention(q, k, v, return_lse=True)
    dq, _, _ = cs.fused_attention_backward(q, k, v, want, lse, g)
    assert torch.equal(out, want) and torch.equal(odd.grad, dq)


def test_outputs_that_overlap_themselves_are_refused():
    q, k, v, _, _, _ = inputs((2, 4, 2, 20, 30, 64, False, None))
    store = torch.empty(2 * 4 * 20 * 64, dtype=torch.bfloat16, device="cuda")
    out = store.as_strided((2, 4, 20, 64), (4 * 20 * 64, 20 * 64, 32, 1))
    with pytest.raises(cs.CsError):
        cs.fused_attention(q, k, v, out=out)


def test_no_queries_behind_work_that_allows_overlap():
    """Gradients of keys without queries, in memory that the kernels before
    still use: the call may not start before they end."""
    k = torch.randn(1, 2, 4096, 64, device="cuda").bfloat16()
    q = k[:, :, :0]
    lse = torch.empty(1, 2, 0, device="cuda")
    qp = torch.randn(4, 8, 128, device="cuda").bfloat16()
    pages = torch.randn(4096, 16, 8, 128, device="cuda").bfloat16()
    table = torch.arange(4096, dtype=torch.int32, device="cuda").view(4, 1024)
    lengths = torch.full((4,), 16384, dtype=torch.int32, device="cuda")
    want = cs.paged_attention(qp, pages, pages, table, lengths)
    for _ in range(5):
        got = cs.paged_attention(qp, pages, pages, table, lengths)
        _, dk, dv = cs.fused_attention_backward(q, k, k, q, lse, q)
        assert torch.equal(got, want)
        assert (dk == 0).all() and (dv == 0).all()


@pytest.mark.parametrize("case", [
    (1, 4, 1, 1100, 300, 64, False, None),     # keys: eight CTAs a tile
    (1, 4, 1, 300, 1100, 128, True, None),     # both by clusters
    (1, 6, 2, 900, 700, 128, True, "left"),    # tiles without blocks among them
    (2, 2, 1, 150, 1500, 40, False, "holes"),
    (1, 8, 1, 1300, 140, 96, True, "right"),   # queries without keys
    (1, 2, 1, 1000, 1000, 64, True, "all"),    # no key at all
], ids=str)
def test_few_tiles(case):
    """Tiles of gradients that several CTAs share, and join."""
    args = inputs(case)
    _, _, grads = check(*args)
    for _ in range(5):
        again = run_both(*args)[2]
        assert all(torch.equal(x, y) for x, y in zip(grads, again))


@pytest.mark.parametrize("case", [
    (1, 2, 1, 1, 5000, 128, False, "right"),   # one query, eight CTAs
    (1, 3, 1, 140, 4100, 64, True, "left"),
    (1, 2, 2, 600, 2500, 72, True, "holes"),
    (2, 2, 1, 700, 600, 128, True, None),      # queries without keys
    (1, 2, 1, 300, 2048, 8, False, "all"),
], ids=str)
def test_few_queries(case):
    """Outputs of tiles whose keys several CTAs share, and join."""
    args = inputs(case)
    out, lse, _ = check(*args)
    q, k, v, _, mask, causal = args
    for _ in range(5):
        again, lse2 = cs.fused_attention(q, k, v, mask, causal,
                                         return_lse=True)
        assert torch.equal(out, again) and torch.equal(lse, lse2)


def test_nan_in_one_share_of_the_keys():
    """Scores of keys far apart, one of them NaN: reported, and only in the
    queries that attend it."""
    q, k, v, _, _, _ = inputs((1, 1, 1, 70, 4096, 64, False, None))
    k[0, 0, 4000, 3] = math.nan
    out = cs.fused_attention(q, k, v)
    assert out.isnan().all() and cs.get_error() == {"NAN_INPUT"}
    keep = torch.ones(1, 4096, dtype=torch.bool, device="cuda")
    keep[0, 4000] = False
    assert cs.fused_attention(q, k, v, keep).isfinite().all()
    assert cs.get_error() == set()
