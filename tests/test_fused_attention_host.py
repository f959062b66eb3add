"""Fused and paged attention on the CPU: argument checks, workspace sizes,
refusals, and the 64-bit reference of the GPU tests pinned by plain loops and
by differences.  No CUDA call is made."""
import ctypes
import math

import pytest

import entropy_bounded_softmax_gb300 as cs
from entropy_bounded_softmax_gb300 import _lib

torch = pytest.importorskip("torch")

from fused_attention_parity import Forward, gradients

OK, DIM, OOM, BAD = 0, 6, 7, 8
A = [1 << (30 + i) for i in range(13)]      # far-apart fake device addresses


def shape(B=2, H=4, Hk=2, Sq=16, Sk=32, D=64, causal=0, scale=0.125, **kw):
    def strides(h, s):
        return (h * s * D, s * D, D)

    s = cs.cs_attention_shape(B, H, Hk, Sq, Sk, D, causal, scale)
    for name, v in dict(q=strides(H, Sq), k=strides(Hk, Sk),
                        v=strides(Hk, Sk), o=strides(H, Sq),
                        go=strides(H, Sq), dq=strides(H, Sq),
                        dk=strides(Hk, Sk), dv=strides(Hk, Sk)).items():
        setattr(s, name + "_stride", (ctypes.c_int64 * 3)(*kw.pop(name, v)))
    s.mask_stride = kw.pop("mask_stride", Sk)
    assert not kw
    return s


def check(s, q=A[0], k=A[1], v=A[2], out=A[3], lse=A[4], mask=None):
    return cs.cs_check_fused_attention_args(q, k, v, out, lse, mask, s)


@pytest.mark.parametrize("kw,status", [
    (dict(), OK),
    (dict(B=0), OK), (dict(Sq=0), OK), (dict(Sk=0), OK),
    (dict(B=-1), DIM), (dict(Sq=-1), DIM), (dict(Sk=-1), DIM),
    (dict(H=0), DIM), (dict(Hk=0), DIM), (dict(H=3), DIM), (dict(D=0), DIM),
    (dict(B=65536), DIM), (dict(H=1 << 21, Hk=1), DIM),
    (dict(Sq=8388481), DIM), (dict(Sk=8388481), DIM),
    (dict(D=136), OOM), (dict(D=12), BAD), (dict(D=8), OK), (dict(D=128), OK),
    (dict(causal=2), BAD),
    (dict(scale=0.0), BAD), (dict(scale=-1.0), BAD),
    (dict(scale=math.inf), BAD), (dict(scale=math.nan), BAD),
    (dict(q=(4096, 1024, 60)), BAD),          # not a multiple of 8
    (dict(k=(4096, 0, 64)), BAD),             # an expanded head
    (dict(v=(-4096, 2048, 64)), BAD),
    (dict(B=1, q=(3, 1024, 64)), OK),         # one batch: its stride is free
    (dict(o=(1 << 40, 1024, 64)), BAD),       # beyond the tensor copies' reach
])
def test_shapes(kw, status):
    assert check(shape(**kw)) == status


def test_pointers():
    s = shape()
    for name in ("q", "k", "v", "out"):
        assert check(s, **{name: None}) == BAD
        assert check(s, **{name: A[7] + 8}) == BAD        # 16-byte alignment
    assert check(s, lse=None) == OK
    assert check(s, lse=A[4] + 2) == BAD
    assert check(s, out=A[0]) == BAD                      # in place
    assert check(s, out=A[1] + 16) == BAD                 # over the keys
    assert check(s, lse=A[3] + 64) == BAD                 # over out
    assert check(s, k=A[0], v=A[0]) == OK                 # inputs may overlap
    assert check(s, mask=A[5] + 3) == OK                  # any byte
    assert check(s, mask=A[3]) == BAD
    assert check(shape(mask_stride=31), mask=A[5]) == BAD
    assert check(shape(B=1, mask_stride=0), mask=A[5]) == OK


def backward(s, ws=A[9], size=None, grads=(A[6], A[7], A[8]), mask=None):
    if size is None:
        size = cs.cs_fused_attention_backward_workspace(s)
    return cs.cs_check_fused_attention_backward_args(
        *A[:6], *grads, mask, s, ws, size)


def test_backward_arguments():
    s = shape()
    need = cs.cs_fused_attention_backward_workspace(s)
    # Two floats for every query row, rows padded to whole tiles of 128.
    assert need == 2 * 4 * 2 * 4 * 128
    assert backward(s) == OK
    assert backward(s, size=need - 1) == BAD
    assert backward(s, ws=None) == BAD
    assert backward(s, ws=A[9] + 8) == BAD
    assert backward(s, ws=A[6]) == BAD                    # over a gradient
    assert backward(s, grads=(A[6], A[7], A[7])) == BAD   # dk over dv
    assert backward(s, grads=(A[0], A[7], A[8])) == BAD   # dq over the query
    assert backward(s, grads=(A[6], None, A[8])) == BAD
    assert backward(shape(dk=(2048, 1024, 12))) == BAD
    assert backward(shape(B=0), ws=None) == OK
    assert cs.cs_fused_attention_backward_workspace(shape(D=12)) < 0
    assert cs.cs_fused_attention_backward_workspace(shape(Sq=0)) == 0


def paged(B=2, H=8, Hk=2, D=64, page=16, pages=100, most=20, fp16=0,
          scale=0.125, q=None, o=None, k=None, v=None, table=None):
    rows = (H * D, D)
    page_strides = (page * Hk * D, Hk * D, D)
    return cs.cs_paged_shape(B, H, Hk, D, page, pages, most, fp16, scale,
                             q or rows, o or rows, k or page_strides,
                             v or page_strides,
                             most if table is None else table)


def check_paged(s, q=A[0], k=A[1], v=A[2], table=A[3], lengths=A[4],
                out=A[5], lse=A[6], ws=A[7], size=1 << 29):
    return cs.cs_check_paged_attention_args(q, k, v, table, lengths, out, lse,
                                            s, ws, size)


@pytest.mark.parametrize("kw,status", [
    (dict(), OK), (dict(B=0), OK), (dict(most=0), OK), (dict(pages=0), OK),
    (dict(fp16=1), OK), (dict(fp16=2), BAD),
    (dict(B=-1), DIM), (dict(H=0), DIM), (dict(H=3), DIM), (dict(Hk=0), DIM),
    (dict(page=0), DIM), (dict(pages=-1), DIM), (dict(most=-1), DIM),
    (dict(D=264), OOM), (dict(D=20), BAD), (dict(D=256), OK),
    (dict(scale=0.0), BAD), (dict(scale=math.nan), BAD),
    (dict(most=1 << 27), DIM),                # 2^31 tokens a row
    (dict(B=65535, most=1 << 22), DIM),       # 2^42 in the batch
    (dict(table=19), BAD), (dict(B=1, table=0), OK),
    (dict(q=(512, 60)), BAD), (dict(o=(512, 0)), BAD), (dict(o=(0, 64)), BAD),
    (dict(k=(-2048, 128, 64)), BAD), (dict(k=(0, 128, 64)), OK),
    (dict(k=(2048, 128, 12)), BAD),
])
def test_paged_shapes(kw, status):
    assert check_paged(paged(**kw)) == status


def test_paged_pointers_and_workspace():
    s = paged()
    for name in ("q", "k", "v", "out"):
        assert check_paged(s, **{name: None}) == BAD
        assert check_paged(s, **{name: A[8] + 8}) == BAD
    assert check_paged(s, table=None) == BAD
    assert check_paged(s, lengths=None) == BAD
    assert check_paged(s, lengths=A[4] + 2) == BAD
    assert check_paged(s, lse=None) == OK
    assert check_paged(s, out=A[0]) == BAD
    assert check_paged(s, lse=A[4]) == BAD
    need = cs.cs_paged_attention_workspace(s)
    assert need > 0
    assert check_paged(s, size=need) == OK
    assert check_paged(s, size=need - 1) == BAD
    assert check_paged(s, ws=None) == BAD
    assert check_paged(s, ws=A[1]) == BAD
    # Up to 256 tokens a sequence no part is written.
    short = paged(most=16)
    assert cs.cs_paged_attention_workspace(short) == 0
    assert check_paged(short, ws=None, size=0) == OK
    # The workspace does not grow with the lengths beyond a wave of CTAs.
    assert (cs.cs_paged_attention_workspace(paged(most=1000))
            == cs.cs_paged_attention_workspace(paged(most=100000)))
    assert cs.cs_paged_attention_workspace(paged(D=20)) < 0


def test_packed_shapes_are_the_structs():
    q, k, v, o, go = ((i, i + 1, i + 2) for i in range(10, 60, 10))
    dq, dk, dv = ((i, i + 1, i + 2) for i in range(60, 90, 10))
    s = _lib.cs_attention_shape(1, 2, 3, 4, 5, 6, 1, 0.5, q, k, v, o, go, dq,
                                dk, dv, 99)
    assert bytes(s) == _lib.pack_attention_backward_shape(
        1, 2, 3, 4, 5, 6, 1, 0.5, q, k, v, o, go, dq, dk, dv, 99)
    s = _lib.cs_attention_shape(1, 2, 3, 4, 5, 6, 1, 0.5, q, k, v, o)
    s.mask_stride = 99
    assert bytes(s) == _lib.pack_attention_shape(1, 2, 3, 4, 5, 6, 1, 0.5, q,
                                                 k, v, o, 99)
    s = _lib.cs_paged_shape(1, 2, 3, 4, 5, 6, 7, 1, 0.5, q[:2], k[:2], v, o,
                            99)
    assert bytes(s) == _lib.pack_paged_shape(1, 2, 3, 4, 5, 6, 7, 1, 0.5, q,
                                             k, v, o, 99)


def test_cpu_tensors_are_refused():
    q = torch.zeros(1, 2, 4, 16, dtype=torch.bfloat16)
    lse = torch.zeros(1, 2, 4)
    with pytest.raises(ValueError):
        cs.fused_attention(q, q, q)
    with pytest.raises(ValueError):
        cs.fused_attention_backward(q, q, q, q, lse, q)
    with pytest.raises(ValueError):
        cs.FusedAttentionFunction.apply(q, q, q)
    with pytest.raises(ValueError):
        cs.paged_attention(q[0], q, q, torch.zeros(2, 1, dtype=torch.int32),
                           torch.zeros(2, dtype=torch.int32))


def small(seed=0, B=2, H=4, Hk=2, Sq=5, Sk=7, D=8):
    gen = torch.Generator().manual_seed(seed)

    def r(*n):
        return torch.randn(*n, generator=gen, dtype=torch.float64)

    mask = torch.rand(B, Sk, generator=gen) < 0.7
    return (r(B, H, Sq, D), r(B, Hk, Sk, D), r(B, Hk, Sk, D),
            r(B, H, Sq, D), mask)


def test_reference_is_the_definition():
    q, k, v, _, mask = small()
    f = Forward(q, k, v, mask, True, 0.3)
    B, H, Sq, D = q.shape
    Sk = k.shape[2]
    for b in range(B):
        for h in range(H):
            for i in range(Sq):
                keep = [j for j in range(Sk)
                        if mask[b, j] and j <= i + Sk - Sq]
                if not keep:
                    assert f.lse[b, h, i] == -math.inf
                    assert (f.out[b, h, i] == 0).all()
                    continue
                e = [math.exp(0.3 * float(q[b, h, i] @ k[b, h // 2, j]))
                     for j in keep]
                want = sum(x * v[b, h // 2, j] for x, j in zip(e, keep))
                assert torch.allclose(f.out[b, h, i], want / sum(e),
                                      rtol=1e-12, atol=1e-12)
                assert abs(float(f.lse[b, h, i]) - math.log(sum(e))) < 1e-12


@pytest.mark.parametrize("causal", [False, True])
def test_reference_gradients_by_differences(causal):
    q, k, v, g, mask = small(1)
    f = Forward(q, k, v, mask, causal, 0.3)
    grads, _ = gradients(f, f.out, g)

    def loss(*x):
        return float((Forward(*x, mask, causal, 0.3).out * g).sum())

    step = 1e-5
    for n, (x, grad) in enumerate(zip((q, k, v), grads)):
        for at in torch.nonzero(torch.ones_like(x))[::7]:
            sides = []
            for sign in (1, -1):
                y = [t.clone() for t in (q, k, v)]
                y[n][tuple(at)] += sign * step
                sides.append(loss(*y))
            slope = (sides[0] - sides[1]) / (2 * step)
            assert abs(slope - float(grad[tuple(at)])) < 1e-8


def test_written_tensors_do_not_overlap_themselves():
    sbhd = (64, 2 * 64, 2 * 2 * 64)            # [S, H, B, D] storage
    assert check(shape(H=2, Hk=2, o=sbhd)) == OK
    packed = (16 * 3 * 4 * 64, 64, 3 * 4 * 64)   # one of three in a row
    assert check(shape(o=packed)) == OK
    assert check(shape(o=(4096, 1024, 56))) == BAD     # rows into each other
    assert check(shape(o=(4096, 960, 64))) == BAD      # heads
    assert check(shape(o=(64, 64, 256))) == BAD        # the same address twice
    assert check(shape(B=1, o=(0, 1024, 64))) == OK
    assert check(shape(q=(4096, 960, 64))) == OK       # an input may
    for name in ("dq", "dk", "dv"):
        assert backward(shape(**{name: (4096, 1024, 56)})) == BAD
    assert check_paged(paged(o=(512, 56))) == BAD
    assert check_paged(paged(o=(448, 64))) == BAD
    assert check_paged(paged(o=(64, 128))) == OK       # [H, B, D] storage


def test_paged_workspace_follows_the_cut():
    """Rows of sequences that can have up to 512 tokens are not cut where
    there are at least 128 of them, one a key head and sequence."""
    def need(B, most):
        return cs.cs_paged_attention_workspace(paged(B=B, most=most))

    assert need(64, 32) == 0 and need(64, 33) > 0      # 2 key heads each
    assert need(63, 32) > 0 and need(63, 16) == 0
    big = paged(B=2, H=64 * 20, Hk=64, most=32)        # two tiles of 16 heads
    assert cs.cs_paged_attention_workspace(big) == 0
