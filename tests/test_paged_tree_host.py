"""paged_extend, paged_write and paged_tree_attention on the CPU: argument
checks, workspace sizes, refusals, and the references of the GPU tests pinned by
plain loops.  No CUDA call is made."""
import ctypes
import math

import pytest

import entropy_bounded_softmax_gb300 as cs
from entropy_bounded_softmax_gb300 import _lib

torch = pytest.importorskip("torch")

from paged_parity import cache, definition, extend, tree_mask

OK, DIM, OOM, BAD = 0, 6, 7, 8
A = [1 << (32 + i) for i in range(13)]      # far-apart fake device addresses


def test_packed_shapes_have_the_structs_layout():
    """The bytes that the calls pack against the structs of the C ABI."""
    st = [(100 * i + 8, 10 * i + 8, 8 * i) for i in range(1, 5)]
    a = cs.cs_extend_shape(1, 2, 3, 4, 5, 6)
    assert bytes(a) == _lib.pack_extend_shape(1, 2, 3, 4, 5, 6)
    arr = [(ctypes.c_int64 * 3)(*x) for x in st]
    b = cs.cs_write_shape(1, 2, 3, 4, 5, 6, *arr, 7)
    assert bytes(b) == _lib.pack_write_shape(1, 2, 3, 4, 5, 6, *st, 7)
    c = cs.cs_tree_shape(1, 2, 3, 4, 5, 6, 7, 8, 1, 0.5, *arr, 9,
                         (ctypes.c_int64 * 2)(10, 11))
    assert bytes(c) == _lib.pack_tree_shape(1, 2, 3, 4, 5, 6, 7, 8, 1, 0.5,
                                            *st, 9, (10, 11))


@pytest.mark.parametrize("size,scale", [(1 << 31, 0.1), (5, 1e39),
                                        (5, "0.1"), (5.5, 0.1)])
def test_what_the_shapes_cannot_hold_is_refused(size, scale):
    st = (64, 64, 8)
    with pytest.raises(ValueError):
        _lib.pack_tree_shape(1, 4, 1, 1, 8, 16, size, 4, 0, scale, st, st, st,
                             st, 4)
    if size != 5 or scale == 0.1:
        with pytest.raises(ValueError):
            _lib.pack_extend_shape(1, 4, size, 16, 3, 4)
        with pytest.raises(ValueError):
            _lib.pack_write_shape(1, 4, 1, 8, 16, size, st, st, st, st, 4)


def extend_shape(**kw):
    s = cs.cs_extend_shape(3, 5, 7, 16, 9, 7)
    for name, value in kw.items():
        setattr(s, name, value)
    return s


def check_extend(s, **kw):
    names = ("table", "lengths", "new", "held", "free", "cursor", "slots",
             "totals", "have", "after")
    return cs.cs_check_paged_extend_args(
        *(kw.get(name, at) for name, at in zip(names, A)), s)


@pytest.mark.parametrize("kw,status", [
    (dict(), OK), (dict(batch=0), OK), (dict(max_new=0), OK),
    (dict(max_pages=0, table_stride=0), OK), (dict(num_free=0), OK),
    (dict(batch=-1), DIM), (dict(max_new=-1), DIM), (dict(max_pages=-1), DIM),
    (dict(page_size=0), DIM), (dict(num_free=-1), DIM),
    (dict(batch=65536), DIM), (dict(batch=65535), OK),
    (dict(page_size=1 << 28), DIM),          # more than 2^30 tokens a row
    (dict(max_new=(1 << 30) + 1), DIM),
    (dict(table_stride=6), BAD), (dict(table_stride=-7), BAD),
    (dict(table_stride=(1 << 62)), BAD), (dict(table_stride=1 << 20), OK),
    (dict(batch=1, table_stride=0), OK),
])
def test_extend_shapes(kw, status):
    # (Large tables far from the rest.)
    assert check_extend(extend_shape(**kw), slots=1 << 50,
                        table=1 << 58) == status


def test_extend_pointers():
    s = extend_shape()
    assert check_extend(s) == OK
    assert check_extend(s, held=None) == OK
    assert check_extend(s, cursor=None) == OK
    for name in ("table", "lengths", "new", "free", "slots", "totals", "have",
                 "after"):
        assert check_extend(s, **{name: None}) == BAD
        assert check_extend(s, **{name: (1 << 60) + 2}) == BAD   # alignment
    for name in ("table", "slots", "totals", "have", "after"):
        for other in A[1:6]:                      # over an input
            if name != "table" or other != A[0]:
                assert check_extend(s, **{name: other}) == BAD
    assert check_extend(s, totals=A[8]) == BAD    # over another result
    assert check_extend(s, lengths=A[2]) == OK    # inputs may be one


def write_shape(**kw):
    s = cs.cs_write_shape(3, 5, 2, 8, 16, 4, (80, 16, 8), (80, 16, 8),
                          (256, 16, 8), (256, 16, 8), 5)
    for name, value in kw.items():
        setattr(s, name, (ctypes.c_int64 * 3)(*value)
                if isinstance(value, tuple) else value)
    return s


def check_write(s, keys=A[0], values=A[1], slots=A[2], k=A[3], v=A[4]):
    return cs.cs_check_paged_write_args(keys, values, slots, k, v, s)


@pytest.mark.parametrize("kw,status", [
    (dict(), OK), (dict(batch=0), OK), (dict(new_tokens=0), OK),
    (dict(num_pages=0), OK),
    (dict(batch=-1), DIM), (dict(new_tokens=-1), DIM), (dict(kv_heads=0), DIM),
    (dict(d_head=0), DIM), (dict(page_size=0), DIM), (dict(num_pages=-1), DIM),
    (dict(d_head=264), OOM), (dict(d_head=12), BAD),
    (dict(kv_heads=(1 << 20) + 1), DIM),
    (dict(batch=1 << 20, new_tokens=1 << 11), DIM),
    (dict(key_stride=(80, 16, 4)), BAD), (dict(key_stride=(80, -16, 8)), BAD),
    (dict(key_stride=(0, 0, 0)), OK),             # one token for all of them
    (dict(k_stride=(256, 16, 0)), BAD),           # pages that share elements
    (dict(k_stride=(128, 16, 8)), BAD),
    (dict(v_stride=(256, 8, 128)), OK),           # heads before slots
    (dict(v_stride=(256, 12, 128)), BAD),
    (dict(slot_stride=4), BAD), (dict(slot_stride=1 << 62), BAD),
    (dict(batch=1, slot_stride=0), OK),
])
def test_write_shapes(kw, status):
    assert check_write(write_shape(**kw)) == status


def test_write_pointers():
    s = write_shape()
    for name in ("keys", "values", "slots", "k", "v"):
        assert check_write(s, **{name: None}) == BAD
        assert check_write(s, **{name: (1 << 60) + 4}) == BAD
    assert check_write(s, values=A[0]) == OK
    assert check_write(s, k=A[0]) == BAD and check_write(s, v=A[2]) == BAD
    assert check_write(s, v=A[3]) == BAD
    # Keys and values of a page side by side in one buffer: pages of 512
    # elements, the values 256 behind the keys, or each slot's 16 behind.
    side = write_shape(k_stride=(512, 16, 8), v_stride=(512, 16, 8))
    assert check_write(side, v=A[3] + 2 * 256) == OK
    assert check_write(side, k=A[4] + 2 * 256) == OK
    assert check_write(side, v=A[3] + 2 * 240) == BAD
    woven = write_shape(k_stride=(512, 32, 8), v_stride=(512, 32, 8))
    assert check_write(woven, v=A[3] + 2 * 16) == OK
    assert check_write(woven, v=A[3] + 2 * 8) == BAD
    other = write_shape(k_stride=(512, 16, 8), v_stride=(512, 8, 128))
    assert check_write(other, v=A[3] + 2 * 256) == BAD    # other strides


def tree_shape(B=2, T=5, H=8, Hk=2, D=64, page=16, pages=100, most=80, fp16=0,
               scale=0.125, table=None, mask=(25, 5), **kw):
    tok = (T * H * D, H * D, D)
    page_strides = (page * Hk * D, Hk * D, D)
    return cs.cs_tree_shape(
        B, T, H, Hk, D, page, pages, most, fp16, scale, kw.pop("q", tok),
        kw.pop("o", tok), kw.pop("k", page_strides), kw.pop("v", page_strides),
        most if table is None else table, mask)


def check_tree(s, q=A[0], k=A[1], v=A[2], table=A[3], lengths=A[4], new=A[5],
               mask=A[6], out=A[7], lse=A[8], ws=A[9], size=1 << 31):
    return cs.cs_check_paged_tree_attention_args(q, k, v, table, lengths, new,
                                                 mask, out, lse, s, ws, size)


@pytest.mark.parametrize("kw,status", [
    (dict(), OK), (dict(B=0), OK), (dict(T=0), OK), (dict(most=0), OK),
    (dict(pages=0), OK),
    (dict(B=-1), DIM), (dict(T=-1), DIM), (dict(H=0), DIM), (dict(Hk=0), DIM),
    (dict(H=7), DIM), (dict(D=0), DIM), (dict(page=0), DIM),
    (dict(pages=-1), DIM), (dict(most=-1), DIM),
    (dict(B=65536), DIM), (dict(H=1 << 21, Hk=1), DIM),
    (dict(D=264), OOM), (dict(D=256), OK), (dict(D=12), BAD), (dict(D=8), OK),
    (dict(fp16=1), OK), (dict(fp16=2), BAD),
    (dict(scale=0.0), BAD), (dict(scale=-1.0), BAD), (dict(scale=math.nan), BAD),
    (dict(scale=2.0 ** 127), OK), (dict(scale=2.0 ** 127.2), BAD),
    (dict(most=1 << 27), DIM),                # more than 2^30 tokens a row
    (dict(T=1 << 29), DIM),                   # more than 2^30 rows
    # More than 2^30 blocks with their starts and ends: 16381 key heads, one by
    # one, of 65535 sequences.
    (dict(B=65535, H=16381, Hk=16381, D=8, most=1, page=1, pages=1), DIM),
    (dict(q=(2560, 512, 60)), BAD), (dict(q=(-2560, 512, 64)), BAD),
    (dict(q=(0, 0, 0)), OK),
    (dict(o=(2560, 512, 32)), BAD), (dict(o=(2560, 0, 64)), BAD),
    (dict(B=1, o=(3, 512, 64)), OK),
    (dict(table=79), BAD), (dict(table=1 << 61), BAD),
    (dict(mask=(0, 5)), OK), (dict(mask=(25, 4)), BAD), (dict(mask=(-1, 5)), BAD),
    (dict(mask=(1 << 60, 5)), BAD), (dict(mask=(25, 1 << 60)), BAD),
    (dict(T=1, mask=(1, 0)), OK), (dict(B=1, mask=(-3, 5)), OK),
])
def test_tree_shapes(kw, status):
    assert check_tree(tree_shape(**kw)) == status


def test_tree_pointers_and_workspace():
    s = tree_shape()
    need = cs.cs_paged_tree_attention_workspace(s)
    # 1280 tokens: 10 blocks, 2 sequences of 2 units: 40 CTAs at most, two parts
    # each of 32 rows, (maximum, sum) and 64 sums.
    assert need == 40 * 2 * 32 * (8 + 4 * 64)
    assert check_tree(s, size=need) == OK
    assert check_tree(s, size=need - 1) == BAD
    assert check_tree(s, ws=None) == BAD and check_tree(s, ws=A[9] + 8) == BAD
    for name in ("q", "k", "v", "out"):
        assert check_tree(s, **{name: None}) == BAD
        assert check_tree(s, **{name: (1 << 60) + 8}) == BAD
    for name in ("table", "lengths"):
        assert check_tree(s, **{name: None}) == BAD
    for name in ("new", "mask", "lse"):
        assert check_tree(s, **{name: None}) == OK
    assert check_tree(s, mask=(1 << 60) + 3) == OK       # any byte
    for other in A[:7]:
        assert check_tree(s, out=other) == BAD
    assert check_tree(s, lse=A[7]) == BAD and check_tree(s, ws=A[8]) == BAD
    assert check_tree(s, k=A[2]) == OK
    assert cs.cs_paged_tree_attention_workspace(tree_shape(D=12)) < 0
    # Short tables are not cut; nor are longer ones where the batch's units fill
    # three quarters of the SMs and no more than them.
    for B, most, cut in ((2, 32, False), (2, 33, True), (57, 33, False),
                         (76, 64, False), (77, 64, True), (76, 65, True),
                         (56, 64, True)):
        size = cs.cs_paged_tree_attention_workspace(tree_shape(B=B, most=most))
        assert (size > 0) == cut, (B, most)
    # A GB300's SMs hold a CTA each.
    large = tree_shape(B=64, T=64, H=32, Hk=8, D=128, most=512)
    assert (cs.cs_paged_tree_attention_workspace(large)
            == 152 * 2 * 256 * (8 + 4 * 128))


def test_cpu_tensors_are_refused():
    q, k, v, table, lengths = cache([40], 3, 4, 2, 64, 16)
    with pytest.raises(ValueError):
        cs.paged_tree_attention(q, k, v, table, lengths)
    with pytest.raises(ValueError):
        cs.paged_write(q[:, :, :2], q[:, :, :2],
                       torch.zeros(1, 3, dtype=torch.int64), k, v)
    with pytest.raises(ValueError):
        cs.paged_extend(table, lengths, lengths, table[0], 16, 3)
    for bad in (None, [1], 3.0):
        with pytest.raises(ValueError):
            cs.paged_tree_attention(bad, k, v, table, lengths)
        with pytest.raises(ValueError):
            cs.paged_write(bad, q, table, k, v)
        with pytest.raises(ValueError):
            cs.paged_extend(bad, lengths, lengths, table[0], 16, 3)


def test_error_names():
    assert cs.ERROR_BITS["OUT_OF_PAGES"] == 1 << 12
    assert cs.cs_status_string(12) == "no free page left"


@pytest.mark.parametrize("masked", [False, True])
def test_reference_by_plain_loops(masked):
    """The definition of the GPU tests, element by element."""
    args = cache([9, 30, 4], 4, 4, 2, 8, 5, seed=3)
    q, k, v, table, lengths = args
    mask = tree_mask(3, 4, seed=1, empty=True) if masked else None
    new = torch.tensor([4, 3, 2])
    out, _, lse, _ = definition(*args, mask, new, 0.4)
    for b, n in enumerate(lengths.tolist()):
        for i in range(4):
            for h in range(4):
                terms = []
                for j in range(n):
                    draft = j - (n - int(new[b]))
                    if i >= new[b] or (draft >= 0 and not (
                            mask[b, i, draft] if masked else draft <= i)):
                        continue
                    row = int(table[b, j // 5])
                    s = sum(float(x) * float(y) for x, y in
                            zip(q[b, i, h], k[row, j % 5, h // 2])) * 0.4
                    terms.append((math.exp(s), v[row, j % 5, h // 2].double()))
                total = sum(e for e, _ in terms)
                if not terms:
                    assert lse[b, i, h] == -math.inf
                    assert (out[b, i, h] == 0).all()
                    continue
                assert abs(float(lse[b, i, h]) - math.log(total)) < 1e-12
                want = sum(e * x for e, x in terms) / total
                assert (out[b, i, h] - want).abs().max() < 1e-12


def test_trees_are_trees():
    """Every node keeps itself and all that its ancestors keep."""
    for mask in tree_mask(5, 12, seed=4):
        for i in range(12):
            assert mask[i, i] and not mask[i, i + 1:].any()
            for j in range(i):
                if mask[i, j]:
                    assert (mask[j] & ~mask[i]).sum() == 0


def test_pages_by_hand():
    """The loop that the GPU tests hold paged_extend to, on a worked example:
    pages of 4, a list whose first page is taken."""
    table, slots, totals, held, cursor = extend(
        [[7, 3, -1], [5, -1, -1], [6, -1, -1]], [7, 0, 4], [3, 2, 5],
        [9, 2, 8, 4], 4, 3 + 2, None, 1)
    assert table == [[7, 3, 2], [8, -1, -1], [6, 4, -1]]
    assert slots == [[15, 8, 9, -1, -1], [32, 33, -1, -1, -1],
                     [16, 17, 18, 19, -1]]
    assert (totals, held, cursor) == ([10, 2, 8], [3, 1, 2], 4)
