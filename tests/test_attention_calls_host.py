"""Fused and paged attention on the CPU: arguments at the far end of their
ranges, and rules of the sources that no GPU here can show.  No CUDA call is
made."""
import ctypes
import glob
import os
import re

import pytest

import entropy_bounded_softmax_gb300 as cs
from entropy_bounded_softmax_gb300 import _lib

CSRC = os.path.join(os.path.dirname(cs.__file__), "csrc")


def _code(path):
    """A source file without its comments."""
    with open(path) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    return re.sub(r"//[^\n]*", "", text)


def test_launches_ask_the_device_for_its_sms():
    """The number of SMs is the device's in every launch; the one literal
    bounds a workspace whose size is worked out without a device."""
    lines = [line.strip() for path in glob.glob(os.path.join(CSRC, "*"))
             for line in _code(path).splitlines()
             if re.search(r"\b152\b", line)]
    assert lines == ["constexpr int kPagedMaxSms = 152;"]


@pytest.mark.parametrize("key_len,scale", [(1 << 31, 0.1), (5, 1e39),
                                           (5, "0.1")])
def test_what_the_shapes_cannot_hold_is_refused(key_len, scale):
    """As other arguments out of range, by ValueError."""
    st = (64, 64, 8)
    with pytest.raises(ValueError):
        _lib.pack_attention_shape(1, 1, 1, 4, key_len, 8, 0, scale, st, st,
                                  st, st)
    with pytest.raises(ValueError):
        _lib.pack_attention_backward_shape(1, 1, 1, 4, key_len, 8, 0, scale,
                                           *[st] * 8)
    with pytest.raises(ValueError):
        _lib.pack_paged_shape(1, 1, 1, 8, 16, key_len, 4, 0, scale, st, st,
                              st, st, 4)


def _attention_shape(**kw):
    """A shape of [B, H, S, D] tensors with these members set."""
    s = cs.cs_attention_shape(3, 2, 2, 4, 5, 8, 0, 0.1)
    for name, length in dict(q=4, o=4, k=5, v=5).items():
        setattr(s, name + "_stride",
                (ctypes.c_int64 * 3)(16 * length, 8 * length, 8))
    s.mask_stride = 5
    for name, value in kw.items():
        setattr(s, name, value)
    return s


def _check(s):
    """The status for far-apart fake device addresses."""
    return cs.cs_check_fused_attention_args(
        *(1 << (30 + i) for i in range(6)), s)


def _paged_shape(**kw):
    s = cs.cs_paged_shape(3, 2, 2, 8, 16, 4, 2, 0, 0.1, (16, 8), (16, 8),
                          (256, 16, 8), (256, 16, 8), 2)
    for name, value in kw.items():
        setattr(s, name, value)
    return s


def _check_paged(s):
    return cs.cs_check_paged_attention_args(
        *(1 << (30 + i) for i in range(7)), s, 1 << 40, 1 << 29)


@pytest.mark.parametrize("scale,status", [(0.1, 0), (2.0 ** 127, 0),
                                          (2.0 ** 127.2, 8), (3e38, 8)])
def test_scales_stay_finite_in_base_2(scale, status):
    """A score of 0 is 0 whatever the scale; 0 times an infinite factor is
    NaN."""
    assert _check(_attention_shape(scale=scale)) == status
    assert _check_paged(_paged_shape(scale=scale)) == status


@pytest.mark.parametrize("stride", [1 << 20, 1 << 59, 1 << 61, 1 << 62,
                                    (1 << 63) - 1, -(1 << 62)])
def test_row_strides_do_not_wrap(stride):
    """Strides of a mask's and a table's rows whose products pass 64 bits:
    refused, instead of an extent that has wrapped around."""
    want = 0 if stride == 1 << 20 else 8
    mask = _attention_shape(mask_stride=stride)
    assert cs.cs_check_fused_attention_args(
        *(1 << (30 + i) for i in range(5)), 1 << 36, mask) == want
    assert _check_paged(_paged_shape(table_stride=stride)) == want
