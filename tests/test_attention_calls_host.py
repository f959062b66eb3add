"""Fused and paged attention on the CPU: arguments at the far end of their
ranges, and rules of the sources that no GPU here can show.  No CUDA call is
made."""
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
