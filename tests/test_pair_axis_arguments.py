"""The axis of each pair as the calls with several-axis positions take it from
Python: any host integers, entry by entry."""
import numpy as np
import pytest
import torch

from fp8_paged_kv_append_gb300 import k16v8 as K
from fp8_paged_kv_append_gb300.rope import rope_pair_axes

AXES = [0] * 16 + [1] * 24 + [2] * 24


@pytest.mark.parametrize("of", [
    list, tuple, bytes, bytearray, lambda a: rope_pair_axes(128, [16, 24, 24]), lambda a: (x for x in a),
    *(lambda a, t=t: np.array(a, t) for t in (np.int8, np.uint8, np.int16, np.int32, np.int64)),
    *(lambda a, t=t: torch.tensor(a, dtype=t) for t in (torch.int8, torch.int32, torch.int64))])
def test_host_integers_of_any_type(of):
    assert K._axes(of(AXES), 64) == bytes(AXES)


@pytest.mark.parametrize("bad", [64, [0.0] * 64, np.zeros(64), [-1] * 64, [256] * 64, None, "0" * 64])
def test_what_is_no_list_of_axes(bad):
    with pytest.raises((TypeError, ValueError)):
        K._axes(bad, 64)


@pytest.mark.parametrize("n", [0, 8, 16, 32, 63, 65])
@pytest.mark.parametrize("t", [np.int8, np.int16, np.int32, np.int64])
def test_an_entry_for_each_pair(n, t):
    with pytest.raises(ValueError, match="64 pairs"):
        K._axes(np.zeros(n, t), 64)
