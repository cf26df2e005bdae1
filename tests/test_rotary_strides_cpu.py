"""Outputs of qk_norm_rope and its gradient whose rows overlap are refused, all others are
taken: the check of the strides against every row's place.  No GPU."""
from __future__ import annotations

import itertools
import random

import pytest
import torch

from io_aware_attention_fwd_gb300.rotary import _strides

D = 4


def overlap(strides, counts):
    """Whether two rows of D elements at these strides share an element."""
    at = sorted(sum(i * s for i, s in zip(x, strides)) for x in itertools.product(*(range(n) for n in counts)))
    return any(b - a < D for a, b in zip(at, at[1:]))


def refused(strides, counts):
    try:
        assert _strides((*strides, 1), (*counts, D), "x", True) == tuple(0 if n < 2 else s for s, n in zip(strides, counts))
    except ValueError:
        return True
    return False


def test_every_small_layout():
    some = [0, 0]
    for counts in itertools.product((1, 2, 3), repeat=3):
        for strides in itertools.product((0, 2, 4, 6, 8, 12, 20), repeat=3):
            want = overlap(strides, counts)
            assert refused(strides, counts) == want, (strides, counts)
            some[want] += 1
    assert min(some) > 1000


def test_random_layouts():
    rng = random.Random(5)
    some = [0, 0]
    for _ in range(4000):
        counts = [rng.choice((1, 2, 3, 5, 8)) for _ in range(3)]
        strides = [rng.randrange(0, rng.choice((10, 40, 200))) for _ in range(3)]
        want = overlap(strides, counts)
        assert refused(strides, counts) == want, (strides, counts)
        some[want] += 1
    assert min(some) > 300


@pytest.mark.parametrize("make", [
    lambda: torch.empty(2, 5, 3, D), lambda: torch.empty(2, 3, 5, D).transpose(1, 2), lambda: torch.empty(5, 2, 3, D).transpose(0, 1),
    lambda: torch.empty(3, 5, 2, D).permute(2, 1, 0, 3), lambda: torch.empty(2, 5, 9, D)[:, :, 2:5], lambda: torch.empty(2, 5, 3, 2 * D)[..., :D],
    lambda: torch.empty(2, 10, 3, D)[:, ::2], lambda: torch.empty(5, 3, D), lambda: torch.empty(3, 5, D).transpose(0, 1),
    lambda: torch.empty(0, 3, D), lambda: torch.empty(2, 0, 3, D),
], ids=str)
def test_views_of_tensors_are_taken(make):
    x = make()
    _strides(x.stride(), x.shape, "x", True)


@pytest.mark.parametrize("make", [
    lambda: torch.empty(2, 1, 3, D).expand(2, 5, 3, D), lambda: torch.empty(2, 5, 1, D).expand(2, 5, 3, D),
    lambda: torch.empty(1, 5, 3, D).expand(2, 5, 3, D), lambda: torch.empty(100).as_strided((5, 3, D), (D, D, 1)),
    lambda: torch.empty(100).as_strided((5, 3, D), (3 * D, D // 2, 1)), lambda: torch.empty(200).as_strided((2, 5, 3, D), (D * 14, D * 3, D, 1)),
])
def test_rows_that_overlap_are_refused(make):
    x = make()
    with pytest.raises(ValueError, match="apart"):
        _strides(x.stride(), x.shape, "x", True)
    _strides(x.stride(), x.shape, "x")  # inputs may be broadcast
