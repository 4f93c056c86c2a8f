"""The stretched frequency tables against their definitions, pair by pair in
fp64, over the range of head sizes, bases and trained lengths."""
import math

import pytest
import torch

import paged_kv_decode_31_b200 as pkv


def _blend(r, base, factor, trained, fast, slow):
    """Interpolation by parts: with d(n) = r ln(trained / (2 pi n)) / (2 ln base)
    the pair index that turns n times within `trained`, a ramp from floor d(fast)
    to ceil d(slow), these held to [0, r - 1]."""
    def index(n):
        return r * math.log(trained / (2 * math.pi * n)) / (2 * math.log(base))

    lo, hi = max(math.floor(index(fast)), 0), min(math.ceil(index(slow)), r - 1)
    table = []
    for i in range(r // 2):
        f = base ** (-2.0 * i / r)
        if hi > lo:
            part = min(max((i - lo) / (hi - lo), 0.0), 1.0)
        else:  # every pair turns more than `fast` times
            part = 0.0
        table.append(f * (1 - part) + f / factor * part)
    return table


@pytest.mark.parametrize("r", [16, 32, 48, 64, 96, 128])
@pytest.mark.parametrize("base", [1e4, 5e5, 1e6])
@pytest.mark.parametrize("factor,fast,slow", [(4.0, 32.0, 1.0), (32.0, 32.0, 1.0), (8.0, 16.0, 2.0)])
def test_blend(r, base, factor, fast, slow):
    for trained in [64, 100, 512] + [1 << k for k in range(10, 21)]:
        f, m = pkv.rope_frequencies(r, base, scaling="blend", factor=factor, original_max=trained, fast=fast,
                                    slow=slow)
        want = _blend(r, base, factor, trained, fast, slow)
        assert m == 0.1 * math.log(factor) + 1
        for i, (got, w) in enumerate(zip(f.tolist(), want)):
            assert abs(got - w) <= (2.0 ** -24 + 2.0 ** -40) * w, (trained, i, got / w)
            turns = trained * base ** (-2.0 * i / r) / (2 * math.pi)
            if turns <= slow:
                assert abs(got * factor * base ** (2.0 * i / r) - 1) <= 2.0 ** -23
            if turns >= fast:
                assert abs(got * base ** (2.0 * i / r) - 1) <= 2.0 ** -23


def test_blend_where_the_last_pair_still_turns():
    """131072 positions turn the last of 64 pairs 2.4 times: more than `slow`, so
    it keeps a part of its frequency."""
    f, _ = pkv.rope_frequencies(128, scaling="blend", factor=4.0, original_max=131072)
    plain, _ = pkv.rope_frequencies(128)
    assert 0.4 < float(f[-1] / plain[-1]) < 0.5


def test_blend_where_no_pair_turns():
    """A trained length within one turn of the fastest pair: all are stretched."""
    f, _ = pkv.rope_frequencies(32, scaling="blend", factor=4.0, original_max=5)
    plain, _ = pkv.rope_frequencies(32)
    assert torch.equal(f, plain / 4)
