"""The scaled frequencies with nothing but the scaling named, against their formulas written out (no GPU)."""
import math

import numpy as np
import pytest
import torch

from w4a8_integer_gemm_b200 import rotary_frequencies


def _plain(rot, base):
    return base ** (-2.0 * np.arange(rot // 2) / rot)


@pytest.mark.parametrize("rot,base,factor,original", [(128, 1e4, 16.0, 4096), (64, 1e4, 4.0, 2048), (128, 1e6, 40.0, 32768)])
def test_yarn_bounds(rot, base, factor, original):
    """Pairs that turn more than 32 times over the original context stay, those below one turn are stretched."""
    f, amp = rotary_frequencies(rot, base, "yarn", factor, original=original)
    g = _plain(rot, base)
    pair = [rot * math.log(original / (n * 2 * math.pi)) / (2 * math.log(base)) for n in (32.0, 1.0)]
    first, last = max(math.floor(pair[0]), 0), min(math.ceil(pair[1]), rot - 1)
    stretch = np.clip((np.arange(rot // 2) - first) / (last - first), 0, 1)
    want = g / factor * stretch + g * (1 - stretch)
    # a few roundings of FP64 each
    assert np.abs(f.numpy() / want - 1).max() < 1e-14 and abs(amp - (0.1 * math.log(factor) + 1)) < 1e-15
    turns = original * g / (2 * math.pi)
    as_is = rotary_frequencies(rot, base)[0]                  # (numpy's power may differ from torch's in the last bit)
    assert ((turns > 32) & (turns < 64)).any() and torch.equal(f[turns > 64], as_is[turns > 64])
    assert torch.equal(f, rotary_frequencies(rot, base, "yarn", factor, original=original, low=1.0, high=32.0)[0])
    assert not torch.equal(f, rotary_frequencies(rot, base, "yarn", factor, original=original, high=4.0)[0])


def test_bands_bounds():
    f, _ = rotary_frequencies(128, 5e5, "bands", 8.0, original=8192)
    assert torch.equal(f, rotary_frequencies(128, 5e5, "bands", 8.0, original=8192, low=1.0, high=4.0)[0])
    g = _plain(128, 5e5)
    turns = 8192 * g / (2 * math.pi)
    keep = np.clip((turns - 1) / 3, 0, 1)
    assert np.abs(f.numpy() / (g * keep + g / 8 * (1 - keep)) - 1).max() < 1e-14


def test_bounds_in_order():
    for scaling in ("bands", "yarn"):
        with pytest.raises(ValueError):
            rotary_frequencies(64, scaling=scaling, low=33.0)
