"""Stretched frequencies of rotary positions at the ends of their ramp.  CPU only."""
import math

import pytest
import torch

import gated_delta_rule_32_gb300 as pkg


@pytest.mark.parametrize("part", [2, 8, 64, 128])
@pytest.mark.parametrize("trained", [1, 4, 6, 7, 64, 4096, 10 ** 9, 10 ** 14])
@pytest.mark.parametrize("fast,slow", [(32.0, 1.0), (2.0, 1.9), (1e4, 1e-2)])
def test_slow_pairs_are_divided_and_fast_ones_kept(part, trained, fast, slow):
    f, _ = pkg.rotary_frequencies(part, device="cpu")
    g, amp = pkg.rotary_frequencies(part, scaling="yarn", factor=4.0, trained=trained, fast=fast,
                                    slow=slow, device="cpu")
    turns = trained * f / (2 * math.pi)
    r = g / f
    assert math.isclose(amp, 0.1 * math.log(4.0) + 1)
    assert ((r >= 0.25 - 1e-12) & (r <= 1 + 1e-12)).all() and (r.diff() <= 1e-12).all()
    # (the ramp runs over whole indices: a pair beside its ends may be on it)
    i = torch.arange(part // 2)
    assert torch.allclose(r[turns >= fast], torch.ones(1, dtype=torch.float64))
    ramp_ends = math.ceil(part * math.log(trained / (2 * math.pi * slow)) / (2 * math.log(10000.0)))
    assert torch.allclose(r[(turns <= slow) & (i >= ramp_ends)], torch.tensor(0.25, dtype=torch.float64))
    if ramp_ends <= 0:
        assert torch.allclose(r, torch.tensor(0.25, dtype=torch.float64))
