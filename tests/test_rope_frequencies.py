"""Frequencies of stretched contexts ("by_parts") against their definition, pair by pair."""
import math

import pytest
import torch

import exact_headdim_attention_gb300 as pkg


def by_parts(rot, base, length, factor, fast, slow):
    """Pair numbers whose angle turns `fast` and `slow` times within `length`, widened to whole pairs;
    what lies between goes linearly from the frequency to the frequency / factor."""
    def number(times):
        return rot * math.log(length / (2 * math.pi * times)) / (2 * math.log(base))

    start, end = max(0, math.floor(number(fast))), min(rot - 1, math.ceil(number(slow)))
    out = []
    for i in range(rot // 2):
        f = base ** (-2 * i / rot)
        part = 0.0 if i <= start else 1.0 if i >= end else (i - start) / (end - start)
        out.append((1 - part) * f + part * f / factor)
    return torch.tensor(out, dtype=torch.float64)


@pytest.mark.parametrize("rot,base,length,factor", [
    (64, 1e4, 131072, 4.0), (64, 1e4, 62832, 4.0), (64, 1e4, 4096, 8.0), (128, 5e5, 8192, 32.0), (128, 1e4, 1 << 20, 2.0),
    (64, 100.0, 4096, 8.0), (512, 1e4, 32768, 16.0), (8, 1e4, 300, 4.0), (64, 1e4, 1 << 17, 1.0)])
@pytest.mark.parametrize("fast,slow", [(32.0, 1.0), (8.0, 4.0)])
def test_by_parts(rot, base, length, factor, fast, slow):
    inv, scale = pkg.rope_inv_freq(rot, base, scaling="by_parts", factor=factor, original_length=length, beta_fast=fast, beta_slow=slow)
    # 64-bit powers, products and sums: each off by 2^-52 or so
    assert torch.allclose(inv, by_parts(rot, base, length, factor, fast, slow), rtol=1e-13, atol=0)
    assert scale == pytest.approx(0.1 * math.log(factor) + 1, abs=1e-15)


def test_by_parts_of_a_context_that_the_last_pair_turns_in():
    """131072 positions, base 10000: the last of 32 pairs turns 2.8 times, more than beta_slow = 1, and
    lies 9 of 13 pairs into the ramp (22 to 35)."""
    inv, _ = pkg.rope_inv_freq(64, scaling="by_parts", factor=4.0, original_length=131072)
    plain, _ = pkg.rope_inv_freq(64)
    assert 131072 * plain[-1] / (2 * math.pi) > 2.7
    assert (inv / plain)[-1].item() == pytest.approx(1 - 9 / 13 * 3 / 4, rel=1e-12)
    assert (inv / plain > 1 / 4).all()


def test_by_parts_of_a_context_that_no_pair_turns_in():
    """Every pair turns less than beta_slow times: each is divided by the whole factor."""
    inv, _ = pkg.rope_inv_freq(64, scaling="by_parts", factor=4.0, original_length=512, beta_fast=400.0, beta_slow=100.0)
    assert torch.allclose(inv, pkg.rope_inv_freq(64)[0] / 4, rtol=1e-14, atol=0)
