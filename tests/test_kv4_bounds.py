"""The bounds of test_gpu_kv4_weights.py see the mistakes that they are for, planted on the CPU."""
import math

import pytest
import torch


@pytest.mark.parametrize("n", [2, 129, 777, 4096, 12000, 20011])
def test_a_lost_or_doubled_key_shows(n):
    """Equal weights, one key left out or taken twice: the log-sum-exp leaves its bound, and up to 12000 tokens so does
    the output at the key's channel (of 128), rounded to bf16."""
    for wrong in (n - 1, n + 1):
        assert abs(math.log(wrong) - math.log(n)) > 2 * 4 * 2.0 ** -24 * math.log(n)
        if n > 12000:
            continue
        count = (n + 127) // 128
        got = float(torch.tensor((count + wrong - n) / wrong).bfloat16()) * n
        assert abs(got - count) > (2.0 ** -8 + 2.0 ** -22) * count


def test_weights_of_8_bits_show():
    """One pair: weights of 1 and 1 - 3 * 2^-10, opposite values.  Rounded to bf16 they leave an error far over the bound,
    with the remainder added one far below it."""
    e = torch.tensor([1.0, 1.0 - 3 * 2.0 ** -10])
    hi = e.bfloat16().float()
    lo = (e - hi).bfloat16().float()
    total, bound = float(e.sum()), 1.01 * 2.0 ** -16 + 2.0 ** -18
    exact = float(e[0] - e[1]) / total
    bound += 2.0 ** -8 * exact
    assert abs(float(hi[0] - hi[1]) / total - exact) > 10 * bound
    assert abs(float(hi[0] - hi[1] + lo[0] - lo[1]) / total - exact) < bound / 3
