"""grad_norm where what a rounding of the sum loses is not to be had from one subtraction: a spike after small
elements, and sums outside fp32's range.

A thread's sum is within 7e-11 of the squares' (the sum of what its roundings lose is itself rounded, up to k 2^-48 of
at most 64 of the largest square at the k-th of sixteen pairs), what adds the threads' sums below 1e-12, and
the norm within half of that; sums out of range are within 2^-32 (32 squares, one by one).  So a norm that is 3e-10 from
the middle of two fp32 numbers goes to the nearer one.
"""
import numpy as np
import pytest
import torch

import rl_fine_tuning_pass_gb300 as rl
from logits_ops_util import DEV
from rl_fine_tuning_pass_gb300 import binding as rp

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.fixture(scope="module", autouse=True)
def _library():
    from rl_fine_tuning_pass_gb300.build import build
    build()
    rp.load_library()


def near_a_middle(x, side):
    """x (bf16 numbers, multiples of 2^-11, whose squares add up exactly in 64 bits) and a few more elements, so that the
    norm is 3e-10 above (side 1) or below (-1) the middle of two fp32 numbers; and the nearer of those."""
    total = float((x * x).sum())
    f = np.nextafter(np.float32(np.sqrt(total)), np.float32(np.inf))
    above = np.nextafter(f, np.float32(np.inf))
    middle = (float(f) + float(above)) / 2
    rest, few = (middle * (1 + side * 3e-10)) ** 2 - total, []
    for _ in range(8):                                # each leaves less than 2^-6 of the rest
        g = torch.tensor(np.sqrt(max(rest, 0.0))).bfloat16()
        if float(g) ** 2 > rest:
            g = (g.view(torch.int16) - 1).view(torch.bfloat16)
        few.append(float(g))
        rest -= few[-1] ** 2
        if rest < 1e-12 * total:
            break
    exact = float(np.sqrt(total + sum(v * v for v in few)))
    assert abs(exact / middle - 1 - side * 3e-10) < 1e-11
    return [torch.tensor(v, dtype=torch.float64).bfloat16().to(DEV) for v in (x, few)], float(above if side > 0 else f)


def check(x, side, dtype, scale=1.0):
    grads, want = near_a_middle(x, side)
    got = float(rl.grad_norm([(g.double() * scale).to(dtype) for g in grads]))
    assert got == want * scale, (got / scale, want)


def numbers(r, n, low, high):
    return r.integers(128, 256, n) * 2.0 ** r.integers(low, high, n) * np.where(r.random(n) < 0.5, -1, 1)


@pytest.mark.parametrize("n", [1 << 16, 1 << 20])     # one launch of a cluster, and the larger form
@pytest.mark.parametrize("side", [1, -1])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_spikes_after_small_elements(n, side, dtype):
    for seed in range(8):
        r = np.random.default_rng(seed)
        x = numbers(r, n, -11, -8)
        spike = (r.random(n) < 1 / 64) & (np.arange(n) % 8192 >= 2048)   # behind a thread's first elements
        x[spike] = numbers(r, n, 0, 3)[spike]
        check(x, side, dtype)


@pytest.mark.parametrize("side", [1, -1])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_elements_in_any_order(side, dtype):
    for seed in range(6):
        check(numbers(np.random.default_rng(seed), 1 << 18, -11, -2), side, dtype)


@pytest.mark.parametrize("scale", [2.0 ** 60, 2.0 ** -60, 2.0 ** 90, 2.0 ** -100])
@pytest.mark.parametrize("side", [1, -1])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_sums_outside_the_range(scale, side, dtype):
    for seed in range(6):
        check(numbers(np.random.default_rng(seed), 1 << 18, -11, -2), side, dtype, scale)
