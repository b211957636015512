"""The gradient of fp32 logits for a log-sum-exp that is given exactly: what the backward's own arithmetic adds.

|g| p_j = 2^t K with t = x_j c - A for a whole number A and c = log2(e) / T rounded.  A t below 16: half a step of
2^-20, times ln 2: 3.3e-7, and 2^-24 of it for c's rounding: 6.6e-7 (what that is of A is in K).  The exponential:
2^-22 = 2.4e-7.  K = |g| 2^(A - lse log2(e) + ...): its exponent half a step of 2^-24 or so, 0.4e-7, the power 2^-22,
the factor and the product 2^-24 each; g itself 2^-23.  In all 1.8e-6 of each element, wherever the logits lie.
"""
import numpy as np
import pytest
import torch

import rl_fine_tuning_pass_gb300 as rl
from logits_ops_util import DEV, f64, place
from rl_fine_tuning_pass_gb300 import binding as rp

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.fixture(scope="module", autouse=True)
def _library():
    from rl_fine_tuning_pass_gb300.build import build
    build()
    rp.load_library()


@pytest.mark.parametrize("T", [1.0, 0.9, 1.3])
@pytest.mark.parametrize("lse", [12.375, -3.5, 1000.375, -517.25])
@pytest.mark.parametrize("out_layout", ["dense", "phase"])
@pytest.mark.parametrize("V", [1003, 4096])
def test_the_exponential_is_taken_near_its_row(T, lse, out_layout, V):
    g = np.random.default_rng(3)
    x = torch.from_numpy((T * (lse - g.uniform(0.0, 11.0, (2, 4, V)))).astype(np.float32)).to(DEV)
    idx = torch.from_numpy(g.integers(0, V, 8)).to(DEV)
    coef, w = torch.tensor([0.5, -0.25], device=DEV), torch.tensor([1.0], device=DEV)
    dx, _ = place(torch.zeros(2, 4, V), out_layout)
    rl.preference_loss_bwd(x, idx, w, coef, torch.full((8,), lse, device=DEV), T=T, dlogits=dx)
    z, factor = f64(x) / T, np.array([0.5] * 4 + [-0.25] * 4) / T
    want = -factor[:, None] * np.exp(z - lse)
    got, other = f64(dx), np.ones((8, V), bool)
    other[np.arange(8), idx.cpu().numpy()] = False      # the tokens' own: sums of the others
    off = np.abs(got - want) / np.abs(want)
    assert off[other].max() <= 1.8e-6, off[other].max()
    total = (np.abs(want) * other).sum(1)
    own = got[~other]
    # a tree of 12 or so additions, half a step each
    assert np.all(np.abs(own - np.sign(factor) * total) <= (1.8e-6 + 16 * 2.0 ** -24) * total)


def test_columns_without_mass():
    """-inf and the type's lowest value in some columns: +0.0 or -0.0 there, and the others as without them."""
    for T in (1.0, 0.9, 1.3):
        x = torch.randn(2, 3, 700, device=DEV)
        idx = torch.zeros(6, dtype=torch.int64, device=DEV)
        coef, w, lse = torch.tensor([0.5, -0.5], device=DEV), torch.ones(1, device=DEV), torch.full((6,), 7.5, device=DEV)
        want = rl.preference_loss_bwd(x, idx, w, coef, lse, T=T)
        y = x.clone()
        y[:, :, 300::2], y[:, :, 301::2] = float("-inf"), torch.finfo(torch.float32).min
        got = rl.preference_loss_bwd(y, idx, w, coef, lse, T=T)
        assert bool((got[:, :, 300:] == 0).all()) and bool((got[:, :, 1:300] == want[:, :, 1:300]).all())
