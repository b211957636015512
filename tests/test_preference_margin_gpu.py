"""The logistic loss of pairs whose margin is large: a function of the margin in two fp32 numbers, not of its rounding.

Both sequences have one token with the same log-prob, so that the margin is beta times the difference of the reference's,
whatever the log-prob's error.  Tolerance: the exponential and the logarithm 2^-23 each, the correction by the margin's
second part and its product 2^-24, the coefficient's two products 2^-24 each: 5 of 2^-23 for either.  (A margin of 32
to 64 rounded to fp32 is up to 1.9e-6 off, and so were these.)
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


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("smoothing", [0.0, 1.0])
def test_large_margins(sign, smoothing):
    P, beta = 256, np.float32(0.1)
    g = np.random.default_rng(4)
    ref = np.concatenate([np.zeros(P), sign * g.uniform(200.0, 700.0, P)]).astype(np.float32)
    x = torch.zeros(2 * P, 1, 2, device=DEV)
    out = rl.preference_loss_fwd(x, torch.zeros(2 * P, dtype=torch.int64, device=DEV), beta=float(beta),
                                 label_smoothing=smoothing, ref_logp=torch.from_numpy(ref).to(DEV))
    h = float(beta) * ref[P:].astype(np.float64)
    z = h if smoothing == 0.0 else -h                        # of the term that is left
    loss, slope = np.logaddexp(0.0, -z), -1.0 / (1.0 + np.exp(z))
    got = out["loss"].double().cpu().numpy()
    assert np.all(np.abs(got - loss) <= 5 * 2.0 ** -23 * loss)
    if z[0] > 0:                                             # else near 1, and no digit is lost
        want = float(beta) * slope * (1 if smoothing == 0.0 else -1)
        coef = out["coef"][:P].double().cpu().numpy()
        if smoothing == 0.0:
            assert np.all(np.abs(coef - want) <= 5 * 2.0 ** -23 * np.abs(want))
        else:                                                # e - sig(-h), a difference from 1
            assert np.all(np.abs(coef - want) <= 5 * 2.0 ** -23 * float(beta))


def test_infinite_margins():
    ref = torch.tensor([0.0, 0.0, float("inf"), float("-inf")], device=DEV)
    x = torch.zeros(4, 1, 2, device=DEV)
    out = rl.preference_loss_fwd(x, torch.zeros(4, dtype=torch.int64, device=DEV), beta=0.5, ref_logp=ref)
    assert out["loss"].tolist() == [0.0, float("inf")]
    assert out["coef"].tolist() == [0.0, -0.5, 0.0, 0.5]      # slopes 0 and -1
