"""Rows in which a mask leaves nothing: every column -inf, the type's lowest value, or another number so far down
(-2^24 T / log2(e) = -1.2e7 T) that their log-sum-exp in fp32 would have no fraction, and their probabilities no digit.

Such a row has an lse of -inf and no log-prob, and its pair's loss and gradients are NaN; other pairs are not touched.
"""
import pytest
import torch

import rl_fine_tuning_pass_gb300 as rl
from logits_ops_util import DEV, place, randn
from rl_fine_tuning_pass_gb300 import binding as rp

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.fixture(scope="module", autouse=True)
def _library():
    from rl_fine_tuning_pass_gb300.build import build
    build()
    rp.load_library()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("layout", ["dense", "phase"])
@pytest.mark.parametrize("T", [1.0, 0.7, 2.5])
@pytest.mark.parametrize("fill", ["-inf", "lowest", -1e30, -1e9, "mixed"])
def test_rows_of_nothing_but_masked_columns(dtype, layout, T, fill):
    P, L, V = 3, 3, 2603
    low = torch.finfo(dtype).min
    x = (randn(2 * P, L, V, seed=2) * 2).to(dtype)
    x[1, 2] = float("-inf") if fill in ("-inf", "mixed") else low if fill == "lowest" else fill
    if fill == "mixed":
        x[1, 2, ::3], x[1, 2, 1::3] = low, -1e25
    x[0, 1, 5:] = low                               # a few columns are left
    x[2, 0] = -1e3                                  # far down, but within
    idx = torch.zeros(2 * P * L, dtype=torch.int64)
    view, _ = place(x, layout)
    out = rl.preference_loss_fused(view, idx.to(DEV), torch.ones(P, device=DEV), T=T)
    assert float(out["lse"][5]) == float("-inf") and bool(torch.isnan(out["logp"][5]))
    others = [r for r in range(2 * P * L) if r != 5]
    assert bool(torch.isfinite(out["lse"][others]).all()) and bool(torch.isfinite(out["logp"][others]).all())
    assert torch.isnan(out["loss"]).tolist() == [False, True, False]
    nan = torch.isnan(out["dlogits"]).reshape(2 * P, -1)
    assert nan.all(1).tolist() == [False, True, False, False, True, False] and nan.any(1).tolist() == nan.all(1).tolist()
