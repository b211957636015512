"""Mixture weights near 0 and near 1, against the fp64 oracle.  Tolerances as in
test_distill_topk_gpu.py."""
import pytest
import torch

from logits_ops_util import DEV, randn
from rl_fine_tuning_pass_gb300 import binding as rp
from test_distill_topk_gpu import check

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.fixture(scope="module", autouse=True)
def _library():
    from rl_fine_tuning_pass_gb300.build import build
    build()
    rp.load_library()


@pytest.mark.parametrize("beta", [1e-30, 1e-9, 2.0 ** -26, 1e-6, 1e-3, 0.999, 1 - 2.0 ** -20, 1 - 2.0 ** -24])
@pytest.mark.parametrize("tail", [False, True])
def test_weights_near_the_ends(beta, tail):
    """Teacher's tokens that the student gives from nearly all to e^-60 of its mass, and back."""
    x = randn(1, 8, 500, seed=1)
    ids = torch.arange(40, 46).repeat(8, 1)
    for r, gap in enumerate((0.0, 1.0, 5.0, 10.0, 17.0, 25.0, 40.0, 60.0)):
        x[0, r, 40] -= gap
        x[0, r, 41] += gap / 4
    lp = torch.tensor([[0.4, 0.3, 0.1, 0.05, 1e-9, 0.1]]).log().repeat(8, 1)
    check(x.to(DEV), ids, lp, 1.0, beta, tail, what=f"beta={beta}")
