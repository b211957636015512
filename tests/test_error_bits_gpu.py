"""Error bits of the operators next to the row pass through their autograd functions."""
import pytest
import torch

import rl_fine_tuning_pass_gb300 as rl
from logits_ops_util import DEV, randn
from rl_fine_tuning_pass_gb300 import binding as rp

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.fixture(scope="module", autouse=True)
def _library():
    from rl_fine_tuning_pass_gb300.build import build
    build()
    rp.load_library()


def test_rules_through_autograd_report_ids_past_the_vocabulary():
    x = randn(2, 3, 40, seed=1).to(DEV).requires_grad_(True)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    tokens = torch.tensor([[1, 2], [3, 40]], device=DEV)
    rep = torch.tensor([1.2, 1.3], device=DEV)
    y = rl.process_logits(x, tokens=tokens, repetition=rep, dev_err=err)
    assert int(err.item()) == rp.GRPO_DEVERR_IDX_OUT_OF_RANGE
    err.zero_()
    y.sum().backward()                      # the word may change between the passes
    assert int(err.item()) == rp.GRPO_DEVERR_IDX_OUT_OF_RANGE
    err.zero_()
    rl.process_logits(x, tokens=tokens.clamp(max=39), repetition=rep, dev_err=err).sum().backward()
    assert int(err.item()) == 0


def test_distillation_through_autograd_reports_why_a_row_is_nan():
    x = randn(1, 3, 40, seed=1).to(DEV).requires_grad_(True)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ids = torch.tensor([[1, 2], [3, 3], [4, 5]], device=DEV)
    lp = torch.full((3, 2), -1.0, device=DEV)
    loss, _ = rl.distill_topk_loss(x, ids, lp, dev_err=err)
    assert loss.isnan().tolist() == [False, True, False] and int(err.item()) == rp.GRPO_DEVERR_DUPLICATE_ID
    loss.sum().backward()
    assert bool(x.grad[0, 1].isnan().all()) and bool(x.grad[0, [0, 2]].isfinite().all())
    err.zero_()
    ids[1, 0] = 40
    rl.distill_topk_loss(x, ids, lp, dev_err=err)
    assert int(err.item()) == rp.GRPO_DEVERR_IDX_OUT_OF_RANGE
